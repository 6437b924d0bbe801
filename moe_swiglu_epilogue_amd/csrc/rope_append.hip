// Rotation of q and k, and the write of k and v into the paged NVFP4 cache
// (include/nvfp4_sparse.h).
//
// A workgroup takes a token. Its first threads look up the token's angles, a
// cosine and sine for each pair, and put them into LDS; then every thread owns
// 8 dimensions, the same for every head that it takes, keeps their cosines and
// signed sines in registers and walks over the heads of q, k and v:
//   out[d] = x[d] c[d] + x[partner of d] s[d],
// a product, a product and a sum in binary32, each rounded, as the definition
// has them. A block of 16 values of k or v is two
// neighbouring lanes', which exchange their largest magnitudes and quantize
// eight values each.
#include "nvfp4_device.hpp"
#include "serving_common.hpp"
#include "nvfp4_sparse.h"

namespace {

constexpr int kThreads = 256;
constexpr int kMostPairs = 256;

typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

struct Append {
    const uint16_t *q, *k, *v;
    uint16_t* q_out;
    const int32_t *positions, *pair_axis;
    const float* cos_sin;
    const float *k_gs, *v_gs;
    const int64_t* slots;
    uint8_t *kp, *ks, *vp, *vs;
    int64_t ld_q, ld_k, ld_v, ld_out, ld_positions, num_slots;
    int tokens, heads, kv_heads, dim, rot, axes, max_position, parts;
};

// How pairs lie: (j, j + rot / 2) with rot / 2 a multiple of 8, so that the
// partners of a thread's 8 dimensions are 8 in a row too; the same with any
// rot; (2 j, 2 j + 1).
enum Pairs { kHalves8, kHalves, kNeighbours };

__device__ __forceinline__ void widen(uint4v w, float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = nvfp4::bf16_lo(w[i]);
        x[2 * i + 1] = nvfp4::bf16_hi(w[i]);
    }
}

// Eight values of a block of 16, whose other half the neighbouring lane holds, to
// their codes; the exact path of nvfp4::half_steps16.
__device__ __forceinline__ uint32_t quantize8(const float (&y)[8], const nvfp4::RowScale& rs, uint32_t& sf)
{
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        amax = __builtin_elementwise_maximum(amax, __builtin_fabsf(y[j]));
    // the lane next to this one (lane ^ 1)
    const float other = __uint_as_float(
        (uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(amax), 0xb1, 0xf, 0xf, true));
    amax = __builtin_elementwise_maximum(amax, other);
    const nvfp4::BlockScale s = nvfp4::block_scale<false>(amax, rs);
    float h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        h[j] = nvfp4::half_steps(y[j], s);
    if (amax * s.rcp > 16.0f) {
        const float lim = 16.0f * s.half_d;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            h[j] = nvfp4::half_steps(__builtin_amdgcn_fmed3f(y[j], -lim, lim), s);
    }
    sf = s.sf;
    uint32_t w = 0;
    w = nvfp4::pack_e2m1<0>(w, h[0], h[1]);
    w = nvfp4::pack_e2m1<1>(w, h[2], h[3]);
    w = nvfp4::pack_e2m1<2>(w, h[4], h[5]);
    w = nvfp4::pack_e2m1<3>(w, h[6], h[7]);
    return w;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    const bf2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

template <Pairs kPairs>
__global__ __launch_bounds__(kThreads) void rope_append_kernel(Append a)
{
    __shared__ float cosines[kMostPairs], sines[kMostPairs];
    __shared__ bool turns[kMostPairs];
    const int half = a.rot / 2;
    const int per_head = a.dim / 8;                 // threads of a head, at most 64
    const int at_once = kThreads / per_head;        // heads that the workgroup takes at once
    const int d0 = threadIdx.x % per_head * 8;
    const int mine = threadIdx.x / per_head;
    const int part = blockIdx.x % a.parts;
    const int units = a.heads + 2 * a.kv_heads;
    const nvfp4::RowScale k_scale = nvfp4::row_scale(a.k_gs ? a.k_gs[0] : 1.0f);
    const nvfp4::RowScale v_scale = nvfp4::row_scale(a.v_gs ? a.v_gs[0] : 1.0f);

    for (int64_t t = blockIdx.x / a.parts; t < a.tokens; t += gridDim.x / a.parts) {
        __syncthreads();
        if ((int)threadIdx.x < half) {
            const int j = threadIdx.x;
            const int axis = a.pair_axis ? a.pair_axis[j] : 0;
            const bool known = axis >= 0 && axis < a.axes;
            const int p = known ? a.positions[axis * a.ld_positions + t] : -1;
            const bool in = p >= 0 && p < a.max_position;
            turns[j] = in;
            if (in) {
                cosines[j] = a.cos_sin[(int64_t)p * a.rot + j];
                sines[j] = a.cos_sin[(int64_t)p * a.rot + half + j];
            }
        }
        __syncthreads();
        if (mine >= at_once)
            continue;
        float c[8], s[8];
        bool turn[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int d = d0 + i;
            const bool second = kPairs == kNeighbours ? i & 1 : d >= half;
            const int j = kPairs == kNeighbours ? d >> 1 : second ? d - half : d;
            turn[i] = d < a.rot && turns[j];
            c[i] = turn[i] ? cosines[j] : 1.0f;
            s[i] = turn[i] ? second ? sines[j] : -sines[j] : 0.0f;
        }
        const int64_t slot = a.slots[t];
        const bool stored = slot >= 0 && slot < a.num_slots;
        for (int unit = part * at_once + mine; unit < units; unit += a.parts * at_once) {
            const bool is_q = unit < a.heads, is_v = unit >= a.heads + a.kv_heads;
            const int h = is_q ? unit : is_v ? unit - a.heads - a.kv_heads : unit - a.heads;
            if (!is_q && !stored)
                continue;
            const uint16_t* head = is_q ? a.q + t * a.ld_q : is_v ? a.v + t * a.ld_v : a.k + t * a.ld_k;
            head += h * a.dim;
            float y[8];
            const uint4v w = *(const uint4v*)(head + d0);
            widen(w, y);
            if (!is_v) {
                float x[8];
                if (kPairs == kNeighbours) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        x[i] = y[i ^ 1];
                } else if (kPairs == kHalves8) {
                    const int at = d0 < half ? d0 + half : d0 < a.rot ? d0 - half : d0;
                    widen(*(const uint4v*)(head + at), x);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int d = d0 + i;
                        const int at = d < half ? d + half : d < a.rot ? d - half : d;
                        x[i] = __uint_as_float((uint32_t)head[at] << 16);
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    y[i] = turn[i] ? y[i] * c[i] + x[i] * s[i] : y[i];
            }
            if (is_q) {
                *(uint4v*)(a.q_out + t * a.ld_out + h * a.dim + d0) =
                    uint4v{bf16x2(y[0], y[1]), bf16x2(y[2], y[3]), bf16x2(y[4], y[5]), bf16x2(y[6], y[7])};
            } else {
                uint32_t sf;
                const uint32_t codes = quantize8(y, is_v ? v_scale : k_scale, sf);
                const int64_t at = slot * a.kv_heads * (a.dim / 16) + h * (a.dim / 16);
                *(uint32_t*)((is_v ? a.vp : a.kp) + at * 8 + d0 / 2) = codes;
                if ((d0 & 8) == 0)
                    (is_v ? a.vs : a.ks)[at + d0 / 16] = (uint8_t)sf;
            }
        }
    }
}

}  // namespace

extern "C" nvfp4_status_t nvfp4_rope_append(
    const uint16_t* q, int64_t tokens, int64_t ld_q, int32_t heads, const uint16_t* k, int64_t ld_k,
    const uint16_t* v, int64_t ld_v, int32_t kv_heads, int32_t head_dim, const int32_t* positions,
    int64_t ld_positions, int32_t num_axes, const int32_t* pair_axis, const float* cos_sin,
    int64_t max_position, int32_t rot_dim, int32_t interleaved, const float* k_gs, const float* v_gs,
    const int64_t* slots, int64_t num_slots, uint8_t* k_packed, uint8_t* k_scales, uint8_t* v_packed,
    uint8_t* v_scales, uint16_t* q_out, int64_t ld_out, hipStream_t stream)
{
    using namespace serving;
    if (tokens < 0 || kv_heads < 1 || head_dim < 1 || (q && heads < 1) || num_axes < 1 || max_position < 0 ||
        rot_dim < 0 || rot_dim > head_dim || num_slots < 0)
        return NVFP4_ERROR_INVALID_VALUE;
    if (!q)
        heads = 0;
    if (head_dim % 16 != 0 || head_dim > 512 || rot_dim % 2 != 0 || num_axes > 16 || heads > 1024 ||
        kv_heads > 1024 || tokens > INT32_MAX || max_position > INT32_MAX)
        return NVFP4_ERROR_UNSUPPORTED_SHAPE;
    const int64_t cols = (int64_t)heads * head_dim, kv_cols = (int64_t)kv_heads * head_dim;
    if (ld_k < kv_cols || ld_v < kv_cols || !extent_ok(tokens, ld_k, 2) || !extent_ok(tokens, ld_v, 2) ||
        (q && (ld_q < cols || ld_out < cols || !extent_ok(tokens, ld_q, 2) || !extent_ok(tokens, ld_out, 2))) ||
        (num_axes > 1 && ld_positions < tokens) || !extent_ok(num_slots, kv_cols, 1) ||
        (num_axes > 1 && !extent_ok(num_axes, ld_positions, 4)))
        return NVFP4_ERROR_INVALID_VALUE;
    if (tokens == 0)
        return NVFP4_SUCCESS;
    if (!k || !v || !slots || (q && !q_out) || (rot_dim > 0 && (!positions || (max_position > 0 && !cos_sin))) ||
        (num_slots > 0 && (!k_packed || !k_scales || !v_packed || !v_scales)))
        return NVFP4_ERROR_INVALID_VALUE;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(cos_sin, 16) ||
        !aligned(slots, 8) || !aligned(k_packed, 8) || !aligned(v_packed, 8) || !aligned(positions, 4) ||
        !aligned(pair_axis, 4) || !aligned(k_gs, 4) || !aligned(v_gs, 4) || ld_k % 8 != 0 || ld_v % 8 != 0 ||
        (q && (ld_q % 8 != 0 || ld_out % 8 != 0)))
        return NVFP4_ERROR_MISALIGNED;
    // a partner may be read behind the write of its turned value
    const int64_t out_bytes = q ? 2 * ((tokens - 1) * ld_out + cols) : 0;
    if (overlap(q_out, out_bytes, q, q ? 2 * ((tokens - 1) * ld_q + cols) : 0) ||
        overlap(q_out, out_bytes, k, 2 * ((tokens - 1) * ld_k + kv_cols)) ||
        overlap(q_out, out_bytes, v, 2 * ((tokens - 1) * ld_v + kv_cols)) ||
        overlap(k_packed, num_slots * (kv_cols / 2), v_packed, num_slots * (kv_cols / 2)) ||
        overlap(k_scales, num_slots * (kv_cols / 16), v_scales, num_slots * (kv_cols / 16)))
        return NVFP4_ERROR_INVALID_VALUE;
    Append a = {q, k, v, q_out, positions, pair_axis, cos_sin, k_gs, v_gs, slots, k_packed, k_scales,
                v_packed, v_scales, q ? ld_q : 0, ld_k, ld_v, q ? ld_out : 0, num_axes > 1 ? ld_positions : 0,
                num_slots, (int)tokens, heads, kv_heads, head_dim, rot_dim, num_axes, (int)max_position, 1};
    // Few tokens: the heads of one are split over workgroups, each of which takes
    // its share at once.
    const int at_once = kThreads / (head_dim / 8), all = ceil_div(heads + 2 * kv_heads, at_once);
    if (tokens * all <= 4096)
        a.parts = all;
    // workgroups beyond 2^22 loop over the tokens (a grid holds less than 2^32 threads)
    const int64_t most = (1 << 22) / a.parts;
    const dim3 grid((unsigned)((tokens < most ? tokens : most) * a.parts));
    if (interleaved)
        hipLaunchKernelGGL((rope_append_kernel<kNeighbours>), grid, dim3(kThreads), 0, stream, a);
    else if (rot_dim % 16 == 0)
        hipLaunchKernelGGL((rope_append_kernel<kHalves8>), grid, dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((rope_append_kernel<kHalves>), grid, dim3(kThreads), 0, stream, a);
    return launched();
}
