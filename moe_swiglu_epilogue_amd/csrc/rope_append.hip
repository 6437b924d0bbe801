// Rotation of q and k, and the write of k and v into the paged NVFP4 cache
// (include/nvfp4_sparse.h).
//
// A workgroup takes some tokens. Its threads look up their angles, a cosine and sine
// for each pair, and put them into LDS; then every thread owns 8 or 16 dimensions
// and walks over the tokens and their heads of q, k and v:
//   out[d] = x[d] c[d] + x[partner of d] s[d]     (s: the sine with its sign),
// a product, a product and a sum in binary32, each rounded, as the definition
// has them. A block of 16 values of k or v is two neighbouring lanes', which
// exchange their largest magnitudes and quantize eight values each.
//
// Bound by memory traffic for long prompts, which needs many loads on their way: the
// rows of several heads are requested at once, the first of them in front of the
// angles. Every value is read once and q is written once, so both pass the caches
// by (non-temporal). 16384 tokens of 64/8 heads of 128: 104 us, 6.1 TB/s, where a
// hand-written copy reaches 6.2; 256 tokens 6.1 us, one 3.9: the start and the chain
// position, angles, rotation.
#include "nvfp4_device.hpp"
#include "serving_common.hpp"
#include "nvfp4_sparse.h"

namespace {

constexpr int kThreads = 256;
constexpr int kMostPairs = 256, kMostTokens = 4;

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
    int tokens, heads, kv_heads, dim, rot, axes, max_position;
    int together, parts;       // tokens of a workgroup, or workgroups of a token
};

// How pairs lie: (j, j + rot / 2), with rot = dim a multiple of 32, so that a thread
// takes 8 dimensions and their 8 partners; with rot / 2 a multiple of 8, so that the
// partners of a thread's 8 dimensions are 8 in a row too, which it reads as well; with
// any rot; (2 j, 2 j + 1).
enum Pairs { kWhole, kHalves8, kHalves, kNeighbours };

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

// What a thread loads of a head: its 8 dimensions, and for pairs in halves their
// partners.
template <Pairs kPairs>
struct Row {
    static constexpr int kWords = kPairs == kNeighbours || kPairs == kHalves ? 1 : 2;
    uint4v w[kWords];
};

// The heads of a token, q's, k's and v's one after the other.
__device__ __forceinline__ const uint16_t* head_of(const Append& a, int64_t t, int unit)
{
    return unit < a.heads ? a.q + t * a.ld_q + unit * a.dim
           : unit < a.heads + a.kv_heads ? a.k + t * a.ld_k + (unit - a.heads) * a.dim
                                         : a.v + t * a.ld_v + (unit - a.heads - a.kv_heads) * a.dim;
}

// partner: where the 8 partners begin, less than 0 where there are none.
template <Pairs kPairs>
__device__ __forceinline__ void load_row(Row<kPairs>& r, const uint16_t* head, int d0, int partner)
{
    r.w[0] = __builtin_nontemporal_load((const uint4v*)(head + d0));
    if (kPairs == kWhole)
        r.w[Row<kPairs>::kWords - 1] = __builtin_nontemporal_load((const uint4v*)(head + partner));
    if (kPairs == kHalves8 && partner >= 0)
        r.w[Row<kPairs>::kWords - 1] = *(const uint4v*)(head + partner);
}

// The angles of a thread's 8 dimensions, a bit for each that turns.
struct Angles {
    float c[8], s[8];
    uint32_t turn;
};

struct Turns {
    __align__(16) float c[kMostTokens * kMostPairs], s[kMostTokens * kMostPairs];
    __align__(16) uint8_t in[kMostTokens * kMostPairs];
    int64_t slot[kMostTokens];
};

// From the pairs' angles of a token, which begin at `at`.
template <Pairs kPairs>
__device__ __forceinline__ Angles angles_of(const Turns& lds, int at, int d0, int half, int rot)
{
    Angles g;
    g.turn = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = d0 + i;
        const bool second = kPairs == kNeighbours ? i & 1 : kPairs != kWhole && d >= half;
        const int j = at + (kPairs == kNeighbours ? d >> 1 : second ? d - half : d);
        const bool inside = kPairs == kWhole || d < rot;
        const float s = inside ? lds.s[j] : 0.0f;
        g.c[i] = inside ? lds.c[j] : 1.0f;
        g.s[i] = second ? s : -s;
        g.turn |= inside && lds.in[j] ? 1u << i : 0;
    }
    return g;
}

struct Scales {
    nvfp4::RowScale k, v;
};

__device__ __forceinline__ void write_row(const Append& a, const Scales& scales, int64_t t, int64_t slot, int unit, int d,
                                          const float (&z)[8])
{
    if (unit < a.heads) {
        __builtin_nontemporal_store(
            uint4v{bf16x2(z[0], z[1]), bf16x2(z[2], z[3]), bf16x2(z[4], z[5]), bf16x2(z[6], z[7])},
            (uint4v*)(a.q_out + t * a.ld_out + unit * a.dim + d));
        return;
    }
    const bool is_v = unit >= a.heads + a.kv_heads;
    const int h = unit - a.heads - (is_v ? a.kv_heads : 0);
    uint32_t sf;
    const nvfp4::RowScale rs = {is_v ? scales.v.gs : scales.k.gs, is_v ? scales.v.k : scales.k.k,
                                is_v ? scales.v.rk : scales.k.rk, is_v ? scales.v.pow2 : scales.k.pow2};
    const uint32_t codes = quantize8(z, rs, sf);
    const int64_t at = (slot * a.kv_heads + h) * (a.dim / 16);
    *(uint32_t*)((is_v ? a.vp : a.kp) + at * 8 + d / 2) = codes;
    if ((d & 8) == 0)
        (is_v ? a.vs : a.ks)[at + d / 16] = (uint8_t)sf;
}

template <Pairs kPairs>
__device__ __forceinline__ void turn_row(const Append& a, const Scales& scales, const Angles& g, const Row<kPairs>& r,
                                         int64_t t, int64_t slot, int unit, int d0, int half)
{
    float y[8], x[8];                                     // its dimensions and their partners
    widen(r.w[0], y);
    if (unit < a.heads + a.kv_heads && g.turn != 0) {
        if (kPairs == kWhole || kPairs == kHalves8) {
            widen(r.w[Row<kPairs>::kWords - 1], x);
        } else if (kPairs == kNeighbours) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = y[i ^ 1];
        } else {
            const uint16_t* head = head_of(a, t, unit);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int d = d0 + i, at = d < half ? d + half : d < a.rot ? d - half : d;
                x[i] = __uint_as_float((uint32_t)head[at] << 16);
            }
        }
        const bool all = g.turn == 255;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float z = y[i] * g.c[i] + x[i] * g.s[i], o = x[i] * g.c[i] + y[i] * -g.s[i];
            x[i] = all || g.turn >> i & 1 ? o : x[i];
            y[i] = all || g.turn >> i & 1 ? z : y[i];
        }
    } else if (kPairs == kWhole) {
        widen(r.w[Row<kPairs>::kWords - 1], x);
    }
    write_row(a, scales, t, slot, unit, d0, y);
    if (kPairs == kWhole)
        write_row(a, scales, t, slot, unit, d0 + half, x);
}

template <Pairs kPairs>
__global__ __launch_bounds__(kThreads) void rope_append_kernel(Append a)
{
    constexpr int kAhead = 2;                             // heads that a thread has in flight
    __shared__ Turns lds;
    const int half = a.rot / 2;
    const int per_head = a.dim / (kPairs == kWhole ? 16 : 8);     // threads of a head, at most 64
    const int at_once = kThreads / per_head;              // heads that the workgroup takes at once
    const int d0 = threadIdx.x % per_head * 8;
    const int mine = threadIdx.x / per_head;
    const int units = a.heads + 2 * a.kv_heads, step = a.parts * at_once;
    const int partner = kPairs == kWhole || d0 < half ? d0 + half : d0 < a.rot ? d0 - half : -1;
    const Scales scales = {nvfp4::row_scale(a.k_gs ? a.k_gs[0] : 1.0f), nvfp4::row_scale(a.v_gs ? a.v_gs[0] : 1.0f)};

    const int64_t groups = ((int64_t)a.tokens + a.together - 1) / a.together;
    for (int64_t group = blockIdx.x / a.parts; group < groups; group += gridDim.x / a.parts) {
        const int t0 = (int)group * a.together, n = min(a.together, a.tokens - t0);
        // the heads of the n tokens one after the other, `step` at a time
        struct At {
            int token, unit;
        };
        auto next = [&](At x) {
            x.unit += step;
            while (x.unit >= units && x.token < n) {
                x.unit -= units;
                ++x.token;
            }
            return x;
        };
        At at[kAhead];
        at[0] = next({0, (int)(blockIdx.x % a.parts) * at_once + mine - step});
        if (mine >= at_once)
            at[0].token = n;
        Row<kPairs> row[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (u)
                at[u] = next(at[u - 1]);
            if (at[u].token < n)
                load_row(row[u], head_of(a, t0 + at[u].token, at[u].unit), d0, partner);
        }

        __syncthreads();                                  // the angles of the tokens before are read
        for (int i = threadIdx.x; i < n * half; i += kThreads) {
            const int token = n == 1 ? 0 : i / half, j = i - token * half;
            const int axis = a.pair_axis ? a.pair_axis[j] : 0;
            const bool known = axis >= 0 && axis < a.axes;
            const int p = known ? a.positions[axis * a.ld_positions + t0 + token] : -1;
            const bool in = p >= 0 && p < a.max_position;
            lds.in[token * kMostPairs + j] = in;
            lds.c[token * kMostPairs + j] = in ? a.cos_sin[(int64_t)p * a.rot + j] : 1.0f;
            lds.s[token * kMostPairs + j] = in ? a.cos_sin[(int64_t)p * a.rot + half + j] : 0.0f;
        }
        if ((int)threadIdx.x < n)
            lds.slot[threadIdx.x] = a.slots[t0 + threadIdx.x];
        __syncthreads();
        while (at[0].token < n) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (at[u].token < n) {
                    const int64_t slot = lds.slot[at[u].token];
                    if (at[u].unit < a.heads || (slot >= 0 && slot < a.num_slots))
                        turn_row<kPairs>(a, scales, angles_of<kPairs>(lds, at[u].token * kMostPairs, d0, half, a.rot), row[u],
                                         t0 + at[u].token, slot, at[u].unit, d0, half);
                }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                at[u] = next(u ? at[u - 1] : at[kAhead - 1]);
                if (at[u].token < n)
                    load_row(row[u], head_of(a, t0 + at[u].token, at[u].unit), d0, partner);
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
                num_slots, (int)tokens, heads, kv_heads, head_dim, rot_dim, num_axes, (int)max_position, 1, 1};
    const Pairs pairs = interleaved ? kNeighbours : rot_dim == head_dim && rot_dim % 32 == 0 ? kWhole
                        : rot_dim % 16 == 0 ? kHalves8 : kHalves;
    // Few tokens: the heads of one are split over workgroups, each of which takes its
    // share at once. Many: a workgroup takes several tokens, until at most a tenth of its
    // threads idle in the last round (5003 tokens of 36 heads, three axes: 25 us with
    // one, 19 with four; 16384 of 80: 116 with one, 105 with two, 111 with four).
    const int at_once = kThreads / (head_dim / (pairs == kWhole ? 16 : 8)), all = ceil_div(heads + 2 * kv_heads, at_once);
    if (tokens * all <= 4096)
        a.parts = all;
    else
        while (a.together < kMostTokens && tokens / a.together >= 2048 &&
               10 * a.together * (heads + 2 * kv_heads) < 9 * ceil_div(a.together * (heads + 2 * kv_heads), at_once) * at_once)
            a.together *= 2;
    // workgroups beyond 2^22 loop over the tokens (a grid holds less than 2^32 threads)
    const int64_t groups = ceil_div(tokens, (int64_t)a.together), most = (1 << 22) / a.parts;
    const dim3 grid((unsigned)((groups < most ? groups : most) * a.parts));
    if (pairs == kWhole)
        hipLaunchKernelGGL((rope_append_kernel<kWhole>), grid, dim3(kThreads), 0, stream, a);
    else if (pairs == kHalves8)
        hipLaunchKernelGGL((rope_append_kernel<kHalves8>), grid, dim3(kThreads), 0, stream, a);
    else if (pairs == kHalves)
        hipLaunchKernelGGL((rope_append_kernel<kHalves>), grid, dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((rope_append_kernel<kNeighbours>), grid, dim3(kThreads), 0, stream, a);
    return launched();
}
