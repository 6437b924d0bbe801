// A whole mixture-of-experts layer for a few tokens (include/nvfp4_serving.h).
//
// The simplest form, two kernels. The first: one workgroup per (token, rank)
// pair and slice of 64 intermediate columns; it finds the pair's expert from
// the logits by counting, and each wave sums the products of its columns. The
// second: one workgroup per token and slice of 64 outputs.
#include "serving_common.hpp"
#include "nvfp4_device.hpp"

namespace {

constexpr int kThreads = 256;

struct Moe {
    const uint16_t* x;
    const float* logits;
    const void *w1, *w2;
    const uint8_t *s1, *s2;
    const float *gs1, *gs2;
    uint16_t* out;
    int32_t* ids;
    float* weights;
    float* h;          // workspace: [tokens * top_k][inter]
    int64_t ld_x, ld_out;
    int tokens, hidden, inter, experts, top_k, renormalize;
};

__device__ __forceinline__ float e2m1(uint32_t c)
{
    const uint32_t m = c & 7u;
    const float v = m < 2 ? 0.5f * m : __uint_as_float((126u + (m >> 1)) << 23 | (m & 1u) << 22);
    return c & 8u ? -v : v;
}

// A logit as it is compared: NaN stands behind everything, with -inf.
__device__ __forceinline__ float logit(const float* row, int e)
{
    const float v = row[e];
    return v == v ? v : -INFINITY;
}

template <bool kFp4>
__device__ __forceinline__ float weight(const void* w, const uint8_t* s, int64_t row, int cols, int c)
{
    if (!kFp4)
        return __uint_as_float((uint32_t)((const uint16_t*)w)[row * cols + c] << 16);
    const uint32_t code = ((const uint8_t*)w)[row * (cols / 2) + c / 2] >> (4 * (c & 1));
    return e2m1(code) * nvfp4::fp8_e4m3_decode(s[row * (cols / 16) + c / 16]);
}

__device__ __forceinline__ float wave_sum(float v)
{
    for (int d = 32; d; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

template <bool kFp4>
__global__ __launch_bounds__(kThreads) void moe_up_kernel(Moe a)
{
    __shared__ int found;
    __shared__ float chosen;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int pair = blockIdx.x, t = pair / a.top_k, k = pair % a.top_k;
    const float* row = a.logits + (int64_t)t * a.experts;
    for (int e = tid; e < a.experts; e += kThreads) {
        const float v = logit(row, e);
        int rank = 0;
        for (int f = 0; f < a.experts; ++f) {
            const float u = logit(row, f);
            rank += u > v || (u == v && f < e);
        }
        if (rank == k) {
            found = v == -INFINITY ? -1 : e;
            chosen = v;
        }
    }
    __syncthreads();
    const int e = found;
    if (blockIdx.y == 0 && tid == 0) {
        float top = -INFINITY, sum = 0;
        for (int f = 0; f < a.experts; ++f)
            top = fmaxf(top, logit(row, f));
        for (int f = 0; f < a.experts; ++f) {
            const float v = logit(row, f);
            sum += v == top ? 1.0f : expf(v - top);
        }
        a.ids[pair] = e;
        a.weights[pair] = e < 0 ? 0.0f : (chosen == top ? 1.0f : expf(chosen - top)) / sum;
    }
    if (e < 0)
        return;
    for (int c = wave; c < 64; c += kThreads / 64) {
        const int j = blockIdx.y * 64 + c;
        if (j >= a.inter)
            break;
        const int64_t r = (int64_t)e * 2 * a.inter + 16 * (j / 8) + j % 8;
        float g = 0, u = 0;
        for (int i = lane; i < a.hidden; i += 64) {
            const float x = __uint_as_float((uint32_t)a.x[t * a.ld_x + i] << 16);
            g = fmaf(x, weight<kFp4>(a.w1, a.s1, r, a.hidden, i), g);
            u = fmaf(x, weight<kFp4>(a.w1, a.s1, r + 8, a.hidden, i), u);
        }
        const float gs = a.gs1 ? a.gs1[e] : 1.0f;
        g = wave_sum(g) * gs;
        u = wave_sum(u) * gs;
        if (lane == 0)
            a.h[(int64_t)pair * a.inter + j] = g / (1.0f + expf(-g)) * u;
    }
}

template <bool kFp4>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(Moe a)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, t = blockIdx.x;
    float total = 0;
    for (int k = 0; k < a.top_k; ++k)
        total += a.weights[t * a.top_k + k];
    for (int c = wave; c < 64; c += kThreads / 64) {
        const int n = blockIdx.y * 64 + c;
        if (n >= a.hidden)
            break;
        float y = 0;
        for (int k = 0; k < a.top_k; ++k) {
            const int e = a.ids[t * a.top_k + k];
            if (e < 0)
                continue;
            float s = 0;
            for (int i = lane; i < a.inter; i += 64)
                s = fmaf(a.h[((int64_t)t * a.top_k + k) * a.inter + i],
                         weight<kFp4>(a.w2, a.s2, (int64_t)e * a.hidden + n, a.inter, i), s);
            float w = a.weights[t * a.top_k + k];
            if (a.renormalize)
                w /= total;
            y += w * wave_sum(s) * (a.gs2 ? a.gs2[e] : 1.0f);
        }
        if (lane == 0)
            a.out[t * a.ld_out + n] = __builtin_bit_cast(uint16_t, (__bf16)y);
    }
}

__global__ void moe_renormalize_kernel(Moe a)
{
    const int t = threadIdx.x;
    float total = 0;
    for (int k = 0; k < a.top_k; ++k)
        total += a.weights[t * a.top_k + k];
    for (int k = 0; k < a.top_k; ++k)
        if (total > 0)
            a.weights[t * a.top_k + k] /= total;
}

nvfp4_status_t check_sizes(int64_t tokens, int64_t hidden, int64_t inter, int32_t experts,
                           int32_t top_k)
{
    if (tokens < 0 || hidden < 0 || inter < 0 || experts < 1 || top_k < 1 || top_k > experts)
        return NVFP4_ERROR_INVALID_VALUE;
    if (tokens > 64 || hidden < 32 || hidden % 32 != 0 || inter < 32 || inter % 32 != 0 ||
        hidden > (1 << 20) || inter > (1 << 20) || experts > 512 || top_k > 32)
        return NVFP4_ERROR_UNSUPPORTED_SHAPE;
    return NVFP4_SUCCESS;
}

template <bool kFp4>
nvfp4_status_t run(Moe a, int64_t hidden, int64_t inter, int64_t workspace_bytes, int64_t tokens,
                   void* workspace, hipStream_t stream)
{
    using namespace serving;
    nvfp4_status_t st = check_sizes(tokens, hidden, inter, a.experts, a.top_k);
    if (st != NVFP4_SUCCESS)
        return st;
    if (a.ld_x < hidden || a.ld_out < hidden || !extent_ok(tokens, a.ld_x, 2) ||
        !extent_ok(tokens, a.ld_out, 2))
        return NVFP4_ERROR_INVALID_VALUE;
    if (tokens == 0)
        return NVFP4_SUCCESS;
    if (!a.x || !a.logits || !a.w1 || !a.w2 || (kFp4 && (!a.s1 || !a.s2)) || !a.out || !a.ids ||
        !a.weights || !workspace)
        return NVFP4_ERROR_INVALID_VALUE;
    if (!aligned(a.x, 16) || !aligned(a.out, 16) || a.ld_x % 8 != 0 || a.ld_out % 8 != 0 ||
        !aligned(a.w1, 16) || !aligned(a.w2, 16) || !aligned(a.s1, 2) || !aligned(a.s2, 2) ||
        !aligned(a.logits, 4) || !aligned(a.gs1, 4) || !aligned(a.gs2, 4) || !aligned(a.ids, 4) ||
        !aligned(a.weights, 4) || !aligned(workspace, 16))
        return NVFP4_ERROR_MISALIGNED;
    if (workspace_bytes < moe_layer_workspace(tokens, hidden, inter, a.experts, a.top_k))
        return NVFP4_ERROR_INVALID_VALUE;
    a.tokens = (int)tokens;
    a.hidden = (int)hidden;
    a.inter = (int)inter;
    a.h = (float*)workspace;
    hipLaunchKernelGGL(moe_up_kernel<kFp4>, dim3(a.tokens * a.top_k, ceil_div(a.inter, 64)),
                       dim3(kThreads), 0, stream, a);
    hipLaunchKernelGGL(moe_down_kernel<kFp4>, dim3(a.tokens, ceil_div(a.hidden, 64)),
                       dim3(kThreads), 0, stream, a);
    if (a.renormalize)
        hipLaunchKernelGGL(moe_renormalize_kernel, dim3(1), dim3(a.tokens), 0, stream, a);
    return launched();
}

}  // namespace

extern "C" int64_t moe_layer_workspace(int64_t tokens, int64_t hidden, int64_t inter,
                                       int32_t num_experts, int32_t top_k)
{
    if (check_sizes(tokens, hidden, inter, num_experts, top_k) != NVFP4_SUCCESS)
        return -1;
    return tokens * top_k * inter * 4;
}

extern "C" nvfp4_status_t moe_layer_nvfp4(
    const uint16_t* x, int64_t tokens, int64_t ld_x, const float* logits, const uint8_t* w1_packed,
    const uint8_t* w1_scales, const float* gs1, const uint8_t* w2_packed, const uint8_t* w2_scales,
    const float* gs2, int64_t hidden, int64_t inter, int32_t num_experts, int32_t top_k,
    int32_t renormalize, uint16_t* out, int64_t ld_out, int32_t* topk_ids, float* topk_weights,
    void* workspace, int64_t workspace_bytes, hipStream_t stream)
{
    Moe a = {x, logits, w1_packed, w2_packed, w1_scales, w2_scales, gs1, gs2, out, topk_ids,
             topk_weights, nullptr, ld_x, ld_out, 0, 0, 0, num_experts, top_k, renormalize};
    return run<true>(a, hidden, inter, workspace_bytes, tokens, workspace, stream);
}

extern "C" nvfp4_status_t moe_layer_bf16(const uint16_t* x, int64_t tokens, int64_t ld_x,
                                         const float* logits, const uint16_t* w1,
                                         const uint16_t* w2, int64_t hidden, int64_t inter,
                                         int32_t num_experts, int32_t top_k, int32_t renormalize,
                                         uint16_t* out, int64_t ld_out, int32_t* topk_ids,
                                         float* topk_weights, void* workspace,
                                         int64_t workspace_bytes, hipStream_t stream)
{
    Moe a = {x, logits, w1, w2, nullptr, nullptr, nullptr, nullptr, out, topk_ids, topk_weights,
             nullptr, ld_x, ld_out, 0, 0, 0, num_experts, top_k, renormalize};
    return run<false>(a, hidden, inter, workspace_bytes, tokens, workspace, stream);
}
