// Attention over the paged NVFP4 cache (include/nvfp4_serving.h).
//
// The simplest form: one wave per (query row, head). Each lane owns head_dim /
// 64 consecutive dimensions of the row; the keys are walked one by one, their
// scores summed over the wave, with the running maximum and sum of the
// softmax in FP32.
#include "serving_common.hpp"
#include "nvfp4_device.hpp"

namespace {

struct Attn {
    const uint16_t* q;
    const uint8_t *kp, *ks, *vp, *vs;
    const int32_t *table, *lens, *offsets;
    const float *k_gs, *v_gs;
    uint16_t* out;
    float* lse;
    int64_t ld_q, ld_out, ld_table, window;
    int tokens, heads, kv_heads, page, num_pages, max_pages, num_seqs, causal;
    float scale;
};

__device__ __forceinline__ float e2m1(uint32_t c)
{
    const uint32_t m = c & 7u;
    const float v = m < 2 ? 0.5f * m : __uint_as_float((126u + (m >> 1)) << 23 | (m & 1u) << 22);
    return c & 8u ? -v : v;
}

template <int D>
__global__ __launch_bounds__(64) void attn_plain_kernel(Attn a)
{
    constexpr int N = D / 64;
    const int lane = threadIdx.x, t = blockIdx.x, h = blockIdx.y;
    int b = 0;
    while (b < a.num_seqs && !(a.offsets[b] <= t && t < a.offsets[b + 1]))
        ++b;
    if (b == a.num_seqs)
        return;
    const int kvh = h / (a.heads / a.kv_heads), cols = a.kv_heads * D;
    const int64_t len = min((int64_t)max(a.lens[b], 0), (int64_t)a.max_pages * a.page);
    const int64_t pos = len - (a.offsets[b + 1] - t);
    const int64_t end = a.causal ? min(pos + 1, len) : len;
    const int64_t start = a.window > 0 ? max(pos - a.window + 1, (int64_t)0) : 0;
    float q[N], o[N], m = -INFINITY, l = 0;
    for (int i = 0; i < N; ++i) {
        const uint32_t w = a.q[t * a.ld_q + h * D + lane * N + i];
        q[i] = __uint_as_float(w << 16) * a.scale * (a.k_gs ? a.k_gs[0] : 1.0f);
        o[i] = 0;
    }
    for (int64_t j = start; j < end; ++j) {
        const int page = a.table[b * a.ld_table + j / a.page];
        if (page < 0 || page >= a.num_pages)
            continue;
        const int64_t slot = (int64_t)page * a.page + j % a.page;
        float s = 0;
        for (int i = 0; i < N; ++i) {
            const int c = kvh * D + lane * N + i;
            const uint32_t code = a.kp[slot * (cols / 2) + c / 2] >> (4 * (c & 1));
            s = fmaf(q[i], e2m1(code) * nvfp4::fp8_e4m3_decode(a.ks[slot * (cols / 16) + c / 16]), s);
        }
        for (int d = 32; d; d >>= 1)
            s += __shfl_xor(s, d);
        const float top = fmaxf(m, s), f = expf(m - top), p = expf(s - top);
        l = l * f + p;
        m = top;
        for (int i = 0; i < N; ++i) {
            const int c = kvh * D + lane * N + i;
            const uint32_t code = a.vp[slot * (cols / 2) + c / 2] >> (4 * (c & 1));
            o[i] = fmaf(p, e2m1(code) * nvfp4::fp8_e4m3_decode(a.vs[slot * (cols / 16) + c / 16]),
                        o[i] * f);
        }
    }
    const float gs = a.v_gs ? a.v_gs[0] : 1.0f;
    for (int i = 0; i < N; ++i) {
        const __bf16 r = (__bf16)(l > 0 ? o[i] * gs / l : 0.0f);
        a.out[t * a.ld_out + h * D + lane * N + i] = __builtin_bit_cast(uint16_t, r);
    }
    if (a.lse && lane == 0)
        a.lse[(int64_t)t * a.heads + h] = l > 0 ? m + logf(l) : -INFINITY;
}

bool sizes_ok(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t head_dim, int64_t num_seqs,
              int64_t max_query_len, int64_t max_seq_len, int64_t window)
{
    return tokens >= 0 && num_seqs >= 0 && max_query_len >= 0 && max_seq_len >= 0 && window >= 0 &&
           heads >= 1 && kv_heads >= 1 && heads % kv_heads == 0;
}

bool sizes_supported(int64_t tokens, int32_t heads, int32_t head_dim, int64_t num_seqs)
{
    return (head_dim == 64 || head_dim == 128 || head_dim == 256) && heads <= 1024 &&
           num_seqs <= 65535 && tokens <= INT32_MAX;
}

}  // namespace

extern "C" int64_t nvfp4_paged_attention_workspace(int64_t tokens, int32_t heads, int32_t kv_heads,
                                                   int32_t head_dim, int64_t num_seqs,
                                                   int64_t max_query_len, int64_t max_seq_len,
                                                   int64_t window)
{
    if (!sizes_ok(tokens, heads, kv_heads, head_dim, num_seqs, max_query_len, max_seq_len,
                  window) ||
        !sizes_supported(tokens, heads, head_dim, num_seqs))
        return -1;
    return 0;
}

extern "C" nvfp4_status_t nvfp4_paged_attention(
    const uint16_t* q, int64_t tokens, int64_t ld_q, int32_t heads, int32_t kv_heads,
    int32_t head_dim, const uint8_t* k_packed, const uint8_t* k_scales, const uint8_t* v_packed,
    const uint8_t* v_scales, int64_t num_slots, int32_t page_size, const int32_t* block_table,
    int64_t ld_table, int64_t max_pages, const int32_t* seq_lens, const int32_t* query_offsets,
    int64_t num_seqs, int64_t max_query_len, int64_t max_seq_len, float scale, int32_t causal,
    int64_t window, const float* k_gs, const float* v_gs, uint16_t* out, int64_t ld_out,
    float* lse, void* workspace, int64_t workspace_bytes, hipStream_t stream)
{
    using namespace serving;
    if (!sizes_ok(tokens, heads, kv_heads, head_dim, num_seqs, max_query_len, max_seq_len,
                  window) ||
        page_size < 1 || num_slots < 0 || num_slots % page_size != 0 || max_pages < 0 ||
        ld_table < max_pages || !extent_ok(num_seqs, ld_table, 4) || ld_q < 0 || ld_out < 0 ||
        workspace_bytes < 0 || !(scale - scale == 0.0f))
        return NVFP4_ERROR_INVALID_VALUE;
    if (!sizes_supported(tokens, heads, head_dim, num_seqs) || num_slots > INT32_MAX ||
        max_pages > INT32_MAX / page_size)
        return NVFP4_ERROR_UNSUPPORTED_SHAPE;
    const int64_t cols = (int64_t)heads * head_dim;
    if (ld_q < cols || ld_out < cols || !extent_ok(tokens, ld_q, 2) || !extent_ok(tokens, ld_out, 2))
        return NVFP4_ERROR_INVALID_VALUE;
    if (tokens == 0 || num_seqs == 0)
        return NVFP4_SUCCESS;
    if (!q || !out || !seq_lens || !query_offsets || (max_pages > 0 && !block_table) ||
        (num_slots > 0 && (!k_packed || !k_scales || !v_packed || !v_scales)))
        return NVFP4_ERROR_INVALID_VALUE;
    const uintptr_t sa = head_dim / 16;
    if (!aligned(q, 16) || !aligned(out, 16) || ld_q % 8 != 0 || ld_out % 8 != 0 ||
        !aligned(k_packed, 16) || !aligned(v_packed, 16) || !aligned(k_scales, sa) ||
        !aligned(v_scales, sa) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(query_offsets, 4) || !aligned(k_gs, 4) || !aligned(v_gs, 4) || !aligned(lse, 4) ||
        !aligned(workspace, 16))
        return NVFP4_ERROR_MISALIGNED;
    const int64_t need = nvfp4_paged_attention_workspace(tokens, heads, kv_heads, head_dim,
                                                         num_seqs, max_query_len, max_seq_len,
                                                         window);
    if (workspace_bytes < need || (need > 0 && !workspace))
        return NVFP4_ERROR_INVALID_VALUE;
    Attn a = {q, k_packed, k_scales, v_packed, v_scales, block_table, seq_lens, query_offsets,
              k_gs, v_gs, out, lse, ld_q, ld_out, ld_table, window, (int)tokens, heads, kv_heads,
              page_size, (int)(num_slots / page_size), (int)max_pages, (int)num_seqs, causal, scale};
    const dim3 grid((unsigned)tokens, (unsigned)heads);
    if (head_dim == 64)
        hipLaunchKernelGGL(attn_plain_kernel<64>, grid, dim3(64), 0, stream, a);
    else if (head_dim == 128)
        hipLaunchKernelGGL(attn_plain_kernel<128>, grid, dim3(64), 0, stream, a);
    else
        hipLaunchKernelGGL(attn_plain_kernel<256>, grid, dim3(64), 0, stream, a);
    return launched();
}
