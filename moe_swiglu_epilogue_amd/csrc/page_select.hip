// Page keys and the selection of pages (include/nvfp4_sparse.h).
#include "fp4_operand.hpp"
#include "nvfp4_device.hpp"
#include "serving_common.hpp"
#include "nvfp4_sparse.h"

namespace {

using fp4op::uint4v;

constexpr int kThreads = 256;
constexpr int kMostPages = 32768, kMostListed = 2048;

struct Requests {
    const int32_t *table, *lens, *offsets;
    int64_t ld_table;
    int num_pages, max_pages, page, num_seqs;
};

__device__ __forceinline__ int length_of(const Requests& r, int b)
{
    return min(max(r.lens[b], 0), r.max_pages * r.page);
}

// ---- page keys -----------------------------------------------------------------
// A workgroup takes a page and up to 64 blocks of 16 dimensions (whole heads): a
// thread owns a block and every so many of the page's tokens. A cache value
// times 2^10 is a whole number below 2^21.4, so a sum of four of them is exact in
// FP32; these go to binary64 sums, which are exact for pages up to 2^31 tokens.
struct PageKeys {
    const uint8_t *kp, *ks;
    int8_t *keys, *exponents;
    Requests r;
    int kv_heads, dim, per_request;
};

template <int D>
__global__ __launch_bounds__(kThreads) void page_keys_kernel(PageKeys a)
{
    constexpr int kHeadBlocks = D / 16;
    __shared__ double sums[kThreads][17];
    __shared__ double largest[64];
    const int b = blockIdx.x / a.per_request;
    const int blocks = a.kv_heads * kHeadBlocks;          // of 16 dimensions, of a token
    const int first_block = blockIdx.y * 64, here = min(blocks - first_block, 64);
    int width = kHeadBlocks;                              // threads over blocks: a power of two
    while (width < here)
        width *= 2;
    const int block = threadIdx.x % width, lane = threadIdx.x / width, lanes = kThreads / width;
    const int len = length_of(a.r, b);
    const int n = max(a.r.offsets[b + 1] - a.r.offsets[b], 0);
    const int begin = max(len - n, 0) / a.r.page, end = len / a.r.page;

    for (int j = begin + blockIdx.x % a.per_request; j < end; j += a.per_request) {
        const int entry = a.r.table[b * a.r.ld_table + j];
        if (entry < 0 || entry >= a.r.num_pages)
            continue;
        double total[16];
        for (int i = 0; i < 16; ++i)
            total[i] = 0;
        if (block < here) {
            const int64_t at = (int64_t)entry * a.r.page * blocks + first_block + block;
            for (int t0 = lane; t0 < a.r.page; t0 += 4 * lanes) {
                float part[16];
                for (int i = 0; i < 16; ++i)
                    part[i] = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int t = t0 + u * lanes;
                    if (t >= a.r.page)
                        break;
                    const uint2 w = *(const uint2*)(a.kp + (at + (int64_t)t * blocks) * 8);
                    float x[16];
                    nvfp4::dequantize16(w, a.ks[at + (int64_t)t * blocks], 1024.0f, x);
                    for (int i = 0; i < 16; ++i)
                        part[i] += x[i];
                }
                for (int i = 0; i < 16; ++i)
                    total[i] += (double)part[i];
            }
        }
        __syncthreads();                                  // the sums of the page before are read
        for (int i = 0; i < 16; ++i)
            sums[threadIdx.x][i] = total[i];
        __syncthreads();
        if (lane == 0 && block < here) {
            for (int k = 1; k < lanes; ++k)
                for (int i = 0; i < 16; ++i)
                    total[i] += sums[k * width + block][i];
            double top = 0;
            for (int i = 0; i < 16; ++i)
                top = fmax(top, fabs(total[i]));
            largest[block] = top;
        }
        __syncthreads();
        if (lane == 0 && block < here) {
            double top = 0;
            for (int i = 0; i < kHeadBlocks; ++i)
                top = fmax(top, largest[block / kHeadBlocks * kHeadBlocks + i]);
            // bits - 7; 2^bits > top >= 2^(bits - 1)
            const int e = top < 128.0 ? 0 : ilogb(top) - 6;
            uint4v w = {0, 0, 0, 0};
            for (int i = 0; i < 16; ++i) {
                const int key = min(max((int)rint(ldexp(total[i], -e)), -127), 127);
                w[i >> 2] |= (uint32_t)(key & 255) << (8 * (i & 3));
            }
            const int64_t at = (int64_t)entry * blocks + first_block + block;
            *(uint4v*)(a.keys + at * 16) = w;
            if (block % kHeadBlocks == 0)
                a.exponents[at / kHeadBlocks] = (int8_t)e;
        }
    }
}

// ---- selection -----------------------------------------------------------------
// A workgroup takes a token and a key/value head: scores of all pages in front of
// the token's own ones as ordered whole numbers in LDS, the top_k-th of them
// by counting their leading bytes, then the listed pages in order.
struct Select {
    const uint16_t* q;
    const int8_t *keys, *exponents;
    int32_t* pages;
    Requests r;
    int64_t ld_q;
    int tokens, heads, kv_heads, top, first, local;
};

// The request of token t, -1 if it is none's: the last b with offsets[b] <= t.
__device__ __forceinline__ int request_of(const Requests& r, int t)
{
    const int lane = threadIdx.x & 63;
    int b = -1;
    for (int base = 0; base <= r.num_seqs; base += 64) {
        const int i = base + lane;
        b += __popcll(__ballot(i <= r.num_seqs && r.offsets[min(i, r.num_seqs)] <= t));
    }
    return b >= r.num_seqs ? -1 : b;
}

// FP32 as whole numbers in the same order; finite ones are above 0 and below 2^32 - 1.
__device__ __forceinline__ uint32_t ordered(float v)
{
    const uint32_t b = __float_as_uint(v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

template <int D>
__global__ __launch_bounds__(kThreads) void select_pages_kernel(Select a)
{
    extern __shared__ uint32_t score[];                   // of each page; 0: not to be chosen
    __shared__ uint32_t q8[64][D / 4];
    __shared__ uint32_t count[256];
    __shared__ uint32_t tops[kThreads / 64], chosen[2];
    __shared__ uint32_t taken[kThreads / 64], ties[kThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int group = a.heads / a.kv_heads, width = a.first + a.top + a.local;
    for (int64_t item = blockIdx.x; item < (int64_t)a.tokens * a.kv_heads; item += gridDim.x) {
        __syncthreads();                                  // the LDS of the item before is read
        const int64_t t = item / a.kv_heads;
        const int h = (int)(item % a.kv_heads);
        const int b = request_of(a.r, (int)t);
        if (b < 0)
            continue;
        int32_t* out = a.pages + (t * a.kv_heads + h) * width;
        const int len = length_of(a.r, b);
        const int64_t p = min((int64_t)len - a.r.offsets[b + 1] + t, (int64_t)len - 1);
        if (p < 0) {
            for (int i = tid; i < width; i += kThreads)
                out[i] = -1;
            continue;
        }
        const int own = (int)(p / a.r.page), before = max(own - a.local + 1, 0);    // [first, before): by score
        const int32_t* table = a.r.table + b * a.r.ld_table;

        // the queries in 8 bits
        const uint16_t* q = a.q + t * a.ld_q + h * group * D;
        uint32_t top = 0;
        for (int i = tid; i < group * D / 8; i += kThreads) {
            const uint4v w = *(const uint4v*)(q + 8 * i);
            for (int k = 0; k < 4; ++k)
                top = max(top, max(w[k] << 16 & 0x7fff0000u, w[k] & 0x7fff0000u));
        }
        for (int d = 32; d; d >>= 1)
            top = max(top, (uint32_t)__shfl_xor((int)top, d));
        if (lane == 0)
            tops[wave] = top;
        __syncthreads();
        for (int w = 0; w < kThreads / 64; ++w)
            top = max(top, tops[w]);
        const int e = top == 0 || top >= 0x7f800000u ? 0 : ilogbf(__uint_as_float(top)) - 6;

        for (int j = tid; j < own + 1; j += kThreads)
            score[j] = 0;
        for (int h0 = 0; h0 < group; h0 += 64) {
            const int rows = min(group - h0, 64);
            __syncthreads();
            for (int i = tid; i < rows * D / 4; i += kThreads) {
                uint32_t w = 0;
                for (int k = 0; k < 4; ++k) {
                    const float x = ldexpf(__uint_as_float((uint32_t)q[h0 * D + 4 * i + k] << 16), -e);
                    w |= (uint32_t)((int)rintf(fminf(fmaxf(x, -127.0f), 127.0f)) & 255) << (8 * k);
                }
                q8[i / (D / 4)][i % (D / 4)] = w;
            }
            __syncthreads();
            for (int j = a.first + tid; j < before; j += kThreads) {
                const int entry = table[j];
                if (entry < 0 || entry >= a.r.num_pages)
                    continue;
                const int64_t at = (int64_t)entry * a.kv_heads + h;
                uint32_t key[D / 4];
                for (int i = 0; i < D / 16; ++i) {
                    const uint4v w = *(const uint4v*)(a.keys + at * D + 16 * i);
                    for (int k = 0; k < 4; ++k)
                        key[4 * i + k] = w[k];
                }
                int best = INT32_MIN;
                for (int r = 0; r < rows; ++r) {
                    int sum = 0;
                    for (int i = 0; i < D / 4; ++i)
                        sum = __builtin_amdgcn_sdot4((int)key[i], (int)q8[r][i], sum, false);
                    best = max(best, sum);
                }
                score[j] = max(score[j], ordered(ldexpf((float)best, a.exponents[at])));
            }
        }
        __syncthreads();

        // The top_k-th largest score, a byte at a time: `above` have larger leading
        // bytes than `prefix`, and the one wanted is the `want`-th of those that share it.
        uint32_t prefix = 0, want = a.top;
        bool all = a.top == 0;          // whether nothing (top 0) or everything is chosen
        for (int shift = 24; shift >= 0 && !all; shift -= 8) {
            count[tid] = 0;
            __syncthreads();
            for (int j = a.first + tid; j < before; j += kThreads) {
                const uint32_t v = score[j];
                if (v != 0 && (shift == 24 || v >> (shift + 8) == prefix >> (shift + 8)))
                    atomicAdd(&count[v >> shift & 255], 1u);
            }
            __syncthreads();
            // thread tid: how many have a byte above tid
            const uint32_t mine = count[tid];
            uint32_t sum = mine;
            for (int d = 1; d < 64; d <<= 1) {
                const uint32_t up = __shfl_down(sum, d);
                if (lane + d < 64)
                    sum += up;
            }
            if (lane == 0)
                tops[wave] = sum;
            if (tid == 0)
                chosen[0] = 256;
            __syncthreads();
            for (int w = wave + 1; w < kThreads / 64; ++w)
                sum += tops[w];
            if (sum >= want && sum - mine < want) {
                chosen[0] = tid;
                chosen[1] = want - (sum - mine);
            }
            __syncthreads();
            if (chosen[0] == 256) {
                all = true;             // fewer than top_k (only in the first round)
            } else {
                prefix |= chosen[0] << shift;
                want = chosen[1];
            }
            __syncthreads();
        }
        // chosen: scores above prefix, and the first `want` that equal it
        const uint32_t limit = a.top == 0 ? ~0u : all ? 0 : prefix;
        const uint32_t equals = a.top == 0 || all ? 0 : want;

        // Each wave takes a run of the pages; first it counts, then it writes.
        const int run = (own / (kThreads / 64) / 64 + 1) * 64;
        const int from = wave * run, to = min(from + run, own + 1);
        auto judge = [&](int j, bool& sure, bool& tie) {
            const bool inside = j < to, scored = inside && j >= a.first && j < before;
            const uint32_t v = scored ? score[j] : 0;
            sure = inside && (scored ? v > limit : true);
            tie = scored && v == limit && v != 0;
        };
        uint32_t n = 0, m = 0;
        for (int j0 = from; j0 < to; j0 += 64) {
            bool sure, tie;
            judge(j0 + lane, sure, tie);
            n += __popcll(__ballot(sure));
            m += __popcll(__ballot(tie));
        }
        if (lane == 0) {
            taken[wave] = n;
            ties[wave] = m;
        }
        __syncthreads();
        uint32_t at = 0, seen = 0, total = 0, all_ties = 0;
        for (int w = 0; w < kThreads / 64; ++w) {
            if (w == wave) {
                at = total;
                seen = all_ties;
            }
            total += taken[w];
            all_ties += ties[w];
        }
        at += min(seen, equals);
        total += min(all_ties, equals);
        for (int j0 = from; j0 < to; j0 += 64) {
            bool sure, tie;
            judge(j0 + lane, sure, tie);
            const uint64_t below = (1ull << lane) - 1;
            const uint64_t tied = __ballot(tie);
            const bool in = sure || (tie && seen + __popcll(tied & below) < equals);
            const uint64_t listed = __ballot(in);
            if (in)
                out[at + __popcll(listed & below)] = j0 + lane;
            at += __popcll(listed);
            seen += __popcll(tied);
        }
        for (uint32_t i = total + tid; i < (uint32_t)width; i += kThreads)
            out[i] = -1;
    }
}

bool requests_ok(int64_t num_slots, int32_t page_size, int64_t ld_table, int64_t max_pages, int64_t num_seqs)
{
    return page_size >= 1 && num_slots >= 0 && num_slots % page_size == 0 && max_pages >= 0 && ld_table >= max_pages &&
           num_seqs >= 0 && serving::extent_ok(num_seqs, ld_table, 4);
}

}  // namespace

extern "C" nvfp4_status_t nvfp4_page_keys(const uint8_t* k_packed, const uint8_t* k_scales, int64_t num_slots,
                                          int32_t kv_heads, int32_t head_dim, int32_t page_size,
                                          const int32_t* block_table, int64_t ld_table, int64_t max_pages,
                                          const int32_t* seq_lens, const int32_t* query_offsets, int64_t num_seqs,
                                          int64_t max_query_len, int8_t* keys, int8_t* exponents,
                                          hipStream_t stream)
{
    using namespace serving;
    if (kv_heads < 1 || max_query_len < 0 || !requests_ok(num_slots, page_size, ld_table, max_pages, num_seqs))
        return NVFP4_ERROR_INVALID_VALUE;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || kv_heads > 1024 || num_seqs > 65535 ||
        num_slots > INT32_MAX || max_pages > (1 << 30) / page_size)
        return NVFP4_ERROR_UNSUPPORTED_SHAPE;
    if (num_seqs == 0 || num_slots == 0 || max_pages == 0)
        return NVFP4_SUCCESS;
    if (!k_packed || !k_scales || !block_table || !seq_lens || !query_offsets || !keys || !exponents)
        return NVFP4_ERROR_INVALID_VALUE;
    if (!aligned(k_packed, 8) || !aligned(keys, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(query_offsets, 4))
        return NVFP4_ERROR_MISALIGNED;
    // a workgroup for each page that the longest request may complete, at most
    // 2^22 in all: a request with more takes several rounds
    int64_t per = ceil_div(max_query_len < (1 << 30) ? max_query_len : (int64_t)1 << 30, (int64_t)page_size);
    const int64_t most = (1 << 22) / num_seqs;
    per = per < 1 ? 1 : per > most ? most : per;
    PageKeys a = {k_packed, k_scales, keys, exponents,
                  {block_table, seq_lens, query_offsets, ld_table, (int)(num_slots / page_size), (int)max_pages,
                   page_size, (int)num_seqs},
                  kv_heads, head_dim, (int)per};
    const dim3 grid((unsigned)(num_seqs * per), (unsigned)ceil_div(kv_heads * (head_dim / 16), 64));
    if (head_dim == 64)
        hipLaunchKernelGGL((page_keys_kernel<64>), grid, dim3(kThreads), 0, stream, a);
    else if (head_dim == 128)
        hipLaunchKernelGGL((page_keys_kernel<128>), grid, dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((page_keys_kernel<256>), grid, dim3(kThreads), 0, stream, a);
    return launched();
}

extern "C" nvfp4_status_t nvfp4_select_pages(const uint16_t* q, int64_t tokens, int64_t ld_q, int32_t heads,
                                             int32_t kv_heads, int32_t head_dim, const int8_t* keys,
                                             const int8_t* exponents, int64_t num_slots, int32_t page_size,
                                             const int32_t* block_table, int64_t ld_table, int64_t max_pages,
                                             const int32_t* seq_lens, const int32_t* query_offsets, int64_t num_seqs,
                                             int32_t top_k, int32_t first, int32_t local, int32_t* pages,
                                             hipStream_t stream)
{
    using namespace serving;
    if (tokens < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads != 0 || top_k < 0 || first < 0 || local < 1 ||
        ld_q < 0 || !requests_ok(num_slots, page_size, ld_table, max_pages, num_seqs))
        return NVFP4_ERROR_INVALID_VALUE;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || heads > 1024 || num_seqs > 65535 ||
        num_slots > INT32_MAX || tokens > (1 << 30) / heads || max_pages > kMostPages ||
        max_pages > (1 << 30) / page_size || top_k > kMostListed || first > kMostListed || local > kMostListed ||
        first + top_k + local > kMostListed)
        return NVFP4_ERROR_UNSUPPORTED_SHAPE;
    if (ld_q < (int64_t)heads * head_dim || !extent_ok(tokens, ld_q, 2))
        return NVFP4_ERROR_INVALID_VALUE;
    if (tokens == 0 || num_seqs == 0)
        return NVFP4_SUCCESS;
    if (!q || !seq_lens || !query_offsets || !pages || (max_pages > 0 && !block_table) ||
        (num_slots > 0 && (!keys || !exponents)))
        return NVFP4_ERROR_INVALID_VALUE;
    if (!aligned(q, 16) || !aligned(keys, 16) || ld_q % 8 != 0 || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(query_offsets, 4) || !aligned(pages, 4))
        return NVFP4_ERROR_MISALIGNED;
    Select a = {q, keys, exponents, pages,
                {block_table, seq_lens, query_offsets, ld_table, (int)(num_slots / page_size), (int)max_pages,
                 page_size, (int)num_seqs},
                ld_q, (int)tokens, heads, kv_heads, top_k, first, local};
    // a grid holds less than 2^32 threads: beyond 2^22 workgroups each takes several tokens
    const int64_t items = tokens * kv_heads;
    const dim3 grid((unsigned)(items < (1 << 22) ? items : 1 << 22));
    const unsigned lds = (unsigned)max_pages * 4;
    if (head_dim == 64)
        hipLaunchKernelGGL((select_pages_kernel<64>), grid, dim3(kThreads), lds, stream, a);
    else if (head_dim == 128)
        hipLaunchKernelGGL((select_pages_kernel<128>), grid, dim3(kThreads), lds, stream, a);
    else
        hipLaunchKernelGGL((select_pages_kernel<256>), grid, dim3(kThreads), lds, stream, a);
    return launched();
}
