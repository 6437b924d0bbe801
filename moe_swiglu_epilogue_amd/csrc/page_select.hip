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
// A workgroup takes a token, or some that follow each other in one request, and a
// key/value head. Scores are products of whole numbers on the matrix cores
// (v_mfma_i32_16x16x64_i8): a page a row, a query row a column, so the largest of a
// token's rows is found within 16 lanes. They go to LDS as FP32, exactly. Then the
// top_k-th largest is searched, by all waves for a single token and by a wave each
// for several, and the listed pages are written in order.
struct Select {
    const uint16_t* q;
    const int8_t *keys, *exponents;
    int32_t* pages;
    Requests r;
    int64_t ld_q;
    int tokens, heads, kv_heads, top, first, local;
    int together;      // tokens that a workgroup takes
    int pitch;         // scores of a token in LDS
};

constexpr int kMostRows = 64;      // query rows that are compared at once

typedef int int4v __attribute__((ext_vector_type(4)));

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

// FP32 as whole numbers in the same order.
__device__ __forceinline__ uint32_t ordered(float v)
{
    const uint32_t b = __float_as_uint(v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float number(uint32_t v)
{
    return __uint_as_float(v & 0x80000000u ? v & 0x7fffffffu : ~v);
}

template <int kCtrl>
__device__ __forceinline__ int other_lane(int v)
{
    return __builtin_amdgcn_mov_dpp(v, kCtrl, 0xf, 0xf, true);
}

// Largest of 2^bits neighbouring lanes, at most 16, in all of them.
__device__ __forceinline__ int max_of(int v, int bits)
{
    const int two = max(v, other_lane<0xb1>(v));            // lane ^ 1
    v = bits > 0 ? two : v;
    const int four = max(v, other_lane<0x4e>(v));           // lane ^ 2
    v = bits > 1 ? four : v;
    const int eight = max(v, other_lane<0x141>(v));         // 7 - lane of eight
    v = bits > 2 ? eight : v;
    const int sixteen = max(v, other_lane<0x140>(v));       // 15 - lane of sixteen
    return bits > 3 ? sixteen : v;
}

// What is chosen by score: scores above `limit` and the first `ties` that equal it.
struct Limit {
    float limit;
    uint32_t ties;
};

template <int W>
struct SelectShared {
    float lo, hi;                      // of all waves' scores, as ordered numbers
    uint32_t n[3], sure[W], ties[W];
};

// The top-th largest of score[first .. before): bisection of the values between the
// smallest and the largest, counting by ballots those not below the middle, until
// the count is right or one value is left. By one wave (W = 1) or by all of a
// workgroup's, which add their counts up in LDS. The first 8 scores of a lane stay
// in registers, which is all up to 512 pages a wave.
template <int W, class Shared>
__device__ __forceinline__ Limit find_limit(Shared& lds, const float* score, int first, int before, int top)
{
    constexpr int kHeld = 8;
    const int lane = threadIdx.x & 63, wave = W == 1 ? 0 : threadIdx.x >> 6;
    if (top == 0 || before <= first)
        return {INFINITY, 0};
    const int from = first + 64 * wave + lane;
    const int rest = first + 64 * W * kHeld;           // pages from here on are read again each time
    float held[kHeld], lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int j = from + 64 * W * i;
        held[i] = j < before ? score[j] : -INFINITY;
        lo = held[i] == -INFINITY ? lo : fminf(lo, held[i]);
        hi = fmaxf(hi, held[i]);
    }
#pragma unroll 1
    for (int j = rest + 64 * wave + lane; j < before; j += 64 * W) {
        const float v = score[j];
        lo = v == -INFINITY ? lo : fminf(lo, v);
        hi = fmaxf(hi, v);
    }
#pragma unroll 1
    for (int d = 32; d; d >>= 1) {
        lo = fminf(lo, __shfl_xor(lo, d));
        hi = fmaxf(hi, __shfl_xor(hi, d));
    }
    if (W > 1) {
        if (lane == 0) {
            atomicMin((int*)&lds.lo, (int)(ordered(lo) ^ 0x80000000u));
            atomicMax((int*)&lds.hi, (int)(ordered(hi) ^ 0x80000000u));
        }
        __syncthreads();
        lo = number(__float_as_uint(lds.lo) ^ 0x80000000u);
        hi = number(__float_as_uint(lds.hi) ^ 0x80000000u);
    }
    if (lo > hi)
        return {INFINITY, 0};
    // the top-th largest is in [lo, hi]; `above` are larger than hi
    int above = 0, turn = 0;
    float mid = lo;
    for (;;) {
        int c = 0;
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            c += __popcll(__ballot(held[i] >= mid));
#pragma unroll 1
        for (int j0 = rest + 64 * wave; j0 < before; j0 += 64 * W)
            c += __popcll(__ballot(j0 + lane < before && score[j0 + lane] >= mid));
        if (W > 1) {
            // the next turn's sum is cleared in front of this turn's barrier; it was last
            // read in front of the barrier before
            if (lane == 0)
                atomicAdd(&lds.n[turn], (uint32_t)c);
            const int next = turn == 2 ? 0 : turn + 1;
            if (threadIdx.x == 0)
                lds.n[next] = 0;
            __syncthreads();
            c = lds.n[turn];
            turn = next;
        }
        if (c >= top) {
            lo = mid;
            if (c == top)
                return {lo, ~0u};
        } else {
            if (mid == lo)                  // all of them, and fewer than top
                return {-INFINITY, 0};
            above = c;
            hi = number(ordered(mid) - 1);  // the next smaller number: not below lo
        }
        if (lo >= hi)
            return {lo, (uint32_t)(top - above)};
        mid = lo + 0.5f * (hi - lo);
        mid = mid > lo ? mid : hi;
    }
}

// Sixteen pages for a wave: their keys as the left operand of the products (lane % 16
// the page, 16 (lane / 16) + 64 k .. the dimensions), their exponents.
template <int D>
struct PageTile {
    int4v key[D / 64];
    int exponent;        // -1: not a page to be chosen
};

template <int D, int W>
__global__ __launch_bounds__(64 * W) void select_pages_kernel(Select a)
{
    constexpr int K = D / 64, kPitch = D + 16;
    extern __shared__ __align__(16) float score[];        // [tokens][pitch]; -inf: not to be chosen
    __shared__ __align__(16) uint8_t q8[kMostRows][kPitch];
    __shared__ SelectShared<W> lds;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, n = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = a.heads / a.kv_heads, listed = a.first + a.top + a.local;
    int bits = 0;                                         // 2^bits columns for a token, at most 16
    while (bits < 4 && 1 << bits < group)
        ++bits;
    const int h = blockIdx.x % a.kv_heads;
    int token = blockIdx.x / a.kv_heads * a.together;
    const int token_end = min(token + a.together, a.tokens);

    // the tokens of one request at a time
    for (int run = 1; token < token_end; token += run) {
        run = 1;
        const int b = request_of(a.r, token);
        if (b < 0)
            continue;
        const int behind = a.r.offsets[b + 1], len = length_of(a.r, b);
        run = min(token_end, behind) - token;
        const int pos0 = min(len - behind + token, len - 1), pos1 = min(pos0 + run, len) - 1;
        const int32_t* table = a.r.table + b * a.r.ld_table;
        const uint16_t* q = a.q + token * a.ld_q + h * group * D;
        // the pages that some token may choose by score
        const int before = pos1 < 0 ? 0 : max(pos1 / a.r.page - a.local + 1, 0);
        __syncthreads();                                  // the LDS of what came before is read
        if (tid == 0) {
            lds.lo = __int_as_float(INT32_MAX);
            lds.hi = __int_as_float(INT32_MIN);
            lds.n[0] = 0;
        }

        // scores, of 64 query rows at a time: run * group rows, or the heads of a token
#pragma unroll 1
        for (int h0 = 0; h0 < group; h0 += kMostRows) {
            const int heads = min(group - h0, kMostRows);
            if (h0)
                __syncthreads();
            else
                // places in the cache, -1 where hidden, wait in LDS where the scores go
#pragma unroll 1
                for (int j = a.first + tid; j < before; j += 64 * W) {
                    const int entry = table[j];
                    score[j] = __int_as_float(entry >= 0 && entry < a.r.num_pages ? entry : -1);
                }
            // queries in 8 bits, a token a wave or a single token by all waves
#pragma unroll 1
            for (int i = run == 1 ? 0 : wave; i < run; i += W) {
                const uint16_t* qi = q + i * a.ld_q;
                uint32_t top = 0;
#pragma unroll 1
                for (int x = lane; x < group * D / 8; x += 64) {
                    const uint4v w = *(const uint4v*)(qi + 8 * x);
                    for (int k = 0; k < 4; ++k)
                        top = max(top, max(w[k] << 16 & 0x7fff0000u, w[k] & 0x7fff0000u));
                }
#pragma unroll 1
                for (int d = 32; d; d >>= 1)
                    top = max(top, (uint32_t)__shfl_xor((int)top, d));
                const int e = top == 0 || top >= 0x7f800000u ? 0 : 6 - ilogbf(__uint_as_float(top));
#pragma unroll 1
                for (int x = (run == 1 ? 64 * wave : 0) + lane; x < heads * D / 8; x += run == 1 ? 64 * W : 64) {
                    const uint4v w = *(const uint4v*)(qi + h0 * D + 8 * x);
                    uint32_t v[2] = {0, 0};
                    for (int k = 0; k < 8; ++k) {
                        const float y = ldexpf(__uint_as_float(k & 1 ? w[k >> 1] & 0xffff0000u : w[k >> 1] << 16), e);
                        v[k >> 2] |= (uint32_t)((int)rintf(__builtin_amdgcn_fmed3f(y, -127.0f, 127.0f)) & 255) << (8 * (k & 3));
                    }
                    *(uint2*)&q8[i * heads + x / (D / 8)][x % (D / 8) * 8] = make_uint2(v[0], v[1]);
                }
            }
            __syncthreads();

            auto load = [&](PageTile<D>& t, int j0) {
                const int j = j0 + n;
                int entry = -1;
                if (j < before)
                    entry = h0 ? table[j] : __float_as_int(score[j]);
                const bool in = entry >= 0 && entry < a.r.num_pages;
                const int64_t at = (int64_t)(in ? entry : 0) * a.kv_heads + h;
                t.exponent = -1;
                if (in) {
                    t.exponent = min(max((int)a.exponents[at], 0), 64);
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        t.key[k] = *(const int4v*)(a.keys + at * D + 64 * k + 16 * g);
                }
            };
            // column tiles: several tokens each, or several for a token
            const int parts = (heads + 15) / 16;
            auto compare = [&](const PageTile<D>& t, int j0) {
                int e[4];
                for (int i = 0; i < 4; ++i)
                    e[i] = __builtin_amdgcn_ds_bpermute((4 * g + i) * 4, t.exponent);
#pragma unroll 1
                for (int t0 = 0; t0 < run; t0 += 16 >> bits) {
                    const int of = t0 + (n >> bits), row0 = min(of, run - 1) * heads, col = n & ((1 << bits) - 1);
                    int best[4] = {INT32_MIN, INT32_MIN, INT32_MIN, INT32_MIN};
#pragma unroll 1
                    for (int p = 0; p < parts; ++p) {
                        const uint8_t* row = q8[row0 + min(16 * p + col, heads - 1)] + 16 * g;
                        int4v sum = {0, 0, 0, 0};
#pragma unroll
                        for (int k = 0; k < K; ++k)
                            sum = __builtin_amdgcn_mfma_i32_16x16x64_i8(t.key[k], *(const int4v*)(row + 64 * k), sum, 0, 0, 0);
                        for (int i = 0; i < 4; ++i)
                            best[i] = max(best[i], sum[i]);
                    }
                    for (int i = 0; i < 4; ++i)
                        best[i] = max_of(best[i], bits);
                    if (col == 0 && of < run) {
                        float* at = score + of * a.pitch + j0 + 4 * g;
                        for (int i = 0; i < 4; ++i) {
                            const float v = e[i] < 0 ? -INFINITY : ldexpf((float)best[i], e[i]);
                            if (j0 + 4 * g + i < before)
                                at[i] = h0 ? fmaxf(at[i], v) : v;
                        }
                    }
                }
            };
            PageTile<D> next;
            load(next, a.first + 16 * wave);
#pragma unroll 1
            for (int j0 = a.first + 16 * wave; j0 < before; j0 += 16 * W) {
                const PageTile<D> tile = next;
                load(next, j0 + 16 * W);
                compare(tile, j0);
            }
        }
        __syncthreads();

        // The listed pages in order: a wave takes a token, or a run of a single token's
        // pages, which it counts first and then writes.
        const int shares = run == 1 ? W : 1;
#pragma unroll 1
        for (int i = run == 1 ? 0 : wave; i < run; i += W) {
            const float* mine = score + i * a.pitch;
            int32_t* out = a.pages + ((int64_t)(token + i) * a.kv_heads + h) * listed;
            const int p = min(pos0 + i, len - 1), pages = p < 0 ? 0 : p / a.r.page + 1, end = max(pages - a.local, 0);
            const Limit l = run == 1 ? find_limit<W>(lds, mine, a.first, end, a.top) : find_limit<1>(lds, mine, a.first, end, a.top);
            const int each = (pages + shares * 64 - 1) / (shares * 64) * 64;
            const int from = run == 1 ? min(wave * each, pages) : 0, to = min(from + each, pages);
            uint32_t at = 0, seen = 0;
#pragma unroll 1
            for (int pass = shares == 1; pass < 2; ++pass) {
                uint32_t sure = 0, tied = seen;
                const uint64_t below = (1ull << lane) - 1;
#pragma unroll 1
                for (int j0 = from; j0 < to; j0 += 64) {
                    const int j = j0 + lane;
                    const bool scored = j >= a.first && j < end;
                    const float v = scored ? mine[j] : 0.0f;
                    const bool tie = scored && v == l.limit && j < to && v != -INFINITY;
                    const uint64_t equal = __ballot(tie);
                    const bool in = j < to && (scored ? v > l.limit || (pass && tie && tied + __popcll(equal & below) < l.ties) : true);
                    const uint64_t taken = __ballot(in);
                    if (pass && in)
                        out[at + sure + __popcll(taken & below)] = j;
                    sure += __popcll(taken);
                    tied += __popcll(equal);
                }
                if (pass == 0) {
                    if (lane == 0) {
                        lds.sure[wave] = sure;
                        lds.ties[wave] = tied;
                    }
                    __syncthreads();
#pragma unroll 1
                    for (int w = 0; w < wave; ++w) {
                        at += lds.sure[w];
                        seen += lds.ties[w];
                    }
                    at += min(seen, l.ties);
                } else if (to == pages && (from < to || run > 1 || wave == 0)) {
                    // the last pages' wave fills the rest of the list
#pragma unroll 1
                    for (int x = (int)(at + sure) + lane; x < listed; x += 64)
                        out[x] = -1;
                }
            }
        }
    }
}

template <int D>
void launch_select(const Select& a, dim3 grid, unsigned lds, hipStream_t stream)
{
    // a grid holds less than 2^32 threads
    if (a.together > 1 || a.r.max_pages <= 512 || grid.x > (1 << 20))
        hipLaunchKernelGGL((select_pages_kernel<D, 4>), grid, dim3(256), lds, stream, a);
    else
        hipLaunchKernelGGL((select_pages_kernel<D, 16>), grid, dim3(1024), lds, stream, a);
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
        num_slots > INT32_MAX || tokens > (1 << 23) / heads || max_pages > kMostPages ||
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
                ld_q, (int)tokens, heads, kv_heads, top_k, first, local, 1, ((int)max_pages + 3) & ~3};
    // Tokens of long chunks go to a workgroup together, as many as 64 query rows and
    // 64 KB of scores hold, at most 16.
    const int group = heads / kv_heads;
    while (a.together < 16 && a.together < tokens / num_seqs && (a.together + 1) * group <= kMostRows &&
           (a.together + 1) * a.pitch * 4 <= 65536)
        ++a.together;
    const int64_t items = ceil_div(tokens, (int64_t)a.together) * kv_heads;
    const dim3 grid((unsigned)items);
    const unsigned lds = (unsigned)(a.together * a.pitch * 4);
    if (head_dim == 64)
        launch_select<64>(a, grid, lds, stream);
    else if (head_dim == 128)
        launch_select<128>(a, grid, lds, stream);
    else
        launch_select<256>(a, grid, lds, stream);
    return launched();
}
