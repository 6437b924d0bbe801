// Page keys and the selection of pages (include/nvfp4_sparse.h).
#include "fp4_operand.hpp"
#include "nvfp4_device.hpp"
#include "serving_common.hpp"
#include "sparse_common.hpp"
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
// thread owns a block and every so many of the page's tokens, 8 of which are on their
// way at a time. A cache value times 2^10 is a whole number below 2^21.4, so a sum
// of four of them is exact in FP32; these go to binary64 sums, which are exact for
// pages up to 2^31 tokens. The threads' sums meet in LDS, where every thread adds
// some up. Bound by memory latency: a workgroup's chain of loads (lengths, table,
// tokens) and its start. A step of 256 requests 6.2 us, 6 prompts of up to 16384 tokens
// (21 MB) 12.
struct PageKeys {
    const uint8_t *kp, *ks;
    int8_t *keys, *exponents;
    Requests r;
    int kv_heads, dim, per_request;
};

// sum[i] += scale * the i-th of 16 codes, exact where the sum is.
__device__ __forceinline__ void add16(float (&sum)[16], uint2 w, float scale)
{
    auto pair = [&](int i, auto v) {
        sum[i] = __builtin_fmaf(v[0], scale, sum[i]);
        sum[i + 1] = __builtin_fmaf(v[1], scale, sum[i + 1]);
    };
    pair(0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w.x, 1.0f, 0));
    pair(2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w.x, 1.0f, 1));
    pair(4, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w.x, 1.0f, 2));
    pair(6, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w.x, 1.0f, 3));
    pair(8, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w.y, 1.0f, 0));
    pair(10, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w.y, 1.0f, 1));
    pair(12, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w.y, 1.0f, 2));
    pair(14, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w.y, 1.0f, 3));
}

template <int D>
__global__ __launch_bounds__(kThreads) void page_keys_kernel(PageKeys a)
{
    constexpr int kHeadBlocks = D / 16, kAhead = 8;
    __shared__ double sums[kThreads][17];
    __shared__ double powers[64];                         // 2^-e, as binary64's pow has them
    // the requests' first pages first: workgroups that find none come last
    const int b = blockIdx.x % a.r.num_seqs;
    const int blocks = a.kv_heads * kHeadBlocks;          // of 16 dimensions, of a token
    const int first_block = blockIdx.y * 64, here = min(blocks - first_block, 64);
    int width = kHeadBlocks;                              // threads over blocks: a power of two
    while (width < here)
        width *= 2;
    const int block = threadIdx.x % width, lane = threadIdx.x / width, lanes = kThreads / width;
    const int len = length_of(a.r, b);
    const int n = max(a.r.offsets[b + 1] - a.r.offsets[b], 0);
    const int begin = max(len - n, 0) / a.r.page, end = len / a.r.page;

    // beside the loads; some are an ulp low, so that a sum half way between two keys
    // goes to the one nearer 0 there and to the even one elsewhere
    if (threadIdx.x < 64 && begin < end)
        powers[threadIdx.x] = pow(2.0, -(double)threadIdx.x);

    for (int j = begin + blockIdx.x / a.r.num_seqs; j < end; j += a.per_request) {
        const int entry = a.r.table[b * a.r.ld_table + j];
        if (entry < 0 || entry >= a.r.num_pages)
            continue;
        double total[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            total[i] = 0;
        if (block < here) {
            const int64_t at = (int64_t)entry * a.r.page * blocks + first_block + block;
#pragma unroll 1
            for (int t0 = lane; t0 < a.r.page; t0 += kAhead * lanes) {
                // tokens behind the page: its last one, with a scale of 0
                uint2 w[kAhead];
                uint32_t sf[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int64_t x = at + (int64_t)min(t0 + u * lanes, a.r.page - 1) * blocks;
                    w[u] = *(const uint2*)(a.kp + x * 8);
                    sf[u] = a.ks[x];
                }
#pragma unroll
                for (int half = 0; half < kAhead; half += 4) {
                    float part[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        part[i] = 0;
#pragma unroll
                    for (int u = half; u < half + 4; ++u)
                        add16(part, w[u], t0 + u * lanes < a.r.page ? 1024.0f * nvfp4::fp8_e4m3_decode(sf[u]) : 0.0f);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        total[i] += (double)part[i];
                }
            }
        }
        __syncthreads();                                  // the sums of the page before are read
#pragma unroll
        for (int i = 0; i < 16; ++i)
            sums[threadIdx.x][i] = total[i];
        __syncthreads();
        // A thread adds up some dimensions of a block; those of a head are in a row of at
        // most 64 threads and find their largest sum by exchanges.
        const int parts = min(lanes, min(16, 64 / kHeadBlocks)), share = 16 / parts;     // threads of a block, dimensions
        if ((int)threadIdx.x < width * parts) {
            const int of = threadIdx.x / parts, d0 = threadIdx.x % parts * share;
            double sum[4], top = 0;                       // share: 1, 2 or 4, as parts is 4, 8 or 16
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sum[i] = 0;
                if (i < share) {
                    for (int k = 0; k < lanes; ++k)
                        sum[i] += sums[k * width + of][d0 + i];
                    top = fmax(top, fabs(sum[i]));
                }
            }
            for (int d = 1; d < kHeadBlocks * parts; d *= 2)
                top = fmax(top, __shfl_xor(top, d));
            // the length of a whole number in binary is its exponent and 1
            const int bits = top < 1.0 ? 0 : (int)(__double_as_longlong(top) >> 52) - 1022;
            const int e = max(bits - 7, 0);
            const double scale = powers[e];               // e is at most 53 - 7
            if (of < here) {
                const int64_t at = (int64_t)entry * blocks + first_block + of;
                uint32_t w = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w |= (uint32_t)(min(max((int)rint(sum[i] * scale), -127), 127) & 255) << (8 * i);
                int8_t* out = a.keys + at * 16 + d0;
                if (share == 4) {
                    *(uint32_t*)out = w;
                } else {
                    out[0] = (int8_t)w;
                    if (share == 2)
                        out[1] = (int8_t)(w >> 8);
                }
                if (of % kHeadBlocks == 0 && d0 == 0)
                    a.exponents[at / kHeadBlocks] = (int8_t)e;
            }
        }
    }
}

// ---- selection -----------------------------------------------------------------
// Scores are products of whole numbers on the matrix cores
// (v_mfma_i32_16x16x64_i8): a query row a row, a page a column, so a lane holds four
// rows of one page, and the largest of a token's rows is found in its registers
// and, from 8 rows on, by one or two exchanges. As FP32 they are exact. Then the
// top_k-th largest is searched and the listed pages are written in order.
//   Many tokens: a workgroup takes some that follow each other in one request and a
// key/value head, keeps their scores in LDS, and a wave each selects; a single
// token's is selected by all waves (select_chunk_kernel).
// 2048 tokens of 32/8 heads of 128 behind 30000 (500 pages of 64): 54 us, some 30 of them
// vector arithmetic, most of it the search's.
//   Few tokens: a compute unit alone reads keys at some 25 GB/s, so their pages go to a
// workgroup for each 256 (score_pages_kernel), and by way of the workspace to a
// workgroup for each list (list_pages_kernel). One request of 2048 pages 12 us, 64 of up
// to 1024 20 us; latency, and for many requests keys of 128 bytes from all over the cache.
struct Select {
    const uint16_t* q;
    const int8_t *keys, *exponents;
    int32_t* pages;
    float* scores;     // workspace
    Requests r;
    int64_t ld_q;
    int tokens, heads, kv_heads, top, first, local;
    int together;      // tokens that a workgroup takes
    int pitch;         // scores of a token
    int chunks;        // workgroups over a token's pages
};

constexpr int kMostRows = 64;      // query rows that are compared at once

typedef int int4v __attribute__((ext_vector_type(4)));

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

// op over the lanes up to each; `none` is what op leaves alone. Row shifts and
// broadcasts: an exchange through LDS takes some ten times as long.
template <class Op>
__device__ __forceinline__ uint32_t up_to_lane(uint32_t v, uint32_t none, Op op)
{
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, 0x111, 0xf, 0xf, false));    // row_shr:1
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, 0x112, 0xf, 0xf, false));
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, 0x114, 0xf, 0xf, false));
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, 0x118, 0xf, 0xf, false));
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, 0x142, 0xa, 0xf, false));    // row_bcast:15
    return op(v, (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, 0x143, 0xc, 0xf, false)); // row_bcast:31
}

__device__ __forceinline__ uint32_t sums_up_to_lane(uint32_t v)
{
    return up_to_lane(v, 0, [](uint32_t x, uint32_t y) { return x + y; });
}

__device__ __forceinline__ uint32_t last_lane(uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, 63); }

__device__ __forceinline__ uint32_t largest_of(uint32_t v)
{
    return last_lane(up_to_lane(v, 0, [](uint32_t x, uint32_t y) { return max(x, y); }));
}

__device__ __forceinline__ uint32_t smallest_of(uint32_t v)
{
    return last_lane(up_to_lane(v, ~0u, [](uint32_t x, uint32_t y) { return min(x, y); }));
}

// What is chosen by score: scores above `limit` and the first `ties` that equal it.
struct Limit {
    float limit;
    uint32_t ties;
};

constexpr int kBins = 256;

template <int W>
struct SelectShared {
    uint32_t bins[W][kBins];           // a wave's own, or two of the workgroup's in turn
    uint32_t lo[2], hi[2], found;      // of all waves' scores, as ordered numbers
    uint32_t counts[W];
};

// The top-th largest of score[first .. before): the scores between the smallest and
// the largest are counted in 256 equal parts, and the search goes on in the part that
// holds the top-th, until all of it is wanted, or one, or it holds one value. By one wave
// (W = 1) in bins of its own, or by all of a workgroup's. The parts that hold the
// smallest and the largest score differ, so every round leaves a score out; one or
// two rounds are usual. (A wave alone takes 8 clocks an instruction: halving the range by
// counts took a dozen rounds of 0.6 us.) The first 8 scores of a lane stay in
// registers, which is all up to 512 pages a wave.
//   Scores that the kernels write are -inf or finite and at most 2^86 in magnitude. Of
// any others (a workspace that another call writes to) the search ends and at most top are
// chosen all the same: NaN is never chosen, and where `scale` is 0, as hi - lo is +inf,
// a round leaves nothing out and is the last.
template <int W, class Shared>
__device__ __forceinline__ Limit find_limit(Shared& lds, const float* score, int first, int before, int top)
{
    constexpr int kHeld = 8;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (top == 0 || before <= first)
        return {INFINITY, 0};
    const int from = first + (W == 1 ? 0 : 64 * wave) + lane;
    const int rest = from + 64 * W * kHeld;            // pages from here on are read again each time
    float held[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int j = from + 64 * W * i;
        held[i] = first + 64 * W * i < before && j < before ? score[j] : -INFINITY;
    }
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (first + 64 * W * i < before)
                f(held[i]);
#pragma unroll 1
        for (int j = rest; j < before; j += 64 * W)
            f(score[j]);
    };
    uint32_t low = ~0u, high = 0, n = 0;
    each([&](float v) {
        const bool in = v > -INFINITY;
        low = min(low, in ? ordered(v) : ~0u);
        high = max(high, in ? ordered(v) : 0);
        n += in;
    });
    low = smallest_of(low);
    high = largest_of(high);
    n = last_lane(sums_up_to_lane(n));
    if (W > 1) {
        if (lane == 0) {
            atomicMin(&lds.lo[0], low);
            atomicMax(&lds.hi[0], high);
            atomicAdd(&lds.found, n);
        }
        __syncthreads();
        low = lds.lo[0];
        high = lds.hi[0];
        n = lds.found;
    }
    if ((int)n <= top)
        return {-INFINITY, 0};
    // the limit is the want-th largest of the n scores in [lo, hi]
    float lo = number(low), hi = number(high);
    uint32_t want = top;
    for (int turn = 0; lo < hi; turn ^= 1) {
        uint32_t* bins = lds.bins[W == 1 ? wave : turn];
        const float scale = (float)kBins / (hi - lo);
        // a larger score never goes to a lower part
        auto part = [&](float v) { return min((int)((v - lo) * scale), kBins - 1); };
        if (W == 1) {
            *(uint4v*)&bins[4 * lane] = uint4v{0, 0, 0, 0};
            asm volatile("" ::: "memory");              // a wave's accesses to LDS keep their order
        }
        each([&](float v) {
            if (v >= lo && v <= hi)
                atomicAdd(&bins[part(v)], 1u);
        });
        if (W > 1) {
            // what the next round adds to was last read in front of the barrier before
            if (wave == 0)
                *(uint4v*)&lds.bins[turn ^ 1][4 * lane] = uint4v{0, 0, 0, 0};
            if (threadIdx.x == 0) {
                lds.lo[turn ^ 1] = ~0u;
                lds.hi[turn ^ 1] = 0;
            }
            __syncthreads();
        }
        asm volatile("" ::: "memory");
        const uint4v mine = *(const uint4v*)&bins[4 * lane];
        const uint32_t sum = mine[0] + mine[1] + mine[2] + mine[3];
        uint32_t above = n - sums_up_to_lane(sum);      // in the lanes above
        uint32_t chosen = 0, more = 0, left = 0;
        bool here = false;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            const bool it = above < want && above + mine[i] >= want;
            chosen = it ? 4 * lane + i : chosen;
            more = it ? above : more;
            left = it ? mine[i] : left;
            here = here || it;
            above += mine[i];
        }
        const int at = __ffsll((long long)__ballot(here)) - 1;
        chosen = (uint32_t)__builtin_amdgcn_readlane((int)chosen, at);
        want -= (uint32_t)__builtin_amdgcn_readlane((int)more, at);
        n = (uint32_t)__builtin_amdgcn_readlane((int)left, at);
        low = ~0u;
        high = 0;
        each([&](float v) {
            const bool in = v >= lo && v <= hi && part(v) == (int)chosen;
            low = min(low, in ? ordered(v) : ~0u);
            high = max(high, in ? ordered(v) : 0);
        });
        low = smallest_of(low);
        high = largest_of(high);
        if (W > 1) {
            if (lane == 0) {
                atomicMin(&lds.lo[turn ^ 1], low);
                atomicMax(&lds.hi[turn ^ 1], high);
            }
            __syncthreads();
            low = lds.lo[turn ^ 1];
            high = lds.hi[turn ^ 1];
        }
        if (number(low) == lo && number(high) == hi)
            return {hi, want};
        lo = number(low);
        hi = number(high);
        if (n == want)
            return {lo, ~0u};
        if (want == 1)
            return {hi, 1};
    }
    return {lo, want};
}

// Where a request's tokens stand: its table, the new tokens' end, its length.
struct Place {
    const int32_t* table;
    int behind, len;
};

__device__ __forceinline__ Place place_of(const Requests& r, int b)
{
    return {r.table + b * r.ld_table, r.offsets[b + 1], length_of(r, b)};
}

// The pages in front of which the one at position p, in a page of its own, chooses
// by score.
__device__ __forceinline__ int scored_before(const Select& a, int p)
{
    return p < 0 ? 0 : max(p / a.r.page - a.local + 1, 0);
}

template <int D>
using Queries = uint8_t[kMostRows][D + 16];

// Rows h0, ... of the `run` tokens' queries (at most 64 rows) in 8 bits: a token a
// wave, or a single token by all W waves.
template <int D, int W>
__device__ __forceinline__ void quantize_queries(Queries<D>& q8, const uint16_t* q, int64_t ld_q, int group, int h0,
                                                 int heads, int run)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll 1
    for (int i = run == 1 ? 0 : wave; i < run; i += W) {
        const uint16_t* qi = q + i * ld_q;
        uint32_t top = 0;
#pragma unroll 1
        for (int x = lane; x < group * D / 8; x += 64) {
            const uint4v w = *(const uint4v*)(qi + 8 * x);
            for (int k = 0; k < 4; ++k)
                top = max(top, max(w[k] << 16 & 0x7fff0000u, w[k] & 0x7fff0000u));
        }
        top = largest_of(top);
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
}

// Sixteen pages for a wave: their keys as the right operand of the products (lane % 16
// the page, 16 (lane / 16) + 64 k .. the dimensions), their exponents.
template <int D>
struct PageTile {
    int4v key[D / 64];
    int exponent;
    bool in;             // a page to be chosen
};

// Loads the tiles of the pages entry[u] (this lane's of each; any number that is none
// reads the cache's first, which must exist). Nothing waits for a load here.
template <int D, int N>
__device__ __forceinline__ void load_pages(PageTile<D> (&t)[N], const Select& a, const int (&entry)[N], int h)
{
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int u = 0; u < N; ++u) {
        t[u].in = entry[u] >= 0 && entry[u] < a.r.num_pages;
        const int64_t at = (int64_t)(t[u].in ? entry[u] : 0) * a.kv_heads + h;
        t[u].exponent = a.exponents[at];
#pragma unroll
        for (int k = 0; k < D / 64; ++k)
            t[u].key[k] = *(const int4v*)(a.keys + at * D + 64 * k + 16 * g);
    }
}

// The scores of a tile's pages: put(token, score) for this lane's page (lane % 16) and
// the tokens below `run` that the lane ends up with.
template <int D, class Put>
__device__ __forceinline__ void compare(const PageTile<D>& t, const Queries<D>& q8, int heads, int bits, int run, Put put)
{
    const int lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
    const int parts = (heads + 15) / 16;
    auto score = [&](int of, int v) {
        if (of < run)
            put(of, t.in ? ldexpf((float)v, min(max(t.exponent, 0), 64)) : -INFINITY);
    };
    // row tiles: several tokens each, or several for a token
#pragma unroll 1
    for (int t0 = 0; t0 < run; t0 += 16 >> bits) {
        const int row0 = min(t0 + (n >> bits), run - 1) * heads, part = n & ((1 << bits) - 1);
        int4v best = {INT32_MIN, INT32_MIN, INT32_MIN, INT32_MIN};
#pragma unroll 1
        for (int p = 0; p < parts; ++p) {
            const uint8_t* row = q8[row0 + min(16 * p + part, heads - 1)] + 16 * g;
            int4v sum = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < D / 64; ++k)
                sum = __builtin_amdgcn_mfma_i32_16x16x64_i8(*(const int4v*)(row + 64 * k), t.key[k], sum, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                best[i] = max(best[i], sum[i]);
        }
        // row 4 g + i of the tile: the token t0 + (4 g + i >> bits)
        if (bits >= 2) {
            int v = max(max(best[0], best[1]), max(best[2], best[3]));
            if (bits >= 3)
                v = max(v, __shfl_xor(v, 16));
            if (bits >= 4)
                v = max(v, __shfl_xor(v, 32));
            if ((4 * g & ((1 << bits) - 1)) == 0)
                score(t0 + (4 * g >> bits), v);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (bits == 0)
                    score(t0 + 4 * g + i, best[i]);
                else if (i % 2 == 0)
                    score(t0 + 2 * g + i / 2, max(best[i], best[i + 1]));
        }
    }
}

// 2^bits rows for a token of `group` heads, at most 16.
__device__ __forceinline__ int bits_of(int group)
{
    int bits = 0;
    while (bits < 4 && 1 << bits < group)
        ++bits;
    return bits;
}

// Writes the list of the token at position p: by one wave (W = 1), or by all of a
// workgroup's. A lane takes pages in a row, an odd number of them (LDS banks): it
// counts, the counts in front of it are summed, then it writes.
template <int W, class Shared>
__device__ __forceinline__ void write_list(Shared& lds, const Select& a, const float* score, int p, int32_t* out)
{
    const int lane = threadIdx.x & 63, wave = W == 1 ? 0 : threadIdx.x >> 6, listed = a.first + a.top + a.local;
    const int pages = p < 0 ? 0 : p / a.r.page + 1, end = max(pages - a.local, 0);
    // up to 512 pages every wave searches for itself, without a barrier
    const Limit l = W == 1 || end - a.first <= 512 ? find_limit<1>(lds, score, a.first, end, a.top)
                                                   : find_limit<W>(lds, score, a.first, end, a.top);
    const int each = (pages + 64 * W - 1) / (64 * W) | 1;
    const int from = min((64 * wave + lane) * each, pages), to = min(from + each, pages);
    auto judge = [&](int j, bool& sure, bool& tie) {
        const bool scored = j >= a.first && j < end;
        const float v = scored ? score[j] : INFINITY;
        sure = !scored || v > l.limit;
        tie = scored && v == l.limit && v != -INFINITY;
    };
    // sure ones, and ties in the upper half: there are at most 32768 pages
    uint32_t count = 0;
#pragma unroll 1
    for (int j = from; j < to; ++j) {
        bool sure, tie;
        judge(j, sure, tie);
        count += sure ? 1 : tie ? 1 << 16 : 0;
    }
    const uint32_t sums = sums_up_to_lane(count);
    uint32_t before = sums - count, all = last_lane(sums);
    if (W > 1) {
        if (lane == 0)
            lds.counts[wave] = all;
        __syncthreads();
        all = 0;
#pragma unroll 1
        for (int w = 0; w < W; ++w) {
            before += w < wave ? lds.counts[w] : 0;
            all += lds.counts[w];
        }
    }
    uint32_t seen = before >> 16, at = (before & 0xffff) + min(seen, l.ties);
#pragma unroll 1
    for (int j = from; j < to; ++j) {
        bool sure, tie;
        judge(j, sure, tie);
        if (sure || (tie && seen < l.ties))
            out[at++] = j;
        seen += !sure && tie;
    }
    const int total = (int)((all & 0xffff) + min(all >> 16, l.ties));
#pragma unroll 1
    for (int i = total + (W == 1 ? lane : threadIdx.x); i < listed; i += 64 * W)
        out[i] = -1;
}

template <int W>
__device__ __forceinline__ void clear(SelectShared<W>& lds)
{
    if (threadIdx.x < 64)
        *(uint4v*)&lds.bins[0][4 * threadIdx.x] = uint4v{0, 0, 0, 0};
    if (threadIdx.x == 0) {
        lds.lo[0] = ~0u;
        lds.hi[0] = 0;
        lds.found = 0;
    }
}

template <int D>
__global__ __launch_bounds__(256, 4) void select_chunk_kernel(Select a)
{
    constexpr int W = 4, kAhead = D > 128 ? 2 : 4;
    extern __shared__ __align__(16) float score[];        // [tokens][pitch]; -inf: not to be chosen
    __shared__ __align__(16) Queries<D> q8;
    __shared__ __align__(16) SelectShared<W> lds;
    const int tid = threadIdx.x, lane = tid & 63, n = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = a.heads / a.kv_heads, listed = a.first + a.top + a.local, bits = bits_of(group);
    const int h = blockIdx.x % a.kv_heads;
    int token = blockIdx.x / a.kv_heads * a.together;
    const int token_end = min(token + a.together, a.tokens);

    // the tokens of one request at a time
    for (int run = 1; token < token_end; token += run) {
        run = 1;
        const int b = sparse::request_of(a.r.offsets, a.r.num_seqs, token);
        if (b < 0)
            continue;
        const Place r = place_of(a.r, b);
        run = min(token_end, r.behind) - token;
        const int pos0 = min(r.len - r.behind + token, r.len - 1), pos1 = min(pos0 + run, r.len) - 1;
        const uint16_t* q = a.q + token * a.ld_q + h * group * D;
        const int before = scored_before(a, pos1);        // for the last of the tokens
        __syncthreads();                                  // the LDS of what came before is read
        clear(lds);

        // scores, of 64 query rows at a time: run * group rows, or the heads of a token
#pragma unroll 1
        for (int h0 = 0; h0 < group; h0 += kMostRows) {
            const int heads = min(group - h0, kMostRows);
            if (h0)
                __syncthreads();
            else
                // places in the cache wait in LDS where the scores go
#pragma unroll 1
                for (int j = a.first + tid; j < before; j += 64 * W)
                    score[j] = __int_as_float(r.table[j]);
            quantize_queries<D, W>(q8, q, a.ld_q, group, h0, heads, run);
            __syncthreads();
            // kAhead tiles of a wave's at a time
#pragma unroll 1
            for (int j0 = a.first + 16 * wave; j0 < before; j0 += 16 * W * kAhead) {
                PageTile<D> tile[kAhead];
                int entry[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int j = min(j0 + 16 * W * u + n, before - 1);
                    entry[u] = h0 ? r.table[j] : __float_as_int(score[j]);
                }
                load_pages(tile, a, entry, h);
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int j = j0 + 16 * W * u + n;
                    if (j - n < before)
                        compare<D>(tile[u], q8, heads, bits, run, [&](int of, float v) {
                            float* at = score + of * a.pitch + j;
                            if (j < before)
                                *at = h0 ? fmaxf(*at, v) : v;
                        });
                }
            }
        }
        __syncthreads();
        int32_t* out = a.pages + ((int64_t)token * a.kv_heads + h) * listed;
        if (run == 1)
            write_list<W>(lds, a, score, pos0, out);
        else
#pragma unroll 1
            for (int i = wave; i < run; i += W)
                write_list<1>(lds, a, score + i * a.pitch, min(pos0 + i, r.len - 1), out + (int64_t)i * a.kv_heads * listed);
    }
}

constexpr int kPagesOfScores = 256;      // that a workgroup of score_pages_kernel takes at a time

template <int D>
__global__ __launch_bounds__(256, 4) void score_pages_kernel(Select a)
{
    constexpr int W = 4, kTiles = kPagesOfScores / 16 / W;
    __shared__ __align__(16) Queries<D> q8;
    const int n = threadIdx.x & 15, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = a.heads / a.kv_heads, bits = bits_of(group);
    const int h = blockIdx.x % a.kv_heads, chunk = blockIdx.x / a.kv_heads % a.chunks;
    int token = blockIdx.x / a.kv_heads / a.chunks * a.together;
    const int token_end = min(token + a.together, a.tokens);
#pragma unroll 1
    for (int run = 1; token < token_end; token += run) {
        run = 1;
        const int b = sparse::request_of(a.r.offsets, a.r.num_seqs, token);
        if (b < 0)
            continue;
        const Place r = place_of(a.r, b);
        run = min(token_end, r.behind) - token;
        const int before = scored_before(a, min(r.len - r.behind + token + run, r.len) - 1);
        const int begin = a.first + chunk * kPagesOfScores + 16 * wave;
        if (begin - 16 * wave >= before)
            continue;
        // table entries and queries are on their way together; a wait for the queries
        // behind the keys would be one for the keys
        auto entries = [&](int first, int (&entry)[kTiles]) {
#pragma unroll
            for (int u = 0; u < kTiles; ++u)
                entry[u] = r.table[min(first + 16 * W * u + n, before - 1)];
        };
        int entry[kTiles];
        entries(begin, entry);
        const uint16_t* q = a.q + token * a.ld_q + h * group * D;
        float* score = a.scores + ((int64_t)token * a.kv_heads + h) * a.pitch;
#pragma unroll 1
        for (int h0 = 0; h0 < group; h0 += kMostRows) {
            const int heads = min(group - h0, kMostRows);
            __syncthreads();                              // the queries of before are read
            quantize_queries<D, W>(q8, q, a.ld_q, group, h0, heads, run);
#pragma unroll 1
            for (int first = begin; first - 16 * wave < before; first += a.chunks * kPagesOfScores) {
                if (first != begin || h0)
                    entries(first, entry);
                PageTile<D> tile[kTiles];
                load_pages(tile, a, entry, h);
                if (first == begin)
                    __syncthreads();
#pragma unroll
                for (int u = 0; u < kTiles; ++u) {
                    const int j = first + 16 * W * u + n;
                    if (j - n < before)
                        compare<D>(tile[u], q8, heads, bits, run, [&](int of, float v) {
                            float* at = score + (int64_t)of * a.kv_heads * a.pitch + j;
                            if (j < before)
                                *at = h0 ? fmaxf(*at, v) : v;
                        });
                }
            }
        }
    }
}

template <int W>
__global__ __launch_bounds__(64 * W) void list_pages_kernel(Select a)
{
    extern __shared__ __align__(16) float score[];
    __shared__ __align__(16) SelectShared<W> lds;
    const int token = blockIdx.x / a.kv_heads;
    // The request that score_pages_kernel has scored the token for: that of the first
    // token of its run. With offsets that fall the token's own may be another one, with
    // pages that nobody has scored.
    Place r;
    for (int at = a.together > 1 ? token - token % a.together : token;;) {
        const int b = sparse::request_of(a.r.offsets, a.r.num_seqs, at);
        if (b < 0) {
            if (at++ == token)
                return;
            continue;
        }
        r = place_of(a.r, b);
        if (r.behind > token)
            break;
        at = r.behind;
    }
    const int p = min(r.len - r.behind + token, r.len - 1), before = scored_before(a, p);
    const float* from = a.scores + (int64_t)blockIdx.x * a.pitch;
    for (int j = a.first + threadIdx.x; j < before; j += 64 * W)
        score[j] = from[j];
    clear(lds);
    __syncthreads();
    write_list<W>(lds, a, score, p, a.pages + (int64_t)blockIdx.x * (a.first + a.top + a.local));
}

// How the work is cut.
struct SelectPlan {
    int together;          // tokens of a workgroup that keeps their scores in LDS
    int chunks;            // workgroups over a token's pages, 0: no such workgroups
    int pitch;
    int64_t workspace;
};

SelectPlan select_plan(int64_t tokens, int32_t heads, int32_t kv_heads, int64_t num_seqs, int64_t max_pages)
{
    SelectPlan p = {1, 0, ((int)max_pages + 3) & ~3, 0};
    // Tokens of long chunks go to a workgroup together, as many as 64 query rows and
    // 16 KB of scores hold, at most 16: four workgroups a compute unit (2048 tokens of
    // 500 pages: 54 us, with 64 KB 71). The table's width stands for the requests' lengths
    // and the batch's average for theirs: a wider table (115 us with 2048 columns, 218 with
    // 2049) and single tokens beside a chunk leave fewer together than would fit.
    const int group = heads / kv_heads;
    while (p.together < 16 && p.together < tokens / (num_seqs < 1 ? 1 : num_seqs) &&
           (p.together + 1) * group <= kMostRows && (int64_t)(p.together + 1) * p.pitch * 4 <= 16384)
        ++p.together;
    // Workgroups for 256 pages at a time, as many as the card holds at once (1024):
    // those of short requests have nothing to do but start (64 requests of up to 1024
    // pages: 2560 of them 16.4 us, 1024 of them 14.5).
    const int64_t bytes = tokens * kv_heads * p.pitch * 4;
    const int64_t items = serving::ceil_div(tokens, (int64_t)p.together) * kv_heads;
    if (items <= 768 && bytes <= 1 << 28) {
        const int64_t most = serving::ceil_div(p.pitch, kPagesOfScores), fit = items < 1 ? 1 : 1024 / items;
        p.chunks = (int)(fit < 1 ? 1 : fit < most ? fit : most);
        p.workspace = bytes;
    }
    return p;
}

template <int D>
void launch_select(const Select& a, hipStream_t stream)
{
    const unsigned items = (unsigned)((a.tokens + (int64_t)a.together - 1) / a.together * a.kv_heads);
    const unsigned lds = (unsigned)(a.together * a.pitch * 4);
    if (a.chunks == 0) {
        hipLaunchKernelGGL((select_chunk_kernel<D>), dim3(items), dim3(256), lds, stream, a);
        return;
    }
    const unsigned lists = (unsigned)(a.tokens * a.kv_heads);
    hipLaunchKernelGGL((score_pages_kernel<D>), dim3(items * a.chunks), dim3(256), 0, stream, a);
    if (a.pitch <= 4096)
        hipLaunchKernelGGL((list_pages_kernel<4>), dim3(lists), dim3(256), a.pitch * 4, stream, a);
    else
        hipLaunchKernelGGL((list_pages_kernel<16>), dim3(lists), dim3(1024), a.pitch * 4, stream, a);
}

bool requests_ok(int64_t num_slots, int32_t page_size, int64_t ld_table, int64_t max_pages, int64_t num_seqs)
{
    return page_size >= 1 && num_slots >= 0 && num_slots % page_size == 0 && max_pages >= 0 && ld_table >= max_pages &&
           num_seqs >= 0 && serving::extent_ok(num_seqs, ld_table, 4);
}

bool select_sizes_ok(int64_t tokens, int32_t heads, int32_t kv_heads, int64_t num_seqs, int64_t max_pages)
{
    return tokens >= 0 && heads >= 1 && kv_heads >= 1 && heads % kv_heads == 0 && num_seqs >= 0 && max_pages >= 0;
}

bool select_sizes_supported(int64_t tokens, int32_t heads, int64_t num_seqs, int64_t max_pages)
{
    return heads <= 1024 && num_seqs <= 65535 && tokens <= (1 << 23) / heads && max_pages <= kMostPages;
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

extern "C" int64_t nvfp4_select_pages_workspace(int64_t tokens, int32_t heads, int32_t kv_heads, int64_t num_seqs,
                                                int64_t max_pages)
{
    if (!select_sizes_ok(tokens, heads, kv_heads, num_seqs, max_pages) ||
        !select_sizes_supported(tokens, heads, num_seqs, max_pages))
        return -1;
    return select_plan(tokens, heads, kv_heads, num_seqs, max_pages).workspace;
}

extern "C" nvfp4_status_t nvfp4_select_pages(const uint16_t* q, int64_t tokens, int64_t ld_q, int32_t heads,
                                             int32_t kv_heads, int32_t head_dim, const int8_t* keys,
                                             const int8_t* exponents, int64_t num_slots, int32_t page_size,
                                             const int32_t* block_table, int64_t ld_table, int64_t max_pages,
                                             const int32_t* seq_lens, const int32_t* query_offsets, int64_t num_seqs,
                                             int32_t top_k, int32_t first, int32_t local, int32_t* pages, void* workspace,
                                             int64_t workspace_bytes, hipStream_t stream)
{
    using namespace serving;
    if (!select_sizes_ok(tokens, heads, kv_heads, num_seqs, max_pages) || top_k < 0 || first < 0 || local < 1 || ld_q < 0 ||
        workspace_bytes < 0 || !requests_ok(num_slots, page_size, ld_table, max_pages, num_seqs))
        return NVFP4_ERROR_INVALID_VALUE;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || !select_sizes_supported(tokens, heads, num_seqs, max_pages) ||
        num_slots > INT32_MAX || max_pages > (1 << 30) / page_size || top_k > kMostListed || first > kMostListed ||
        local > kMostListed || first + top_k + local > kMostListed)
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
    const SelectPlan p = select_plan(tokens, heads, kv_heads, num_seqs, max_pages);
    if (!aligned(workspace, 16))
        return NVFP4_ERROR_MISALIGNED;
    if (workspace_bytes < p.workspace || (p.workspace > 0 && !workspace))
        return NVFP4_ERROR_INVALID_VALUE;
    // A lane without a page reads the cache's first; without a cache it reads q, which is
    // as long as a page's keys, and does not use it.
    if (num_slots == 0)
        keys = exponents = (const int8_t*)q;
    const Select a = {q, keys, exponents, pages, (float*)workspace,
                      {block_table, seq_lens, query_offsets, ld_table, (int)(num_slots / page_size), (int)max_pages,
                       page_size, (int)num_seqs},
                      ld_q, (int)tokens, heads, kv_heads, top_k, first, local, p.together, p.pitch, p.chunks};
    if (head_dim == 64)
        launch_select<64>(a, stream);
    else if (head_dim == 128)
        launch_select<128>(a, stream);
    else
        launch_select<256>(a, stream);
    return launched();
}
