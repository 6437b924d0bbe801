// Attention over pages of the NVFP4 cache for few query rows: what the kernels of
// paged_attention.hip and sparse_attention.hip share. A tile of 32 tokens is loaded
// by a wave (load_tile), its scores, exponentials and products are added up in
// registers (attend_tile.inc), a workgroup's waves are joined (join_waves.inc), and
// the parts of a range that was split over workgroups are joined by a kernel of its
// own (attn_join_kernel).
#pragma once

#include "attention_plan.hpp"
#include "fp4_operand.hpp"

namespace {

using namespace fp4op;
using attention::make_plan;
using attention::Plan;

typedef _Float16 half4v __attribute__((ext_vector_type(4)));
typedef float float16v __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;

struct Attn {
    const uint16_t* q;
    const uint8_t *kp, *ks, *vp, *vs;
    const int32_t *table, *lens, *offsets;
    const float *k_gs, *v_gs;
    uint16_t* out;
    float* lse;
    float* part;       // workspace
    int64_t ld_q, ld_out, ld_table, window;
    int tokens, heads, kv_heads, page, num_pages, max_pages, num_seqs, causal;
    float scale;
    uint32_t page_magic, page_shift;   // t / page == t * magic >> shift for 0 <= t < 2^31
    int splits, chunk, row_blocks;
};

// What the rows of one block of a request see, and how a long range of tokens
// is cut into splits. The same for the kernel that computes a split and the
// one that joins them.
struct Span {
    int first, rows, len;      // first row of q, query rows (tokens x group), cached tokens
    int begin, end, chunk;     // tokens that some row of the block sees (begin: a multiple of 32)
    int all_begin, all_end;    // tokens that every row of the block sees
};

__device__ __forceinline__ Span request_span(const Attn& a, int b, int group)
{
    Span s;
    s.first = min(max(a.offsets[b], 0), a.tokens);
    s.rows = (min(max(a.offsets[b + 1], s.first), a.tokens) - s.first) * group;
    s.len = a.num_pages > 0 ? min(max(a.lens[b], 0), a.max_pages * a.page) : 0;
    return s;
}

// The tokens [lo, hi) that query `i` of `n` sees.
__device__ __forceinline__ void sees(const Attn& a, int len, int n, int i, int& lo, int& hi)
{
    const int pos = len - n + i;
    hi = a.causal ? min(pos + 1, len) : len;
    lo = a.window > 0 ? (int)max((int64_t)pos - a.window + 1, (int64_t)0) : 0;
}

__device__ __forceinline__ void block_span(const Attn& a, Span& s, int group, int row0, int block)
{
    const int n = s.rows / group;
    int lo0, hi0, lo1, hi1;
    sees(a, s.len, n, row0 / group, lo0, hi0);
    sees(a, s.len, n, min(row0 + block, s.rows) / group - (min(row0 + block, s.rows) % group == 0),
         lo1, hi1);
    s.begin = lo0 & ~31;
    s.end = max(hi1, s.begin);
    s.all_begin = lo1;
    s.all_end = hi0;
    s.chunk = attention::chunk_of(a.chunk, a.splits, s.end - s.begin);
}

// The workspace: each split's output rows, its (reference, sum) pairs, and, written
// by split 0, how many splits a row has.
__device__ __forceinline__ int* used_splits(const Attn& a, int D)
{
    return (int*)(a.part + (int64_t)a.splits * a.tokens * a.heads * (D + 2));
}

// Writes a row's reference and sum of one split.
__device__ __forceinline__ void write_part(const Attn& a, int D, int split, int64_t row, float m, float l)
{
    const int64_t rows = (int64_t)a.tokens * a.heads;
    *(float2*)(a.part + a.splits * rows * D + 2 * (split * rows + row)) = make_float2(m, l);
}

__device__ __forceinline__ uint32_t page_of(const Attn& a, uint32_t t)
{
    return (uint32_t)(((uint64_t)t * a.page_magic) >> a.page_shift);
}

__device__ __forceinline__ uint32_t from_lane(uint32_t v, int lane)
{
    return (uint32_t)__builtin_amdgcn_ds_bpermute(lane * 4, (int)v);
}

// Largest / sum over the four lanes that hold one query row (lane % 16).
__device__ __forceinline__ float row_max(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}

__device__ __forceinline__ float row_sum(float v)
{
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Largest of a matrix result's registers. The asm keeps it where it is written,
// right behind the matrix instructions: compiled code that first reads their
// result behind a branch has been seen to read it too early (the wait states
// on the path that takes the branch were missing), with wrong scores.
template <int N, class T>
__device__ __forceinline__ float largest_of(const T& v)
{
    float top = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i)
        top = fmaxf(top, v[i]);
    asm volatile("" : "+v"(top));
    return top;
}

__device__ __forceinline__ float largest(const float (&v)[8]) { return largest_of<8>(v); }
__device__ __forceinline__ float largest(const float16v& v) { return largest_of<16>(v); }

// A query row's values for one matrix operand: BF16 to FP16 with the row's
// power of two 2^e and, for a negative scale, its sign.
__device__ __forceinline__ half8v scaled_half8(uint4v w, int e, bool negative)
{
    const float f = negative ? -ldexpf(1.0f, e) : ldexpf(1.0f, e);
    half8v r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[2 * i] = (_Float16)(__uint_as_float(w[i] << 16) * f);
        r[2 * i + 1] = (_Float16)(__uint_as_float(w[i] & 0xffff0000u) * f);
    }
    return r;
}

// What a product with such a row is multiplied by to give its score in base 2:
// positive, so that the largest product gives the largest score, and not 0, which
// would turn a hidden token's -inf into NaN. A NaN stays one.
__device__ __forceinline__ float score_factor(float k_scale, int e)
{
    const float f = ldexpf(fabsf(k_scale), -e);
    return f < 0x1p-126f ? 0x1p-126f : f;
}

__device__ __forceinline__ uint32_t largest_bits(uint4v w, uint32_t top)
{
    for (int i = 0; i < 4; ++i)
        top = max(top, max((w[i] << 16) & 0x7fff0000u, w[i] & 0x7fff0000u));
    return top;
}

// The bits from, ..., to - 1 of 32.
__device__ __forceinline__ uint32_t bits_between(int from, int to)
{
    const uint32_t below_to = to <= 0 ? 0 : ~0u >> (32 - min(to, 32));
    return from >= 32 ? 0 : below_to & (~0u << max(from, 0));
}

// ---- few query rows ----------------------------------------------------------
// One workgroup per (request, block of 16 RT query rows, key/value head,
// split of the tokens); query rows are tokens x the heads that share the
// key/value head. Its four waves take tiles of 32 tokens in turn, each with
// its own reference, sum and output, joined through LDS at the end.
//
// Scores are computed transposed, S^T = K Q^T (v_mfma_f32_16x16x32_f16): a lane
// holds one query row (lane % 16) and the tokens 4 (lane / 16) + r of each
// half tile, which is the layout of the second product's right operand as it
// stands if that product sums over the tokens in the order (half 0: 4g .. 4g+3,
// half 1: 4g .. 4g+3) for lane group g. Its left operand V^T needs, per lane,
// eight tokens of one dimension: a lane loads the same 8 dimensions of its
// eight tokens and pairs their codes by two nibble merges per token pair; the
// conversion then picks a byte (a dimension) of each pair. So nothing crosses
// lanes but the scale bytes.
//
// Exponentials are taken in base 2 against a reference of each row that stands
// kHeadroom below the largest score at the time it was set, and that is raised
// only when a score exceeds that score by more than kSlack; most tiles then need
// no rescaling and no exchange. Probabilities therefore reach 2^15, what FP16
// holds, and they lose bits only below 2^-14: their rounding is off by at most
// 2^-11 relative or 2^-25 absolute, 2^-36 of the row's largest. Without the
// headroom whatever lies 25 powers of two below the largest would vanish from
// the product with v, however many tokens there are, and stay in the sum. (A
// slack of 4 costs nothing against 8; 2 takes 2000 rows of head_dim 256 behind
// 16000 tokens from 455 to 463 us.)
constexpr float kSlack = 4.0f, kHeadroom = 15.0f - kSlack;

template <int D>
struct Tile {
    static constexpr int C = D > 64 ? D / 128 : 1;    // 128-wide chunks
    static constexpr int KW = D > 64 ? 4 : 2;         // words of a lane's keys per chunk
    static constexpr int VM = D > 64 ? 8 : 4;         // dimensions of a lane's values per chunk
    uint32_t k[2][C][KW];
    uint32_t v[8][C];
    uint32_t ks[C], vs[C];
    bool shown;                                       // this lane's token (lane % 32) counts
};

// The table entries of a tile's two halves of 16 tokens if each lies in one page
// (page_size a multiple of 16), -1 behind `last`. Read through the scalar
// cache (the table does not change while a kernel runs): a vector load of
// them would have to wait for every load of keys and values before it.
struct Entries {
    int e[2];
};

__device__ __forceinline__ Entries entries_of(const Attn& a, const int32_t* table, int t0, int last)
{
    typedef const int32_t __attribute__((address_space(4)))* scalar_ptr;
    Entries r;
    for (int hh = 0; hh < 2; ++hh) {
        const int t = t0 + 16 * hh;
        const int p = (int)page_of(a, max(t, 0));
        const bool in = t < last && p < a.max_pages;
        const int entry = ((scalar_ptr)table)[in ? p : 0];
        r.e[hh] = in ? entry : -1;
    }
    return r;
}

// The slot of a half's first token; 0 with `hidden` set where its page does not
// count.
struct Half {
    int64_t slot;
    bool hidden;
};

__device__ __forceinline__ Half half_tile(const Attn& a, int entry, int first)
{
    Half h;
    h.hidden = entry < 0 || entry >= a.num_pages;
    h.slot = h.hidden ? 0 : (int64_t)entry * a.page + (first - (int)page_of(a, first) * a.page);
    return h;
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000);
}

// Loads the tile at t0. kPaged16: codes through a buffer of the half's 16 slots,
// or of none where it is hidden, which reads as 0 without a memory access; so a
// tile behind the last one can be requested without a branch. (Scales of a
// hidden half come from the cache's first slots and are not used.) Otherwise
// table[p] is the entry of page p of the range.
template <int D, bool kPaged16, class Table>
__device__ __forceinline__ void load_tile(Tile<D>& t, const Attn& a, Table table, Entries e, int h, int t0,
                                          int begin, int end, int lane)
{
    using T = Tile<D>;
    const int g = lane >> 4, n = lane & 15, tok = lane & 31;
    const uint32_t row = a.kv_heads * (D / 2), srow = a.kv_heads * (D / 16);
    const uint8_t* kp = a.kp + h * (D / 2);
    const uint8_t* vp = a.vp + h * (D / 2);
    const uint8_t* ks = a.ks + h * (D / 16);
    const uint8_t* vs = a.vs + h * (D / 16);
    uint64_t mine;                 // slot of this lane's token
    if (kPaged16) {
        const Half half[2] = {half_tile(a, e.e[0], t0), half_tile(a, e.e[1], t0 + 16)};
        t.shown = !(tok < 16 ? half[0].hidden : half[1].hidden);
        mine = (uint64_t)(tok < 16 ? half[0].slot : half[1].slot) + (tok & 15);
        for (int hh = 0; hh < 2; ++hh) {
            const uint32_t bytes = half[hh].hidden ? 0 : 16 * row;
            const __amdgpu_buffer_rsrc_t k = buffer(kp + half[hh].slot * row, bytes);
            const __amdgpu_buffer_rsrc_t v = buffer(vp + half[hh].slot * row, bytes);
            for (int c = 0; c < T::C; ++c) {
                if (D > 64) {
                    const auto w = __builtin_amdgcn_raw_buffer_load_b128(k, n * row + 16 * g + 64 * c, 0, 0);
                    for (int i = 0; i < 4; ++i)
                        t.k[hh][c][i % T::KW] = w[i];
                } else {
                    const auto w = __builtin_amdgcn_raw_buffer_load_b64(k, n * row + 8 * g, 0, 0);
                    t.k[hh][c][0] = w[0];
                    t.k[hh][c][1] = w[1];
                }
                for (int j = 0; j < 4; ++j)
                    t.v[4 * hh + j][c] =
                        D > 64 ? (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(v, 4 * g * row + 4 * n + 64 * c, j * row, 0)
                               : (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(v, 4 * g * row + 2 * n, j * row, 0);
            }
        }
    } else {
        const int at = t0 + tok;
        const int p = (int)page_of(a, at);
        const int entry = at < end ? table[p] : -1;
        t.shown = entry >= 0 && entry < a.num_pages;
        const uint32_t slot = t.shown ? entry * a.page + (at - p * a.page) : 0;
        mine = slot;
        for (int c = 0; c < T::C; ++c) {
            for (int hh = 0; hh < 2; ++hh) {
                const uint8_t* from = kp + (uint64_t)from_lane(slot, n + 16 * hh) * row + 64 * c + (D > 64 ? 16 : 8) * g;
                if (D > 64) {
                    const uint4v w = *(const uint4v*)from;
                    for (int i = 0; i < 4; ++i)
                        t.k[hh][c][i % T::KW] = w[i];
                } else {
                    const uint2v w = *(const uint2v*)from;
                    t.k[hh][c][0] = w[0];
                    t.k[hh][c][1] = w[1];
                }
            }
            for (int j = 0; j < 8; ++j) {
                const uint8_t* from = vp + (uint64_t)from_lane(slot, 16 * (j >> 2) + 4 * g + (j & 3)) * row + 64 * c +
                                      (D > 64 ? 4 : 2) * n;
                t.v[j][c] = D > 64 ? *(const uint32_t*)from : *(const uint16_t*)from;
            }
        }
    }
    t.shown = t.shown && t0 + tok >= begin && t0 + tok < end;
    // scales: a lane takes 4 bytes of its token (the second half of the wave the
    // next 4), handed to the lanes that need them when used
    for (int c = 0; c < T::C; ++c) {
        const uint64_t at = mine * srow + (D > 64 ? 8 * c + 4 * (lane >> 5) : 0);
        t.ks[c] = *(const uint32_t*)(ks + at);
        t.vs[c] = *(const uint32_t*)(vs + at);
    }
}

// Joins the splits of the query rows: kWaves waves a (token, head), which take a
// share of the splits each. Bound by latency: everything it needs to know, which
// rows count and how many splits they have, is loaded at once. A row counts where its
// token is a request's, or (kMarked) where it has splits.
template <int D, int kWaves, bool kMarked>
__global__ __launch_bounds__(256) void attn_join_kernel(Attn a)
{
    constexpr int kLanes = D / 4, kAtOnce = 64 / kLanes * kWaves;    // lanes a row of D; splits read at once
    constexpr int kRows = 4 / kWaves;
    __shared__ float4v o_lds[4][kLanes];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t rows = (int64_t)a.tokens * a.heads;
    const int64_t row = (int64_t)blockIdx.x * kRows + wave / kWaves;
    const bool mine = row < rows;
    const int64_t at = mine ? row : 0;
    const int token = (int)(at / a.heads), head = (int)(at % a.heads);
    const int used = min(max(used_splits(a, D)[at], 0), a.splits);
    const float* ml = a.part + a.splits * rows * D;
    float m[4], l[4], top = -INFINITY;
    for (int i = 0; i < 4; ++i) {
        const int split = 64 * i + lane;
        m[i] = -INFINITY;
        l[i] = 0;
        if (split < a.splits) {
            const float2 v = *(const float2*)(ml + 2 * (split * rows + at));
            m[i] = split < used ? v.x : -INFINITY;
            l[i] = split < used ? v.y : 0.0f;
        }
        top = fmaxf(top, m[i]);
    }
    const bool shown = mine && (kMarked ? used > 0 : token >= a.offsets[0] && token < a.offsets[a.num_seqs]);
    for (int d = 32; d; d >>= 1)
        top = fmaxf(top, __shfl_xor(top, d));
    float total = 0;
    for (int i = 0; i < 4; ++i) {
        m[i] = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[i] - top);
        total += m[i] * l[i];
    }
    for (int d = 32; d; d >>= 1)
        total += __shfl_xor(total, d);

    const int x = lane % kLanes, first = wave % kWaves * (64 / kLanes) + lane / kLanes;
    float4v o = {0, 0, 0, 0};
    for (int i = 0; i < 4; ++i) {
        // the splits 64 i .. 64 i + 63, whose weights the lanes' m[i] hold
        const int n = min(used - 64 * i, 64);
        for (int base = 0; base < n; base += 4 * kAtOnce) {
            float4v v[4];
            float f[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int k = base + u * kAtOnce + first;
                f[u] = __shfl(m[i], k & 63);
                v[u] = float4v{0, 0, 0, 0};
                if (k < n)
                    v[u] = *(const float4v*)(a.part + ((64 * i + k) * rows + at) * D + 4 * x);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                o += f[u] * v[u];
        }
    }
    for (int d = kLanes; d < 64; d <<= 1)
        for (int j = 0; j < 4; ++j)
            o[j] += __shfl_xor(o[j], d);
    if (kWaves > 1) {
        if (lane < kLanes)
            o_lds[wave][lane] = o;
        __syncthreads();
        o = float4v{0, 0, 0, 0};
        for (int w = 0; w < kWaves; ++w)
            o += o_lds[wave / kWaves * kWaves + w][x];
    }
    if (shown && wave % kWaves == 0 && lane < kLanes) {
        o *= total != 0 ? (a.v_gs ? a.v_gs[0] : 1.0f) / total : 0.0f;
        *(uint2v*)(a.out + token * a.ld_out + head * D + 4 * x) = uint2v{bf16x2(o[0], o[1]), bf16x2(o[2], o[3])};
        if (x == 0 && a.lse)
            a.lse[row] = total != 0 ? (top + __builtin_amdgcn_logf(total)) * kLn2 : -INFINITY;
    }
}

}  // namespace
