// Attention over the paged NVFP4 cache (include/nvfp4_serving.h).
//
// Both products run on the FP16 matrix cores with FP32 sums, on cache values
// converted in registers (exact in FP16). Global scales are folded into the
// softmax scale and the output.
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

__device__ __forceinline__ void write_split(const Attn& a, const Span& s, int D, int split, int64_t row,
                                            float m, float l)
{
    const int64_t rows = (int64_t)a.tokens * a.heads;
    *(float2*)(a.part + a.splits * rows * D + 2 * (split * rows + row)) = make_float2(m, l);
    if (split == 0)
        used_splits(a, D)[row] = max(1, (s.end - s.begin + s.chunk - 1) / s.chunk);
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
// hidden half come from the cache's first slots and are not used.)
template <int D, bool kPaged16>
__device__ __forceinline__ void load_tile(Tile<D>& t, const Attn& a, const int32_t* table, Entries e,
                                          int h, int t0, int begin, int end, int lane)
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

// Waves a SIMD (workgroups a compute unit) that the registers allow without
// spilling (one row tile of head_dim 128: 62 us for 64 requests with three, 72 with
// two or four).
template <int D, int RT, bool kPaged16>
constexpr int kRowsWaves = RT == 1 && D <= 128 && kPaged16 ? 3 : D * RT <= 256 ? 2 : 1;

template <int D, int RT, bool kPaged16>
__global__ __launch_bounds__(256, (kRowsWaves<D, RT, kPaged16>)) void attn_rows_kernel(Attn a)
{
    using T = Tile<D>;
    constexpr int C = T::C, KF = D / 32, VM = T::VM;
    constexpr int kPad = D + 4;
    __shared__ float o_lds[4][16][kPad];
    __shared__ float m_lds[4][16], l_lds[4][16];

    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, n = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = a.heads / a.kv_heads;

    // Workgroups go to the 8 XCDs in turn. All key/value heads of one range of
    // tokens go to the same XCD one after the other: their rows lie side by
    // side in memory, 64 bytes of codes and 8 of scales each, and share its L2.
    const int per_split = a.num_seqs * a.row_blocks;
    const int j = blockIdx.x >> 3;
    const int work = (j / a.kv_heads) * 8 + (blockIdx.x & 7);
    const int h = j % a.kv_heads;
    if (work >= per_split * a.splits)
        return;
    const int split = work / per_split;
    // requests rotate with the split, so that no XCD gets only first splits
    const int item = (work % per_split + split) % per_split;
    const int b = item / a.row_blocks;
    Span s = request_span(a, b, group);
    const int32_t* table = a.table + b * a.ld_table;
    const float k_scale = a.scale * (a.k_gs ? a.k_gs[0] : 1.0f) * kLog2e;

    for (int row0 = (item % a.row_blocks) * 16 * RT; row0 < s.rows;
         row0 += a.row_blocks * 16 * RT) {
        block_span(a, s, group, row0, 16 * RT);
        const int first = s.begin + split * s.chunk;
        const int last = attention::last_of(first, s.chunk, s.end);
        if (first >= last && split > 0)
            continue;

        // What is loaded goes out in the order in which it is wanted: table
        // entries, query rows, the first tiles; then the rows are converted.
        // Two tiles a wave are in flight, in registers of their own; a tile is
        // requested as soon as the one before in its registers is used up.
        auto entries = [&](int t0) { return kPaged16 ? entries_of(a, table, t0, last) : Entries{}; };
        auto request = [&](Tile<D>& t, Entries e, int t0) {
            if (!kPaged16 && t0 >= last)
                return;
            load_tile<D, kPaged16>(t, a, table, e, h, t0, s.begin, s.end, lane);
            __builtin_amdgcn_sched_barrier(0);      // no use of the other tile moves up here
        };
        int t0 = first + 32 * wave;
        Entries e0 = entries(t0), e1 = entries(t0 + 128);

        uint4v w[RT][KF];
        int lo[RT], hi[RT];
        for (int rt = 0; rt < RT; ++rt) {
            const int r = row0 + 16 * rt + n;
            lo[rt] = hi[rt] = 0;
            // a row behind the last one: the last one's values, nothing to see
            const int rr = min(r, s.rows - 1);
            const uint16_t* src = a.q + (s.first + rr / group) * a.ld_q + (h * group + rr % group) * D;
            for (int f = 0; f < KF; ++f) {
                // D > 64: chunk f / 4, dimensions 32 g + 8 (f % 4); else 16 g + 8 f
                const int d = D > 64 ? 128 * (f / 4) + 32 * g + 8 * (f % 4) : 16 * g + 8 * f;
                w[rt][f] = *(const uint4v*)(src + d);
            }
            if (r < s.rows)
                sees(a, s.len, s.rows / group, r / group, lo[rt], hi[rt]);
        }
        __builtin_amdgcn_sched_barrier(0);
        Tile<D> even, odd;
        request(even, e0, t0);
        request(odd, e1, t0 + 128);
        e0 = entries(t0 + 256);
        e1 = entries(t0 + 384);

        // the query rows as the right operand: lane = row, 8 values a register
        half8v q[RT][KF];
        float factor[RT];
        for (int rt = 0; rt < RT; ++rt) {
            uint32_t top = 0;
            for (int f = 0; f < KF; ++f)
                top = largest_bits(w[rt][f], top);
            top = max(top, (uint32_t)__shfl_xor((int)top, 16));
            top = max(top, (uint32_t)__shfl_xor((int)top, 32));
            const int e = fp16_exponent(top);
            for (int f = 0; f < KF; ++f)
                q[rt][f] = scaled_half8(w[rt][f], e, k_scale < 0);
            factor[rt] = score_factor(k_scale, e);
        }

        float4v o[RT][C][VM];
        float m[RT], l[RT];
        for (int rt = 0; rt < RT; ++rt) {
            m[rt] = -INFINITY;
            l[rt] = 0;
            for (int c = 0; c < C; ++c)
                for (int i = 0; i < VM; ++i)
                    o[rt][c][i] = float4v{0, 0, 0, 0};
        }

        auto compute = [&](const Tile<D>& t, int t0) {
            // S^T = K Q^T
            float4v sc[RT][2];
            for (int hh = 0; hh < 2; ++hh)
                for (int rt = 0; rt < RT; ++rt)
                    sc[rt][hh] = float4v{0, 0, 0, 0};
            for (int c = 0; c < C; ++c) {
                const uint32_t mine = t.shown ? t.ks[c] : 0;
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t w = from_lane(mine, n + 16 * hh + (D > 64 ? 32 * (g >> 1) : 0));
                    w >>= D > 64 ? 16 * (g & 1) : 8 * g;
                    const half2v sk = e4m3x2(w);
                    for (int i = 0; i < T::KW; ++i) {
                        const half8v kf = fp4x8(t.k[hh][c][i], D > 64 ? sk[i >> 1] : sk[0]);
                        for (int rt = 0; rt < RT; ++rt)
                            sc[rt][hh] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                                kf, q[rt][T::KW * c + i], sc[rt][hh], 0, 0, 0);
                    }
                }
            }

            // exponentials: base 2, against the row's reference
            const uint32_t hid = ~(uint32_t)__ballot(t.shown);     // bit j: token j does not count
            const bool whole = hid == 0 && t0 >= s.all_begin && t0 + 32 <= s.all_end;
            half8v p[RT];
            for (int rt = 0; rt < RT; ++rt) {
                float x[8];
                for (int i = 0; i < 8; ++i)
                    x[i] = sc[rt][i >> 2][i & 3];
                float top = largest(x);
                if (!whole) {
                    const uint32_t seen = ~hid & bits_between(lo[rt] - t0, hi[rt] - t0);
                    for (int i = 0; i < 8; ++i) {
                        const int in = 16 * (i >> 2) + 4 * g + (i & 3);
                        x[i] = seen >> in & 1 ? x[i] : -INFINITY;
                    }
                    top = largest(x);
                }
                top *= factor[rt];
                if (__any(top > m[rt] + (kHeadroom + kSlack))) {
                    const float up = fmaxf(m[rt], row_max(top) - kHeadroom);
                    const float f = m[rt] == up ? 1.0f : __builtin_amdgcn_exp2f(m[rt] - up);
                    m[rt] = up;
                    l[rt] *= f;
                    for (int c = 0; c < C; ++c)
                        for (int i = 0; i < VM; ++i)
                            o[rt][c][i] *= f;
                }
                // a row that has seen nothing keeps m = -inf: its terms are 0
                const float base = m[rt] == -INFINITY ? 0.0f : m[rt];
                for (int i = 0; i < 8; ++i) {
                    x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], factor[rt], -base));
                    l[rt] += x[i];
                    p[rt][i] = (_Float16)x[i];
                }
            }

            // O^T += V^T P^T
            for (int c = 0; c < C; ++c) {
                const uint32_t mine = t.shown ? t.vs[c] : 0;
                const uint32_t byte = D > 64 ? (n >> 1) & 3 : n >> 2;
                const uint32_t sel = byte | (4 + byte) << 8 | 0x0c0c0000u;
                half2v sv[4];
                uint32_t even[4], odd[4];       // dimensions 2x, 2x + 1 of token pairs, a byte each
                for (int u = 0; u < 4; ++u) {
                    const int tok = 16 * (u >> 1) + 4 * g + 2 * (u & 1) + (D > 64 ? 32 * (n >> 3) : 0);
                    sv[u] = e4m3x2(__builtin_amdgcn_perm(from_lane(mine, tok + 1), from_lane(mine, tok), sel));
                    const uint32_t x = t.v[2 * u][c], y = t.v[2 * u + 1][c];
                    even[u] = (x & 0x0f0f0f0fu) | (y << 4 & 0xf0f0f0f0u);
                    odd[u] = (x >> 4 & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u);
                }
                for (int i = 0; i < VM; ++i) {
                    const uint32_t* w = i & 1 ? odd : even;
                    const half8v vf = join(fp4x2(w[0], i >> 1) * sv[0], fp4x2(w[1], i >> 1) * sv[1],
                                           fp4x2(w[2], i >> 1) * sv[2], fp4x2(w[3], i >> 1) * sv[3]);
                    for (int rt = 0; rt < RT; ++rt)
                        o[rt][c][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, p[rt], o[rt][c][i], 0, 0, 0);
                }
            }
        };
        for (; t0 < last; t0 += 256) {
            compute(even, t0);
            request(even, e0, t0 + 256);
            e0 = entries(t0 + 512);
            if (t0 + 128 < last)
                compute(odd, t0 + 128);
            request(odd, e1, t0 + 384);
            e1 = entries(t0 + 640);
        }

        // Join the four waves, a row tile at a time.
        for (int rt = 0; rt < RT; ++rt) {
            const float sum = row_sum(l[rt]);
            __syncthreads();
            for (int c = 0; c < C; ++c)
                for (int r = 0; r < 4; ++r)
                    for (int i = 0; i < VM; i += 4)
                        *(float4v*)&o_lds[wave][n][128 * c + VM * (4 * g + r) + i] =
                            float4v{o[rt][c][i][r], o[rt][c][i + 1][r], o[rt][c][i + 2][r], o[rt][c][i + 3][r]};
            if (g == 0) {
                m_lds[wave][n] = m[rt];
                l_lds[wave][n] = sum;
            }
            __syncthreads();
            const int row = tid >> 4, r = row0 + 16 * rt + row;
            if (r >= s.rows)
                continue;
            float top = -INFINITY, total = 0, f[4];
            for (int w = 0; w < 4; ++w)
                top = fmaxf(top, m_lds[w][row]);
            for (int w = 0; w < 4; ++w) {
                f[w] = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m_lds[w][row] - top);
                total += f[w] * l_lds[w][row];
            }
            const int64_t token = s.first + r / group;
            const int head = h * group + r % group;
            const bool whole_row = a.splits == 1;
            const float norm = whole_row ? (total != 0 ? (a.v_gs ? a.v_gs[0] : 1.0f) / total : 0.0f) : 1.0f;
            for (int d = (tid & 15) * 4; d < D; d += 64) {
                float4v v = {0, 0, 0, 0};
                for (int w = 0; w < 4; ++w)
                    v += f[w] * *(float4v*)&o_lds[w][row][d];
                v *= norm;
                if (whole_row)
                    *(uint2v*)(a.out + token * a.ld_out + head * D + d) = uint2v{bf16x2(v[0], v[1]), bf16x2(v[2], v[3])};
                else
                    *(float4v*)(a.part + (((int64_t)split * a.tokens + token) * a.heads + head) * D + d) = v;
            }
            if ((tid & 15) == 0) {
                if (!whole_row) {
                    write_split(a, s, D, split, token * a.heads + head, top, total);
                } else if (a.lse) {
                    a.lse[token * a.heads + head] = total != 0 ? (top + __builtin_amdgcn_logf(total)) * kLn2 : -INFINITY;
                }
            }
        }
    }
}

// ---- many query rows -----------------------------------------------------------
// One workgroup of eight waves per (request, block of 256 query rows, key/value
// head, split), 32 rows a wave. A tile of keys and values (128 tokens; 64 for
// head_dim 256) is converted to FP16 once for all of them and kept in LDS,
// the values transposed; the next tile is converted into a second buffer while
// the waves are at different places of this one, so a tile takes one barrier.
//
// v_mfma_f32_32x32x16_f16, S^T = K Q^T again: a lane holds query row lane % 32
// and, with h = lane / 32, the tokens 8 (r / 4) + 4 h + r % 4 of 32 in its 16
// registers r. The second product, O^T = V^T P^T, sums over 16 tokens at a time,
// its right operand the registers 8 u .. 8 u + 7 as they stand; so a row of V^T
// in LDS keeps each 16 tokens in the order 0-3, 8-11, 4-7, 12-15.
template <int D>
struct Prompt {
    static constexpr int kTokens = D > 128 ? 64 : 128;      // of a tile
    static constexpr int kGroups = kTokens / 32;
    static constexpr int kStep = D > 128 ? 1 : 2;           // groups of 32 tokens a wave takes at once
    // Rows of keys lie 4 banks apart (of 64). Rows of V^T lie 8 banks apart and
    // every eight of them another 4, so that neighbouring rows (reads) as well
    // as every eighth (writes) cover all banks.
    static constexpr int kKeyPitch = D + 8;                 // FP16 elements
    static constexpr int kValPitch = kTokens + 16;
    static constexpr int kVals = D * kValPitch + D;
    static __device__ __forceinline__ int val(int d) { return d * kValPitch + (d >> 3) * 8; }
};

// What a lane loads of a tile: 32 tokens' keys (as in Tile) or values, of one
// 128-wide chunk.
struct Part {
    uint32_t w[8], sc;
    bool shown;
};

template <int D, bool kPaged16>
__device__ __forceinline__ void load_part(Part& t, const Attn& a, const int32_t* table, int h,
                                          int t0, int begin, int end, int lane, bool values, int c)
{
    const int g = lane >> 4, n = lane & 15, tok = lane & 31;
    const uint32_t row = a.kv_heads * (D / 2), srow = a.kv_heads * (D / 16);
    const uint8_t* codes = (values ? a.vp : a.kp) + h * (D / 2) + 64 * c;
    const uint8_t* scales = (values ? a.vs : a.ks) + h * (D / 16) + 8 * c;
    const uint32_t scale_at = D > 64 ? 4 * (lane >> 5) : 0;
    bool shown;
    if (kPaged16) {
        // addresses are a scalar and a lane's fixed offset
        const Entries e = entries_of(a, table, t0, end);
        const Half at[2] = {half_tile(a, e.e[0], t0), half_tile(a, e.e[1], t0 + 16)};
        const uint8_t* half[2] = {codes + at[0].slot * row, codes + at[1].slot * row};
        shown = !(tok < 16 ? at[0].hidden : at[1].hidden);
        t.sc = *(const uint32_t*)(scales + (tok < 16 ? at[0].slot : at[1].slot) * srow + (tok & 15) * srow + scale_at);
        if (values) {
            for (int j = 0; j < 8; ++j) {
                const uint8_t* from = half[j >> 2] + (j & 3) * row;
                t.w[j] = D > 64 ? *(const uint32_t*)(from + (4 * g * row + 4 * n))
                                : *(const uint16_t*)(from + (4 * g * row + 2 * n));
            }
        } else {
            for (int hh = 0; hh < 2; ++hh) {
                if (D > 64) {
                    const uint4v w = *(const uint4v*)(half[hh] + (n * row + 16 * g));
                    for (int i = 0; i < 4; ++i)
                        t.w[4 * hh + i] = w[i];
                } else {
                    const uint2v w = *(const uint2v*)(half[hh] + (n * row + 8 * g));
                    t.w[2 * hh] = w[0];
                    t.w[2 * hh + 1] = w[1];
                }
            }
        }
    } else {
        const int at = t0 + tok;
        const int p = (int)page_of(a, at);
        const int entry = at < end ? table[p] : -1;
        shown = entry >= 0 && entry < a.num_pages;
        const uint32_t s = shown ? entry * a.page + (at - p * a.page) : 0;
        t.sc = *(const uint32_t*)(scales + (uint64_t)s * srow + scale_at);
        if (values) {
            for (int j = 0; j < 8; ++j) {
                const uint64_t from = (uint64_t)from_lane(s, 16 * (j >> 2) + 4 * g + (j & 3)) * row;
                t.w[j] = D > 64 ? *(const uint32_t*)(codes + from + 4 * n) : *(const uint16_t*)(codes + from + 2 * n);
            }
        } else {
            for (int hh = 0; hh < 2; ++hh) {
                const uint64_t from = (uint64_t)from_lane(s, n + 16 * hh) * row;
                if (D > 64) {
                    const uint4v w = *(const uint4v*)(codes + from + 16 * g);
                    for (int i = 0; i < 4; ++i)
                        t.w[4 * hh + i] = w[i];
                } else {
                    const uint2v w = *(const uint2v*)(codes + from + 8 * g);
                    t.w[2 * hh] = w[0];
                    t.w[2 * hh + 1] = w[1];
                }
            }
        }
    }
    t.shown = shown && t0 + tok >= begin && t0 + tok < end;
}

// Converts it into LDS: group `grp` of 32 tokens, chunk c.
template <int D>
__device__ __forceinline__ void store_part(const Part& t, _Float16* keys, _Float16* vals, int grp,
                                           int lane, bool values, int c)
{
    using P = Prompt<D>;
    const int g = lane >> 4, n = lane & 15;
    const uint32_t mine = t.shown ? t.sc : 0;
    if (values) {
        constexpr int VM = D > 64 ? 8 : 4;
        const uint32_t byte = D > 64 ? (n >> 1) & 3 : n >> 2;
        const uint32_t sel = byte | (4 + byte) << 8 | 0x0c0c0000u;
        half2v sv[4];
        uint32_t even[4], odd[4];
        for (int u = 0; u < 4; ++u) {
            const int tok = 16 * (u >> 1) + 4 * g + 2 * (u & 1) + (D > 64 ? 32 * (n >> 3) : 0);
            sv[u] = e4m3x2(__builtin_amdgcn_perm(from_lane(mine, tok + 1), from_lane(mine, tok), sel));
            const uint32_t x = t.w[2 * u], y = t.w[2 * u + 1];
            even[u] = (x & 0x0f0f0f0fu) | (y << 4 & 0xf0f0f0f0u);
            odd[u] = (x >> 4 & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u);
        }
        for (int i = 0; i < VM; ++i) {
            const uint32_t* w = i & 1 ? odd : even;
            const int d = 128 * c + VM * n + i;
            for (int hh = 0; hh < 2; ++hh) {
                // tokens 4 g .. 4 g + 3 of 16: the first half of unit g & 1, or
                // the second (the order 0-3, 8-11, 4-7, 12-15)
                const half2v x = fp4x2(w[2 * hh], i >> 1) * sv[2 * hh];
                const half2v y = fp4x2(w[2 * hh + 1], i >> 1) * sv[2 * hh + 1];
                *(half4v*)(vals + P::val(d) + 32 * grp + 16 * hh + 8 * (g & 1) + 4 * (g >> 1)) =
                    half4v{x[0], x[1], y[0], y[1]};
            }
        }
    } else {
        for (int hh = 0; hh < 2; ++hh) {
            uint32_t w = from_lane(mine, n + 16 * hh + (D > 64 ? 32 * (g >> 1) : 0));
            w >>= D > 64 ? 16 * (g & 1) : 8 * g;
            const half2v sk = e4m3x2(w);
            _Float16* dst = keys + (32 * grp + 16 * hh + n) * P::kKeyPitch + 128 * c + (D > 64 ? 32 : 16) * g;
            for (int i = 0; i < (D > 64 ? 4 : 2); ++i)
                *(half8v*)(dst + 8 * i) = fp4x8(t.w[(D > 64 ? 4 : 2) * hh + i], D > 64 ? sk[i >> 1] : sk[0]);
        }
    }
}

// count matrix instructions, each with an operand read from LDS, `ahead` reads in
// flight before each; left alone, the compiler waits for every read right behind
// it. Vector and scalar arithmetic may move between them.
template <int count, int ahead, typename Read, typename Use>
__device__ __forceinline__ void in_turn(Read read, Use use)
{
    constexpr int kArithmetic = 0x6;
    half8v ring[ahead];
#pragma unroll
    for (int x = 0; x < ahead; ++x)
        ring[x] = read(x);
    __builtin_amdgcn_sched_barrier(kArithmetic);
#pragma unroll
    for (int x = 0; x < count; ++x) {
        use(x, ring[x % ahead]);
        if (x + ahead < count)
            ring[x % ahead] = read(x + ahead);
        __builtin_amdgcn_sched_barrier(kArithmetic);
    }
}

template <int D, bool kPaged16>
__global__ __launch_bounds__(512) void attn_prompt_kernel(Attn a)
{
    using P = Prompt<D>;
    constexpr int kRows = 256, KF = D / 16, MT = D / 32;
    // head_dim 256 has no registers left for more: spilled values are loaded back
    // behind the tile that is in flight, and wait for it (16000 cached tokens, 2000
    // rows of 16 heads: 494 us; two and four reads 524, three and three 580)
    constexpr int kKeysAhead = D > 128 ? 1 : 6, kValsAhead = D > 128 ? 2 : 6;
    __shared__ __attribute__((aligned(16))) _Float16 keys[2][P::kTokens * P::kKeyPitch];
    __shared__ __attribute__((aligned(16))) _Float16 vals[2][P::kVals];
    __shared__ uint32_t shown_lds[2][P::kGroups];

    const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = a.heads / a.kv_heads;
    // each request's blocks from its end: those with the most tokens to see go
    // first, and the short ones fill up the end
    // Workgroups go to the 8 XCDs in turn: requests and heads rotate from one
    // block to the next, so that a long request's do not share an XCD.
    const int pairs = a.num_seqs * a.kv_heads, turn = blockIdx.x / pairs;
    const int pair = (blockIdx.x + turn) % pairs, h = pair % a.kv_heads, b = pair / a.kv_heads;
    const int split = turn % a.splits;
    Span s = request_span(a, b, group);
    const int32_t* table = a.table + b * a.ld_table;
    const float k_scale = a.scale * (a.k_gs ? a.k_gs[0] : 1.0f) * kLog2e;
    // this wave's share of a tile's conversion
    const bool values = wave >= 4;
    const int grp = wave % P::kGroups, chunk = D > 128 ? (wave & 3) >> 1 : 0;

    for (int row0 = ((s.rows - 1) / kRows - turn / a.splits) * kRows; row0 >= 0 && s.rows > 0;
         row0 -= a.row_blocks * kRows) {
        block_span(a, s, group, row0, kRows);
        const int first = s.begin + split * s.chunk;
        const int last = attention::last_of(first, s.chunk, s.end);
        if (first >= last && split > 0)
            continue;

        const int r = row0 + 32 * wave + col;
        half8v q[KF];
        int lo = 0, hi = 0;
        float factor;
        {
            uint4v w[KF];
            uint32_t top = 0;
#pragma unroll
            for (int f = 0; f < KF; ++f)
                w[f] = uint4v{0, 0, 0, 0};
            if (r < s.rows) {
                const uint16_t* src = a.q + (s.first + r / group) * a.ld_q + (h * group + r % group) * D;
#pragma unroll
                for (int f = 0; f < KF; ++f) {
                    w[f] = *(const uint4v*)(src + 16 * f + 8 * half);
                    top = largest_bits(w[f], top);
                }
                sees(a, s.len, s.rows / group, r / group, lo, hi);
            }
            top = max(top, (uint32_t)__shfl_xor((int)top, 32));
            const int e = fp16_exponent(top);
#pragma unroll
            for (int f = 0; f < KF; ++f)
                q[f] = scaled_half8(w[f], e, k_scale < 0);
            factor = score_factor(k_scale, e);
        }
        // the tokens that some, and that all, rows of this wave see
        Span mine = s;
        const bool any_row = row0 + 32 * wave < s.rows;
        if (any_row)
            block_span(a, mine, group, row0 + 32 * wave, 32);

        float16v o[MT];
        float m = -INFINITY, l = 0;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < 16; ++j)
                o[i][j] = 0;

        Part part;
        auto load = [&](int t0) {
            load_part<D, kPaged16>(part, a, table, h, t0 + 32 * grp, s.begin, s.end, lane, values, chunk);
        };
        auto store = [&](int buf) {
            // head_dim 256: LDS addresses are formed anew for each tile, from a lane
            // number that the compiler cannot see through; kept, they would spill
            int x = lane;
            if (D > 128)
                asm volatile("" : "+v"(x));
            store_part<D>(part, keys[buf], vals[buf], grp, x, values, chunk);
            const uint32_t bits = (uint32_t)__ballot(part.shown);
            if (!values && chunk == 0 && lane == 0)
                shown_lds[buf][grp] = bits;
        };
        __syncthreads();            // the row block before may still read
        if (first < last) {
            load(first);
            store(0);
            if (first + P::kTokens < last)
                load(first + P::kTokens);
        }
        for (int t0 = first, buf = 0; t0 < last; t0 += P::kTokens, buf ^= 1) {
            __syncthreads();
#pragma unroll 1
            for (int sub = 0; sub < P::kGroups; sub += P::kStep) {
                constexpr int N = P::kStep;
                const int ts = t0 + 32 * sub;
                if (!any_row || ts >= mine.end || ts + 32 * N <= mine.begin || ts >= last)
                    continue;
                float16v sc[N];
#pragma unroll
                for (int t = 0; t < N; ++t)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        sc[t][j] = 0;
                const _Float16* kf = keys[buf] + (32 * sub + col) * P::kKeyPitch + 8 * half;
                in_turn<KF * N, kKeysAhead>(
                    [&](int x) { return *(const half8v*)(kf + 32 * (x % N) * P::kKeyPitch + 16 * (x / N)); },
                    [&](int x, half8v k) {
                        sc[x % N] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[x / N], sc[x % N], 0, 0, 0);
                    });

                uint32_t shown[N];
                bool whole = ts >= mine.all_begin && ts + 32 * N <= mine.all_end;
#pragma unroll
                for (int t = 0; t < N; ++t) {
                    shown[t] = __builtin_amdgcn_readfirstlane(shown_lds[buf][sub + t]);
                    whole = whole && shown[t] == 0xffffffffu;
                }
                float top = -INFINITY;
#pragma unroll
                for (int t = 0; t < N; ++t)
                    top = fmaxf(top, largest(sc[t]));
                if (!whole) {
                    top = -INFINITY;
#pragma unroll
                    for (int t = 0; t < N; ++t) {
                        const uint32_t seen = shown[t] & bits_between(lo - ts - 32 * t, hi - ts - 32 * t);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const int in = 8 * (j >> 2) + 4 * half + (j & 3);
                            sc[t][j] = seen >> in & 1 ? sc[t][j] : -INFINITY;
                        }
                        top = fmaxf(top, largest(sc[t]));
                    }
                }
                top *= factor;
                if (__any(top > m + (kHeadroom + kSlack))) {
                    const float up = fmaxf(m, fmaxf(top, __shfl_xor(top, 32)) - kHeadroom);
                    const float f = m == up ? 1.0f : __builtin_amdgcn_exp2f(m - up);
                    m = up;
                    l *= f;
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            o[i][j] *= f;
                }
                const float base = m == -INFINITY ? 0.0f : m;
                half8v p[N][2];
#pragma unroll
                for (int t = 0; t < N; ++t)
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float e = __builtin_amdgcn_exp2f(fmaf(sc[t][j], factor, -base));
                        l += e;
                        p[t][j >> 3][j & 7] = (_Float16)e;
                    }
                const _Float16* vf = vals[buf] + P::val(col) + 32 * sub + 8 * half;
                in_turn<2 * MT * N, kValsAhead>(
                    [&](int x) {
                        return *(const half8v*)(vf + P::val(32 * (x % MT)) + 32 * (x / MT >> 1) + 16 * (x / MT & 1));
                    },
                    [&](int x, half8v v) {
                        o[x % MT] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, p[x / MT >> 1][x / MT & 1], o[x % MT], 0, 0, 0);
                    });
            }
            if (t0 + P::kTokens < last) {
                store(buf ^ 1);
                if (t0 + 2 * P::kTokens < last)
                    load(t0 + 2 * P::kTokens);
            }
        }

        const float total = l + __shfl_xor(l, 32);
        if (r < s.rows) {
            const int64_t token = s.first + r / group;
            const int head = h * group + r % group;
            const bool whole_row = a.splits == 1;
            const float norm = whole_row ? (total != 0 ? (a.v_gs ? a.v_gs[0] : 1.0f) / total : 0.0f) : 1.0f;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int d = 32 * i + 8 * j + 4 * half;
                    const float4v v = float4v{o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]} * norm;
                    if (whole_row)
                        *(uint2v*)(a.out + token * a.ld_out + head * D + d) = uint2v{bf16x2(v[0], v[1]), bf16x2(v[2], v[3])};
                    else
                        *(float4v*)(a.part + (((int64_t)split * a.tokens + token) * a.heads + head) * D + d) = v;
                }
            if (half == 0) {
                if (!whole_row) {
                    write_split(a, s, D, split, token * a.heads + head, m, total);
                } else if (a.lse) {
                    a.lse[token * a.heads + head] = total != 0 ? (m + __builtin_amdgcn_logf(total)) * kLn2 : -INFINITY;
                }
            }
        }
    }
}

// Joins the splits of the query rows: kWaves waves a (token, head), which take a
// share of the splits each. Bound by latency: everything it needs to know, which
// rows count and how many splits they have, is loaded at once.
template <int D, int kWaves>
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
    const bool shown = mine && token >= a.offsets[0] && token < a.offsets[a.num_seqs];
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

// ---- host -------------------------------------------------------------------
// Pages of whole 16 tokens are read a half tile at a time, also where nothing is
// there to see; so there must be a page and a table entry.
bool whole_halves(const Attn& a) { return a.page % 16 == 0 && a.num_pages > 0 && a.max_pages > 0; }

template <int D, int RT>
void launch_rows(const Attn& a, dim3 grid, hipStream_t stream)
{
    if (whole_halves(a))
        hipLaunchKernelGGL((attn_rows_kernel<D, RT, true>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((attn_rows_kernel<D, RT, false>), grid, dim3(256), 0, stream, a);
}

template <int D>
void launch(const Attn& a, int block, hipStream_t stream)
{
    const int64_t work = (int64_t)a.num_seqs * a.row_blocks * a.splits;
    const dim3 grid((unsigned)((work + 7) / 8 * 8 * a.kv_heads));
    if (block == 256) {
        const dim3 all((unsigned)(work * a.kv_heads));
        if (whole_halves(a))
            hipLaunchKernelGGL((attn_prompt_kernel<D, true>), all, dim3(512), 0, stream, a);
        else
            hipLaunchKernelGGL((attn_prompt_kernel<D, false>), all, dim3(512), 0, stream, a);
    } else if (block == 16) {
        launch_rows<D, 1>(a, grid, stream);
    } else if constexpr (D <= 128) {
        if (block == 32)
            launch_rows<D, 2>(a, grid, stream);
        else if (block == 48)
            launch_rows<D, 3>(a, grid, stream);
        else
            launch_rows<D, 4>(a, grid, stream);
    }
    if (a.splits > 16)
        hipLaunchKernelGGL((attn_join_kernel<D, 4>), dim3((unsigned)(a.tokens * a.heads)), dim3(256), 0, stream, a);
    else if (a.splits > 1)
        hipLaunchKernelGGL((attn_join_kernel<D, 1>), dim3((unsigned)(a.tokens * a.heads + 3) / 4), dim3(256), 0, stream, a);
}

bool sizes_ok(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t head_dim, int64_t num_seqs,
              int64_t max_query_len, int64_t max_seq_len, int64_t window)
{
    return tokens >= 0 && num_seqs >= 0 && max_query_len >= 0 && max_seq_len >= 0 && window >= 0 &&
           heads >= 1 && kv_heads >= 1 && heads % kv_heads == 0;
}

bool sizes_supported(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t head_dim,
                     int64_t num_seqs)
{
    return (head_dim == 64 || head_dim == 128 || head_dim == 256) && heads <= 1024 &&
           num_seqs <= 65535 && num_seqs * kv_heads <= (1 << 22) && tokens <= (1 << 30) / heads;
}

}  // namespace

extern "C" int64_t nvfp4_paged_attention_workspace(int64_t tokens, int32_t heads, int32_t kv_heads,
                                                   int32_t head_dim, int64_t num_seqs,
                                                   int64_t max_query_len, int64_t max_seq_len,
                                                   int64_t window)
{
    if (!sizes_ok(tokens, heads, kv_heads, head_dim, num_seqs, max_query_len, max_seq_len,
                  window) ||
        !sizes_supported(tokens, heads, kv_heads, head_dim, num_seqs))
        return -1;
    const Plan p = make_plan(tokens, heads, kv_heads, head_dim, num_seqs, max_query_len, max_seq_len, window);
    // a split's outputs and (reference, sum) pairs of every row, and the rows' splits
    return p.splits > 1 ? tokens * heads * 4 * ((head_dim + 2) * p.splits + 1) : 0;
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
    if (!sizes_supported(tokens, heads, kv_heads, head_dim, num_seqs) || num_slots > INT32_MAX ||
        max_pages > (1 << 30) / page_size)
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
    const Plan p = make_plan(tokens, heads, kv_heads, head_dim, num_seqs, max_query_len, max_seq_len, window);
    Attn a = {q, k_packed, k_scales, v_packed, v_scales, block_table, seq_lens, query_offsets,
              k_gs, v_gs, out, lse, (float*)workspace, ld_q, ld_out, ld_table,
              window > INT32_MAX ? 0 : window,      // which hides nothing
              (int)tokens,
              heads, kv_heads, page_size, (int)(num_slots / page_size), (int)max_pages,
              (int)num_seqs, causal, scale};
    int shift = 0;
    while (((int64_t)1 << shift) < page_size)
        ++shift;
    a.page_shift = 31 + shift;
    a.page_magic = (uint32_t)((((uint64_t)1 << a.page_shift) + page_size - 1) / page_size);
    a.splits = p.splits;
    a.chunk = p.chunk;
    a.row_blocks = p.row_blocks;
    if (head_dim == 64)
        launch<64>(a, p.block, stream);
    else if (head_dim == 128)
        launch<128>(a, p.block, stream);
    else
        launch<256>(a, p.block, stream);
    return launched();
}
