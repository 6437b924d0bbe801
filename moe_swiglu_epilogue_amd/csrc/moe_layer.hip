// A whole mixture-of-experts layer for a few tokens (include/nvfp4_serving.h).
//
// Bound by memory: every weight of the reached experts is read once. Three
// kernels. The first two are one grouped product each, h = swiglu(x W1^T) and
// y = h W2^T, with a workgroup per (expert, 64 weight rows); a row tile of 16
// weights stands in the left operand of the matrix instructions, straight from
// memory, the expert's tokens in the right one, from LDS. The third adds up a
// token's top_k rows of y with the routing weights. The first finds the
// routing itself: each workgroup counts, for the tokens, how many logits stand
// before its expert's. (In every workgroup, which with many experts costs more
// than the weights: 4096 x 1024, top 8, 32 tokens, 60 reached of 64 experts 114 us,
// 178 reached of 512 627 us.)
#include "fp4_operand.hpp"
#include "serving_common.hpp"

namespace {

using namespace fp4op;

typedef __bf16 bf8v __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;
constexpr int kMaxTokens = 64, kMaxExperts = 512, kMaxTopK = 32;

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
    float* y;          // workspace: [tokens * top_k][hidden]
    int64_t ld_x, ld_out;
    int tokens, hidden, inter, experts, top_k, renormalize;
    int by_pair;       // workgroups go by (token, rank) pairs, not by experts
};

// A logit as it is compared: NaN stands behind everything, with -inf.
__device__ __forceinline__ float logit(const Moe& a, int t, int e)
{
    const float v = a.logits[t * a.experts + e];
    return v == v ? v : -INFINITY;
}

// The pairs (token * top_k + rank) routed to a workgroup's expert, in the order
// of the tokens.
struct Group {
    int pairs[kMaxTokens];
    int count, expert;
    int part[kThreads / 64][kMaxTokens];
    float row[kMaxExperts];
};

// The expert with rank slot % top_k for token slot / top_k: four lanes an
// expert count the logits in front of its own.
__device__ int expert_of_pair(const Moe& a, Group& s, int slot, int tid)
{
    const int t = slot / a.top_k, k = slot % a.top_k;
    for (int f = tid; f < a.experts; f += kThreads)
        s.row[f] = logit(a, t, f);
    __syncthreads();
    for (int f = tid >> 2; f < a.experts; f += kThreads / 4) {
        const float v = s.row[f];
        int rank = 0;
#pragma unroll 4
        for (int u = tid & 3; u < a.experts; u += 4) {
            const float w = s.row[u];
            rank += w > v || (w == v && u < f);
        }
        rank += __shfl_xor(rank, 1);
        rank += __shfl_xor(rank, 2);
        if (rank == k)
            s.expert = f;
    }
    __syncthreads();
    return s.expert;
}

// Collects the tokens that the lanes of wave 0 report (lane = token).
__device__ __forceinline__ void collect(const Moe& a, Group& s, bool in, int rank, int lane)
{
    const uint64_t all = __ballot(in);
    if (in)
        s.pairs[__popcll(all & ((1ull << lane) - 1))] = lane * a.top_k + rank;
    if (lane == 0)
        s.count = __popcll(all);
}

// The pairs of expert e from the logits: lane = token, each wave counts a
// quarter of the experts. A workgroup told to also writes the ids of its
// expert (of its own pair alone, where it goes by pairs).
__device__ void route(const Moe& a, Group& s, int slot, int e, bool write, int tid)
{
    const int lane = tid & 63, wave = tid >> 6;
    const float v = lane < a.tokens ? logit(a, lane, e) : -INFINITY;
    int rank = 0;
    if (lane < a.tokens) {
        const int quarter = (a.experts + 3) / 4, last = min(a.experts, (wave + 1) * quarter);
#pragma unroll 8
        for (int f = wave * quarter; f < last; ++f) {
            const float u = logit(a, lane, f);
            rank += u > v || (u == v && f < e);
        }
    }
    s.part[wave][lane] = rank;
    __syncthreads();
    if (wave == 0) {
        rank = s.part[0][lane] + s.part[1][lane] + s.part[2][lane] + s.part[3][lane];
        const bool in = lane < a.tokens && rank < a.top_k;
        if (write && in && (!a.by_pair || lane * a.top_k + rank == slot))
            a.ids[lane * a.top_k + rank] = v == -INFINITY ? -1 : e;
        collect(a, s, in && v != -INFINITY, rank, lane);
    }
    __syncthreads();
}

// The same from the ids that the first kernel wrote.
__device__ void routed(const Moe& a, Group& s, int e, int tid)
{
    const int lane = tid & 63;
    if (tid < 64) {
        int rank = kMaxTopK;
        if (lane < a.tokens)
#pragma unroll 8
            for (int k = 0; k < a.top_k; ++k)
                if (a.ids[lane * a.top_k + k] == e)
                    rank = k;
        collect(a, s, e >= 0 && rank < a.top_k, rank, lane);
    }
    __syncthreads();
}

// Chunk of the summed axis that is staged at a time, and what a lane (g = lane /
// 16, n = lane % 16) feeds the matrix instructions of a 16-row weight tile:
// row n; NVFP4: step s is 16 bytes, k = 128 s + 32 g .. + 31, with two scale
// bytes; BF16: 16 bytes, k = 32 s + 8 g .. + 7. The loads are made by lane 4 n +
// g instead, so that four neighbouring lanes read 64 bytes of one row, and
// handed over in registers: loaded by the lane that needs them, neighbouring
// lanes read 16 different rows and every load takes the L1 64 accesses for 16
// (32 tokens: 218 and 128 us against 199 and 116 for the two products).
template <bool kFp4, bool kDown, int NT>
struct Shape {
    // the longer axis of the first product takes the longer chunk (one token:
    // 28 us with 512, 32 with 256; second product 18 and 16); the two halves of h
    // a shorter one, so that more workgroups fit into LDS (57 tokens, BF16: 46 us
    // with 256, 40 with 128; no difference for 3 tokens)
    static constexpr int KC = kFp4 ? (NT == 1 && !kDown ? 512 : 256) : kDown ? 128 : 256;
    static constexpr int kRun = kFp4 ? 128 : 32;       // k of a step
    static constexpr int S = KC / kRun;
    static constexpr int kPitch = KC + 8;              // 16-bit elements: rows 4 banks apart
};

// Scales: a lane's two bytes of each step, or (kWide, for a summed axis of whole
// steps) 8 bytes of one step of its row, the one with the lane's group's
// number, which are dealt to the four groups when they are used. Loaded step by
// step, the scales of 16 rows take 16 cache lines for 8 bytes each time, which
// are gone from the L1 when the next step wants them (one token: 39 us against
// 28 for the first product).
template <bool kFp4, bool kDown, int NT, bool kWide>
struct Weights {
    uint4v w[Shape<kFp4, kDown, NT>::S];
    uint16_t sc[kFp4 && !kWide ? Shape<kFp4, kDown, NT>::S : 1];
    uint2v wide;
};

// All loads of the product loop are buffer loads, issued whether or not there
// is something to load: what lies behind the summed axis or the last token
// gets an offset out of the buffer's range, which reads as 0 without a memory
// access. So the loop has no branch around a load, behind which the compiler
// would have to wait for everything in flight. The scalar offset, k's part, is
// 0 behind the axis: it never passes the buffer's end, so that a lane's offset
// alone is out of range whichever way the range check counts the scalar one.
constexpr uint32_t kOutside = 0x7fffff00u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000);
}

// A row tile's weights and scales, and where a lane's part of them lies,
// relative to the tile's first row.
struct Tile {
    const uint8_t *w, *sc;
    uint32_t w_bytes, sc_bytes, w_at, sc_at;
};

// kWide (and BF16, whose steps are 32 long): a step lies before or behind the
// end of the axis as a whole, so that the scalar unit alone handles it, with a
// buffer of no bytes; a lane's offsets never change.
template <bool kFp4, bool kDown, int NT, bool kWide>
__device__ __forceinline__ void load_weights(Weights<kFp4, kDown, NT, kWide>& r, const Tile& t, int k0, int K, int g)
{
    using X = Shape<kFp4, kDown, NT>;
    if (kFp4 && kWide) {
        const int k = k0 + 128 * (g & (X::S - 1));
        r.wide = __builtin_bit_cast(uint2v, __builtin_amdgcn_raw_buffer_load_b64(
            buffer(t.sc, t.sc_bytes), k < K ? t.sc_at : kOutside, k0 < K ? k0 / 16 : 0, 0));
    }
    for (int s = 0; s < X::S; ++s) {
        const int k = k0 + X::kRun * s, at = k < K ? k : 0;
        if (kWide || !kFp4) {
            r.w[s] = __builtin_bit_cast(uint4v, __builtin_amdgcn_raw_buffer_load_b128(
                buffer(t.w, k < K ? t.w_bytes : 0), t.w_at, kFp4 ? at / 2 : 2 * at, 0));
        } else {
            const bool in = k + 32 * g < K;
            r.w[s] = __builtin_bit_cast(uint4v, __builtin_amdgcn_raw_buffer_load_b128(
                buffer(t.w, t.w_bytes), in ? t.w_at : kOutside, at / 2, 0));
            r.sc[kFp4 && !kWide ? s : 0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(
                buffer(t.sc, t.sc_bytes), in ? t.sc_at : kOutside, at / 16, 0);
        }
    }
}

// What lane 4 n + g loaded, in lane 16 g + n. The asm keeps the compiler from
// moving the exchange in front of later loads, where it would wait for them.
__device__ __forceinline__ uint32_t handed(uint32_t v, int from)
{
    asm volatile("" : "+v"(v));
    return (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v);
}

__device__ __forceinline__ uint4v handed(uint4v v, int from)
{
    for (int i = 0; i < 4; ++i)
        v[i] = handed(v[i], from);
    return v;
}

// The two scale bytes of each step for this lane (in the low half of sc[s]).
template <bool kFp4, bool kDown, int NT, bool kWide>
__device__ __forceinline__ void deal_scales(const Weights<kFp4, kDown, NT, kWide>& r, uint32_t* sc, int g, int from)
{
    if (!kWide) {
        for (int s = 0; s < Shape<kFp4, kDown, NT>::S; ++s) {
            uint16_t pair = r.sc[kFp4 && !kWide ? s : 0];
            asm volatile("" : "+v"(pair));
            sc[s] = handed((uint32_t)pair, from);
        }
        return;
    }
    const uint32_t x = handed(r.wide[0], from), y = handed(r.wide[1], from);
    // group s holds step s's pairs (0, 1) in x, (2, 3) in y. Upper half of x
    // against lower half of y: groups 0, 1 then have the pairs (0, 1) of
    // steps 0, 1 in x and of 2, 3 in y, groups 2, 3 the pairs (2, 3). Then
    // each row pair gets both rows of either.
    const auto h = __builtin_amdgcn_permlane32_swap(x, y, false, false);
    const auto a = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
    sc[0] = a[0] >> (16 * (g & 1));
    sc[1] = a[1] >> (16 * (g & 1));
    if (Shape<kFp4, kDown, NT>::S > 2) {
        const auto b = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
        sc[Shape<kFp4, kDown, NT>::S > 2 ? 2 : 0] = b[0] >> (16 * (g & 1));
        sc[Shape<kFp4, kDown, NT>::S > 2 ? 3 : 0] = b[1] >> (16 * (g & 1));
    }
}

// The tokens' side of a chunk: kLanes lanes a token, 8 elements each; a wave
// takes every fourth group of kAtOnce tokens. Columns behind the last token
// are left as they are: they only reach columns of the result that nothing
// reads.
template <bool kFp4, bool kDown, int NT>
struct Tokens {
    static constexpr int kLanes = Shape<kFp4, kDown, NT>::KC / 8;
    static constexpr int kAtOnce = 64 / kLanes;
    static constexpr int R = 4 * NT / kAtOnce;              // turns of a wave
    static constexpr int kWords = kDown ? 8 : 4;            // FP32 h or BF16 x
    uint32_t v[R][kWords];
};

// `at`: byte offsets of this lane's part of its tokens, kOutside for none.
template <bool kFp4, bool kDown, int NT>
__device__ __forceinline__ void load_tokens(Tokens<kFp4, kDown, NT>& r, __amdgpu_buffer_rsrc_t src,
                                            const uint32_t* at, int k0, int K, int lane)
{
    using X = Tokens<kFp4, kDown, NT>;
    const bool in = k0 + 8 * (lane % X::kLanes) < K;
    const int step = k0 < K ? k0 * (kDown ? 4 : 2) : 0;
    for (int i = 0; i < X::R; ++i)
        for (int w = 0; w < X::kWords / 4; ++w) {
            const uint4v u = __builtin_bit_cast(uint4v, __builtin_amdgcn_raw_buffer_load_b128(
                src, (in ? at[i] : kOutside) + 16 * w, step, 0));
            for (int j = 0; j < 4; ++j)
                r.v[i][4 * w + j] = u[j];
        }
}

// Largest over the lanes that share a token, in all of them: within rows of 16
// lanes by row permutations, across them by row swaps; nothing goes through
// LDS.
template <int kLanes>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xb1, 0xf, 0xf, true));     // lane ^ 1
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4e, 0xf, 0xf, true));     // lane ^ 2
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true));    // 8 mirrored
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true));    // 16 mirrored
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(a[0], a[1]);
    if (kLanes == 64) {
        const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = max(b[0], b[1]);
    }
    return v;
}

// FP32 values of a run of 8.
template <bool kDown>
__device__ __forceinline__ void values(const uint32_t* v, float* f)
{
    for (int j = 0; j < 8; ++j)
        f[j] = kDown ? __uint_as_float(v[kDown ? j : 0])
                     : __uint_as_float(j & 1 ? v[j >> 1] & 0xffff0000u : v[j >> 1] << 16);
}

template <bool kFp4, bool kDown, int NT, bool kWide>
__global__ __launch_bounds__(kThreads) void moe_product_kernel(Moe a)
{
    using X = Shape<kFp4, kDown, NT>;
    constexpr bool kSplit = !kFp4 && kDown;      // h as a sum of two BF16 numbers
    __shared__ Group s;
    __shared__ __attribute__((aligned(16))) uint16_t tok_lds[2][kSplit ? 2 : 1][16 * NT][X::kPitch];
    __shared__ float scale_lds[2][16 * NT];      // 2^-e of a token's chunk

    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, n = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int from = 4 * (4 * n + g);
    const int slot = blockIdx.y;
    // (a pair without an expert, id -1, finds no token below and leaves)
    const int e = !a.by_pair ? slot : kDown ? a.ids[slot] : expert_of_pair(a, s, slot, tid);
    const int expert = max(e, 0);
    const int rows = kDown ? a.hidden : 2 * a.inter, K = kDown ? a.inter : a.hidden;
    const int row0 = blockIdx.x * 64 + 16 * wave;
    const bool mine = row0 < rows;
    const int64_t row = (int64_t)expert * rows + (mine ? row0 : 0);
    const int pitch = kFp4 ? K / 2 : 2 * K;
    const Tile tile = {(const uint8_t*)(kDown ? a.w2 : a.w1) + row * pitch,
                       kFp4 ? (kDown ? a.s2 : a.s1) + row * (K / 16) : nullptr, 16u * pitch, (uint32_t)K,
                       (uint32_t)((lane >> 2) * pitch + 16 * (lane & 3)),
                       (uint32_t)((lane >> 2) * (K / 16) + (kWide ? 8 * (lane & 3 & (X::S - 1)) : 2 * (lane & 3)))};
    // x or h: at most 2^31 bytes, checked on the host
    const __amdgpu_buffer_rsrc_t src =
        kDown ? buffer(a.h, (uint32_t)(a.tokens * a.top_k) * K * 4)
              : buffer(a.x, (uint32_t)((a.tokens - 1) * a.ld_x + K) * 2);

    using Tok = Tokens<kFp4, kDown, NT>;
    const float gs = !kFp4 ? 1.0f : kDown ? (a.gs2 ? a.gs2[expert] : 1.0f) : (a.gs1 ? a.gs1[expert] : 1.0f);

    // the first weights are requested before the tokens are known
    Weights<kFp4, kDown, NT, kWide> even, odd;
    load_weights<kFp4, kDown, NT, kWide>(even, tile, 0, K, lane & 3);
    if (kDown)
        routed(a, s, e, tid);
    else
        route(a, s, slot, e, blockIdx.x == 0, tid);
    // no token is here, or an earlier token's workgroup has this expert
    if (s.count == 0 || (a.by_pair && s.pairs[0] != slot))
        return;

    // Tokens beyond 16 NT take another pass over the weights.
    for (int col0 = 0; col0 < s.count; col0 += 16 * NT) {
        const int* pairs = s.pairs + col0;
        const int count = min(s.count - col0, 16 * NT), tiles = (count + 15) >> 4;
        float4v acc[NT];
        for (int nt = 0; nt < NT; ++nt)
            acc[nt] = float4v{0, 0, 0, 0};

        Tok tokens;
        uint32_t at[Tok::R];
        for (int i = 0; i < Tok::R; ++i) {
            const int col = (wave + 4 * i) * Tok::kAtOnce + lane / Tok::kLanes;
            at[i] = kOutside;
            if (col < count)
                at[i] = (kDown ? pairs[col] * K * 4 : (uint32_t)(pairs[col] / a.top_k * a.ld_x * 2)) +
                        (lane % Tok::kLanes) * (kDown ? 32 : 16);
        }
        auto stage = [&](int buf) {
#pragma unroll
            for (int i = 0; i < Tok::R; ++i) {
                const int first = (wave + 4 * i) * Tok::kAtOnce;
                if (first >= count)
                    continue;
                const int col = first + lane / Tok::kLanes, at = 8 * (lane % Tok::kLanes);
                uint4v* dst = (uint4v*)&tok_lds[buf][0][col][at];
                if (!kFp4 && !kDown) {
                    const uint32_t* v = tokens.v[i];
                    *dst = uint4v{v[0], v[1], v[2], v[3]};
                    continue;
                }
                float f[8];
                values<kDown>(tokens.v[i], f);
                if (kFp4) {
                    uint32_t top = 0;
                    for (int j = 0; j < 8; ++j)
                        top = max(top, __float_as_uint(f[j]) & 0x7fffffffu);
                    top = lanes_max<Tok::kLanes>(top);
                    const int ex = fp16_exponent(top);
                    const float up = ldexpf(1.0f, ex);
                    if (at == 0)
                        scale_lds[buf][col] = ldexpf(1.0f, -ex);
                    half8v h;
                    for (int j = 0; j < 8; ++j)
                        h[j] = (_Float16)(f[j] * up);
                    *dst = __builtin_bit_cast(uint4v, h);
                } else {
                    bf8v hi, lo;
                    for (int j = 0; j < 8; ++j) {
                        hi[j] = (__bf16)f[j];
                        lo[j] = (__bf16)(f[j] - (float)hi[j]);
                    }
                    *dst = __builtin_bit_cast(uint4v, hi);
                    *(uint4v*)&tok_lds[buf][kSplit ? 1 : 0][col][at] = __builtin_bit_cast(uint4v, lo);
                }
            }
        };
        auto request = [&](Weights<kFp4, kDown, NT, kWide>& next, int k0) {
            // The tokens first, as they are wanted first; and no use of
            // other weights moves in front of these loads, where it would
            // wait for all of them.
            load_tokens<kFp4, kDown, NT>(tokens, src, at, k0, K, lane);
            __builtin_amdgcn_sched_barrier(0);
            load_weights<kFp4, kDown, NT, kWide>(next, tile, k0, K, lane & 3);
            __builtin_amdgcn_sched_barrier(0);
        };
        auto compute = [&](const Weights<kFp4, kDown, NT, kWide>& now, int buf) {
            float4v c[NT];
            for (int nt = 0; nt < NT; ++nt)
                c[nt] = kFp4 ? float4v{0, 0, 0, 0} : acc[nt];
            uint32_t pair[X::S];
            if (kFp4)
                deal_scales<kFp4, kDown, NT, kWide>(now, pair, g, from);
            for (int st = 0; st < X::S; ++st) {
                if (kFp4) {
                    const half2v sv = e4m3x2(pair[st]);
                    const uint4v w = handed(now.w[st], from);
                    for (int i = 0; i < 4; ++i) {
                        const half8v wf = fp4x8(w[i], sv[i >> 1]);
                        for (int nt = 0; nt < NT; ++nt)
                            if (nt < tiles)
                                c[nt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                                    wf, *(const half8v*)&tok_lds[buf][0][16 * nt + n][128 * st + 32 * g + 8 * i],
                                    c[nt], 0, 0, 0);
                    }
                } else {
                    const bf8v wf = __builtin_bit_cast(bf8v, handed(now.w[st], from));
                    for (int nt = 0; nt < NT; ++nt)
                        if (nt < tiles) {
                            c[nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                wf, *(const bf8v*)&tok_lds[buf][0][16 * nt + n][32 * st + 8 * g], c[nt], 0, 0, 0);
                            if (kSplit)
                                c[nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                    wf, *(const bf8v*)&tok_lds[buf][kSplit ? 1 : 0][16 * nt + n][32 * st + 8 * g],
                                    c[nt], 0, 0, 0);
                        }
                }
            }
            for (int nt = 0; nt < NT; ++nt)
                acc[nt] = kFp4 ? acc[nt] + c[nt] * scale_lds[buf][16 * nt + n] : c[nt];
        };

        // A chunk is staged in one LDS buffer while the other is in use, so
        // one barrier a chunk suffices; its weights go out two chunks ahead,
        // into the registers that the chunk in front has just left.
        load_tokens<kFp4, kDown, NT>(tokens, src, at, 0, K, lane);
        if (col0 > 0)
            load_weights<kFp4, kDown, NT, kWide>(even, tile, 0, K, lane & 3);
        stage(0);
        request(odd, X::KC);
        for (int k0 = 0; k0 < K; k0 += 2 * X::KC) {
            __syncthreads();
            compute(even, 0);
            stage(1);
            request(even, k0 + 2 * X::KC);
            __syncthreads();
            compute(odd, 1);                // zeros behind the end of the axis
            stage(0);
            request(odd, k0 + 3 * X::KC);
        }

        for (int nt = 0; nt < NT; ++nt) {
            const int col = 16 * nt + n;
            const float4v v = acc[nt] * gs;
            if (kDown) {
                if (mine && col < count)
                    *(float4v*)(a.y + (int64_t)pairs[col] * rows + row0 + 4 * g) = v;
            } else {
                // rows 0..7 of the tile (g = 0, 1) are gates, 8..15 their ups
                float4v h;
                for (int r = 0; r < 4; ++r) {
                    const float up = __shfl_xor(v[r], 32);
                    h[r] = v[r] / (1.0f + expf(-v[r])) * up;
                }
                if (mine && g < 2 && col < count)
                    *(float4v*)(a.h + (int64_t)pairs[col] * a.inter + row0 / 2 + 4 * g) = h;
            }
        }
    }
}

// out[t] = sum_k w[t][k] y[t][k], in the order of k, for a token and 1024
// columns; the first workgroup of a token also writes its weights.
__global__ __launch_bounds__(kThreads) void moe_sum_kernel(Moe a)
{
    __shared__ float w[kMaxTopK], wave_sum[kThreads / 64];
    __shared__ int id[kMaxTopK];
    const int t = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
    const int n = (blockIdx.x * kThreads + tid) * 4;
    const float* y = a.y + (int64_t)t * a.top_k * a.hidden + min(n, a.hidden - 4);
    float4v v[8];       // a row that no expert wrote is loaded, not added
    for (int k = 0; k < 8; ++k)
        v[k] = *(const float4v*)(y + (int64_t)min(k, a.top_k - 1) * a.hidden);

    // The first choice has the largest logit. An infinite one would make
    // inf - inf: equal logits are compared, not subtracted.
    const int mine = lane < a.top_k ? a.ids[t * a.top_k + lane] : -1;
    const float l = mine >= 0 ? logit(a, t, mine) : -INFINITY;
    const float top = __shfl(l, 0);
    const float p = mine < 0 ? 0.0f : l == top ? 1.0f : expf(l - top);
    float sum = 0;
    if (a.renormalize) {
        sum = p;
    } else {
        for (int f = tid; f < a.experts; f += kThreads) {
            const float u = logit(a, t, f);
            sum += u == -INFINITY ? 0.0f : u == top ? 1.0f : expf(u - top);
        }
    }
    for (int d = 32; d; d >>= 1)
        sum += __shfl_xor(sum, d);
    if (lane == 0)
        wave_sum[tid >> 6] = sum;
    __syncthreads();
    if (!a.renormalize)
        sum = wave_sum[0] + wave_sum[1] + wave_sum[2] + wave_sum[3];
    if (tid < a.top_k) {
        w[tid] = mine < 0 ? 0.0f : p / sum;
        id[tid] = mine;
        if (blockIdx.x == 0)
            a.weights[t * a.top_k + tid] = w[tid];
    }
    __syncthreads();
    if (n >= a.hidden)
        return;
    float4v o = {0, 0, 0, 0};
    for (int k = 0; k < 8; ++k)
        if (k < a.top_k && id[k] >= 0)
            o += w[k] * v[k];
    for (int k = 8; k < a.top_k; ++k)
        if (id[k] >= 0)
            o += w[k] * *(const float4v*)(y + (int64_t)k * a.hidden);
    *(uint2v*)(a.out + t * a.ld_out + n) = uint2v{bf16x2(o[0], o[1]), bf16x2(o[2], o[3])};
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

template <bool kFp4, bool kDown, int NT>
void launch_product(const Moe& a, hipStream_t stream)
{
    const int rows = kDown ? a.hidden : 2 * a.inter, K = kDown ? a.inter : a.hidden;
    const dim3 grid(serving::ceil_div(rows, 64), a.by_pair ? a.tokens * a.top_k : a.experts);
    if (kFp4 && K % 128 == 0 && serving::aligned(kDown ? a.s2 : a.s1, 8))
        hipLaunchKernelGGL((moe_product_kernel<kFp4, kDown, NT, kFp4>), grid, dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((moe_product_kernel<kFp4, kDown, NT, false>), grid, dim3(kThreads), 0, stream, a);
}

template <bool kFp4, int NT>
void launch_both(const Moe& a, hipStream_t stream)
{
    launch_product<kFp4, false, NT>(a, stream);
    launch_product<kFp4, true, NT>(a, stream);
    hipLaunchKernelGGL(moe_sum_kernel, dim3(serving::ceil_div(a.hidden, 4 * kThreads), a.tokens),
                       dim3(kThreads), 0, stream, a);
}

template <bool kFp4>
void launch_products(const Moe& a, int nt, hipStream_t stream)
{
    if (nt == 1)
        launch_both<kFp4, 1>(a, stream);
    else if (nt == 2)
        launch_both<kFp4, 2>(a, stream);
    else
        launch_both<kFp4, 4>(a, stream);
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
    // rows are addressed with 31-bit offsets from the first one
    const int64_t most = INT32_MAX - 4096;
    if (tokens * a.top_k * inter * 4 > most || (tokens - 1) * a.ld_x + hidden > most / 2)
        return NVFP4_ERROR_UNSUPPORTED_SHAPE;
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
    a.y = a.h + tokens * a.top_k * inter;
    // the reached experts are few: one workgroup column per pair, where pairs
    // with an expert that an earlier token has leave at once; else per expert
    a.by_pair = tokens * a.top_k <= a.experts;
    // columns of 16 tokens for twice an expert's share: more take another pass, which
    // reads the weights again (4096 x 1024, 64 tokens on one of 64 experts: four
    // passes, 91 us, against 79 for the one pass of a layer with one expert)
    const int64_t share = a.experts == 1 ? tokens : 2 * tokens * a.top_k / a.experts;
    const int64_t cols = share < tokens ? share : tokens;
    const int nt = cols <= 16 ? 1 : cols <= 32 ? 2 : 4;
    launch_products<kFp4>(a, nt, stream);
    return launched();
}

}  // namespace

extern "C" int64_t moe_layer_workspace(int64_t tokens, int64_t hidden, int64_t inter,
                                       int32_t num_experts, int32_t top_k)
{
    if (check_sizes(tokens, hidden, inter, num_experts, top_k) != NVFP4_SUCCESS)
        return -1;
    return tokens * top_k * (inter + hidden) * 4;
}

extern "C" nvfp4_status_t moe_layer_nvfp4(
    const uint16_t* x, int64_t tokens, int64_t ld_x, const float* logits, const uint8_t* w1_packed,
    const uint8_t* w1_scales, const float* gs1, const uint8_t* w2_packed, const uint8_t* w2_scales,
    const float* gs2, int64_t hidden, int64_t inter, int32_t num_experts, int32_t top_k,
    int32_t renormalize, uint16_t* out, int64_t ld_out, int32_t* topk_ids, float* topk_weights,
    void* workspace, int64_t workspace_bytes, hipStream_t stream)
{
    Moe a = {x, logits, w1_packed, w2_packed, w1_scales, w2_scales, gs1, gs2, out, topk_ids,
             topk_weights, nullptr, nullptr, ld_x, ld_out, 0, 0, 0, num_experts, top_k, renormalize};
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
             nullptr, nullptr, ld_x, ld_out, 0, 0, 0, num_experts, top_k, renormalize};
    return run<false>(a, hidden, inter, workspace_bytes, tokens, workspace, stream);
}
