// Attention over listed pages of the paged NVFP4 cache (include/nvfp4_sparse.h).
//
// A workgroup takes some tokens that follow each other and a key/value head; its
// query rows are the heads that share the key/value head, of all its tokens. It
// first looks the tokens' lists up and joins them into one list of pages, with a
// bit for each token that has listed the page. The pages, one behind the other,
// are a range of tokens that its waves walk in tiles of 32 as the rows kernel of
// paged_attention.hip does with a request's tokens (attention_rows.hpp); what a
// row sees of a tile is a word of bits made from the page's bits and the row's
// position. A page that several tokens list is loaded and converted once.
//
// Single tokens are bound by scattered loads: a head's 64 bytes of codes a token (of
// 128 dimensions) are half of a line, so twice the bytes come from memory (64 requests,
// 64 pages of 32, 64/8 heads: 58 us for 153 MB, loads alone 53, arithmetic alone 34).
// Chunks are bound by vector arithmetic, 306 instructions for a tile of 32 tokens and 16
// rows (1000 tokens, 32 pages of 64, 32/8 heads of 128: 226 us, loads alone 152, arithmetic
// alone 216): hence 16 rows of tokens together, no more, as their joined lists grow
// (2, 4, 8 tokens of 32 pages: 47, 65, 86 pages).
#include "attention_rows.hpp"
#include "sparse_common.hpp"
#include "nvfp4_sparse.h"

namespace {

constexpr int kMostListed = 2048, kWaves = 4, kThreads = 64 * kWaves;

struct Sparse {
    Attn a;
    const int32_t* pages;
    int list_len;
    int together;      // tokens that a workgroup takes
};

// The listed pages that some token sees: the page in the cache, the position of its
// first token in the request, and a bit for each token that listed it. While the
// list is made: `first` is the page's number in the request, -1 for an entry that
// shows nothing.
struct Listed {
    int page[kMostListed], first[kMostListed];
    uint16_t by[kMostListed];
};

template <int D>
struct Joined {
    float o[kWaves][16][D + 4];
    float m[kWaves][16], l[kWaves][16];
};

template <int D>
union Shared {
    Joined<D> joined;
    Listed list;
};

// A part of a row's listed tokens: all parts hold some.
__device__ __forceinline__ void write_split(const Attn& a, int D, int split, int64_t row, float m, float l)
{
    write_part(a, D, split, row, m, l);
    if (split == 0)
        used_splits(a, D)[row] = a.splits;
}

struct Counts {
    int n[kWaves];
    int repeated;
};

// Looks up the lists of the tokens t, ..., t + run - 1 of request b, the first of them
// at position pos0, and joins them. Returns the number of pages; `run` becomes 1
// where a token has listed a page twice, which then counts twice.
__device__ __forceinline__ int make_list(const Sparse& s, Listed& list, Counts& counts, int b, int t, int h, int pos0,
                                         int& run)
{
    const Attn& a = s.a;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int pitch = (s.list_len + 3) & ~3;
    int entries = run * pitch;
    // entry e of the lists: the page in the cache, and in the request or -1
    auto look_up = [&](int e, int& page) {
        const int token = run == 1 ? 0 : e / pitch, i = e - token * pitch;
        const int p = i < s.list_len ? s.pages[((int64_t)(t + token) * a.kv_heads + h) * s.list_len + i] : -1;
        page = -1;
        if (p >= 0 && p < a.max_pages && (int64_t)p * a.page <= pos0 + token)
            page = a.table[b * a.ld_table + p];
        return page >= 0 && page < a.num_pages ? p : -1;
    };
    const bool alone = run == 1;
    if (!alone) {
        if (tid == 0)
            counts.repeated = 0;
        for (int e = tid; e < entries; e += kThreads) {
            int page;
            const int p = look_up(e, page);
            list.page[e] = page;
            list.first[e] = p;
            list.by[e] = p >= 0 ? 1 : 0;
        }
        __syncthreads();
        // an entry stands for its page if no token before has listed it
        for (int e = tid; e < entries; e += kThreads) {
            const int p = list.first[e], token = e / pitch;
            if (p < 0)
                continue;
            int by = 0, own = 0;
            for (int other = 0; other < run; ++other) {
                int found = 0;
                for (int i = 0; i < pitch; i += 4) {
                    const int4 v = *(const int4*)&list.first[other * pitch + i];
                    found += (v.x == p) + (v.y == p) + (v.z == p) + (v.w == p);
                }
                by |= found ? 1 << other : 0;
                own = other == token ? found : own;
            }
            if (own > 1)
                counts.repeated = 1;
            list.by[e] = (uint16_t)(by & ((1 << token) - 1) ? 0 : by);
        }
        __syncthreads();
        if (counts.repeated) {
            run = 1;
            entries = pitch;
            for (int e = tid; e < entries; e += kThreads)
                list.by[e] = list.first[e] >= 0 ? 1 : 0;
            __syncthreads();
        }
    }
    // the entries that stand for a page, moved to the front
    int total = 0;
    for (int base = 0; base < entries; base += kThreads) {
        const int e = base + tid;
        int by = 0, page = 0, p = 0;
        if (e < entries) {
            if (alone) {
                p = look_up(e, page);
                by = p >= 0;
            } else {
                by = list.by[e];
                page = list.page[e];
                p = list.first[e];
            }
        }
        const uint64_t in = __ballot(by != 0);
        if (lane == 0)
            counts.n[wave] = __popcll(in);
        __syncthreads();
        int at = total + __popcll(in & ((1ull << lane) - 1));
        for (int w = 0; w < kWaves; ++w) {
            at += w < wave ? counts.n[w] : 0;
            total += counts.n[w];
        }
        if (by) {
            list.page[at] = page;
            list.first[at] = p * a.page;
            list.by[at] = (uint16_t)by;
        }
        __syncthreads();
    }
    return total;
}

// A value's scale that is NaN would reach the rows that do not see its token, as 0
// times NaN is NaN: it is taken out of the tile, and the rows that see the token get it.
template <int D, int RT>
__device__ __forceinline__ void part_nans(Tile<D>& t, const uint32_t (&sees)[RT], int lane,
                                          float4v (&o)[RT][Tile<D>::C][Tile<D>::VM])
{
    const int g = lane >> 4;
#pragma unroll
    for (int c = 0; c < Tile<D>::C; ++c) {
        const uint32_t nan = t.shown ? ((t.vs[c] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u : 0;
        if (__any(nan != 0)) {
            // byte b of a lane: 16 dimensions, those of the lanes g = b, or for 128 dimensions
            // those 2 (b % 2) + (0, 1) of g = b / 2 and, of the second half wave, g = 2 + b / 2
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const uint64_t tokens = __ballot(nan >> (8 * b + 7) & 1);
                const uint32_t mine = D > 64 && g >= 2 ? (uint32_t)(tokens >> 32) : (uint32_t)tokens;
                const bool own = D > 64 ? (g & 1) == b >> 1 : g == b;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int i = 0; i < Tile<D>::VM; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (D == 64 || r >> 1 == (b & 1))
                                o[rt][c][i][r] = own && (mine & sees[rt]) ? NAN : o[rt][c][i][r];
            }
            t.vs[c] &= ~((nan >> 7) * 255u);
        }
    }
}

// Workgroups a compute unit, as many as the registers of the rows hold.
template <int D, int RT, bool kPaged16>
constexpr int kResident = RT == 1 && D <= 128 && kPaged16 ? 3 : D * RT <= 256 ? 2 : 1;

template <int D, int RT, bool kPaged16>
__global__ __launch_bounds__(kThreads, (kResident<D, RT, kPaged16>)) void sparse_rows_kernel(Sparse s)
{
    using T = Tile<D>;
    constexpr int C = T::C, KF = D / 32, VM = T::VM, kStep = 32 * kWaves;
    __shared__ Shared<D> lds;
    __shared__ Counts counts;
    const Attn& a = s.a;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, n = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = a.heads / a.kv_heads;
    const float k_scale = a.scale * (a.k_gs ? a.k_gs[0] : 1.0f) * kLog2e;

    // Workgroups go to the 8 XCDs in turn. Tokens of many requests: all key/value
    // heads of a token go to one XCD one after the other, as in the rows kernel.
    // Tokens that share pages: an XCD takes a run of the tokens for one head after
    // the other, so that its L2 holds little but what they share.
    const uint32_t groups = (uint32_t)(a.tokens + s.together - 1) / s.together;
    const uint32_t per_split = groups * a.row_blocks, works = per_split * a.splits;
    const uint32_t xcd = blockIdx.x & 7, j = blockIdx.x >> 3;
    uint32_t work, h;
    if (s.together > 1) {
        const uint32_t run = (works * a.kv_heads + 7) / 8, at = xcd * run + j;
        h = at / works;
        work = at % works;
        if (j >= run || h >= (uint32_t)a.kv_heads)
            return;
    } else {
        work = j / a.kv_heads * 8 + xcd;
        h = j % a.kv_heads;
        if (work >= works)
            return;
    }
    const int split = (int)(work / per_split);
    const uint32_t item = work % per_split;
    const int row0 = (int)(item % a.row_blocks) * 16 * RT;
    int token = (int)(item / a.row_blocks) * s.together;
    const int token_end = min(token + s.together, a.tokens);
    // the tokens of one request at a time
    for (int run = 1; token < token_end; token += run) {
        run = 1;
        const int b = sparse::request_of(a.offsets, a.num_seqs, token);
        if (b < 0) {
            // the join leaves a token of no request alone
            if (a.splits > 1 && split == 0 && tid < 16 * RT && row0 + tid < group)
                used_splits(a, D)[(int64_t)token * a.heads + h * group + row0 + tid] = 0;
            continue;
        }
        const int behind = a.offsets[b + 1];
        run = min(token_end, behind) - token;
        const int len = a.num_pages > 0 ? min(max(a.lens[b], 0), a.max_pages * a.page) : 0;
        const int pos0 = min(len - behind + token, len - 1);
        __syncthreads();                        // the LDS of what came before is read
        const int range = make_list(s, lds.list, counts, b, token, h, pos0, run) * a.page;
        // the splits take equal parts of what there is
        const int chunk = a.splits == 1 ? range : ((range + a.splits - 1) / a.splits + 127) & ~127;
        const int first = split * chunk, last = __builtin_amdgcn_readfirstlane(min(first + chunk, range));

        auto entries = [&](int t0) {
            Entries r;
            for (int hh = 0; hh < 2; ++hh) {
                const int at = t0 + 16 * hh;
                const bool in = kPaged16 && at < last;
                r.e[hh] = in ? __builtin_amdgcn_readfirstlane(lds.list.page[page_of(a, at)]) : -1;
            }
            return r;
        };
        auto request = [&](Tile<D>& t, Entries e, int t0) {
            if (!kPaged16 && t0 >= last)
                return;
            load_tile<D, kPaged16>(t, a, lds.list.page, e, h, t0, first, last, lane);
            __builtin_amdgcn_sched_barrier(0);      // no use of the other tile moves up here
        };
        int t0 = first + 32 * wave;
        Entries e0 = entries(t0), e1 = entries(t0 + kStep);

        uint4v w[RT][KF];
        int bit[RT], pos[RT];
        for (int rt = 0; rt < RT; ++rt) {
            const int r = row0 + 16 * rt + n, rr = min(r, run * group - 1);
            const int of = run == 1 ? 0 : rr / group;
            bit[rt] = r < run * group ? of : 31;
            pos[rt] = pos0 + of;
            const uint16_t* src = a.q + (token + of) * a.ld_q + (h * group + rr - of * group) * D;
            for (int f = 0; f < KF; ++f)
                w[rt][f] = *(const uint4v*)(src + (D > 64 ? 128 * (f / 4) + 32 * g + 8 * (f % 4) : 16 * g + 8 * f));
        }
        __builtin_amdgcn_sched_barrier(0);
        Tile<D> even, odd;
        request(even, e0, t0);

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
        const int everyone = (1 << run) - 1;
        auto compute = [&](Tile<D>& t, int t0) {
            bool all = true;
            uint32_t sees_of[RT];
            if (kPaged16) {
                int place[2], by[2];
                for (int hh = 0; hh < 2; ++hh) {
                    const int at = min(t0 + 16 * hh, last - 16), i = (int)page_of(a, at);
                    place[hh] = __builtin_amdgcn_readfirstlane(lds.list.first[i]) + (at - i * a.page);
                    by[hh] = __builtin_amdgcn_readfirstlane(lds.list.by[i]);
                    all = all && by[hh] == everyone && place[hh] + 15 <= pos0;
                }
                // what lies behind the request's tokens may be anything
                t.shown = t.shown && ((lane & 16) ? place[1] : place[0]) + n < len;
                for (int rt = 0; rt < RT; ++rt)
                    sees_of[rt] = ~0u;
                if (!all)
                    for (int rt = 0; rt < RT; ++rt) {
                        sees_of[rt] = 0;
                        for (int hh = 0; hh < 2; ++hh)
                            sees_of[rt] |= by[hh] >> bit[rt] & 1 ? bits_between(0, min(pos[rt] - place[hh] + 1, 16)) << 16 * hh : 0;
                    }
            } else {
                const int at = t0 + (lane & 31), i = (int)page_of(a, min(at, last - 1));
                const int place = lds.list.first[i] + (at - i * a.page);
                const int by = at < last ? lds.list.by[i] : 0;
                t.shown = t.shown && place < len;
                for (int rt = 0; rt < RT; ++rt)
                    sees_of[rt] = 0;
                for (int k = 0; k < run; ++k) {
                    const uint32_t shows = (uint32_t)__ballot((by >> k & 1) && place <= pos0 + k);
                    all = all && shows == ~0u;
                    for (int rt = 0; rt < RT; ++rt)
                        sees_of[rt] = bit[rt] == k ? shows : sees_of[rt];
                }
            }
            if (!all)
                part_nans<D, RT>(t, sees_of, lane, o);
#define WHOLE all
#define SEEN(rt) sees_of[rt]
#include "attend_tile.inc"
        };
        // A wave with one tile asks for no more, as tiles that are not there take time too: 32
        // pages of 64 for one token, 16 splits, 11.8 us instead of 12.7 (with the join).
        if (t0 + kStep >= last) {
            if (t0 < last)
                compute(even, t0);
        } else {
            request(odd, e1, t0 + kStep);
            e0 = entries(t0 + 2 * kStep);
            e1 = entries(t0 + 3 * kStep);
            for (; t0 < last; t0 += 2 * kStep) {
                compute(even, t0);
                request(even, e0, t0 + 2 * kStep);
                e0 = entries(t0 + 4 * kStep);
                if (t0 + kStep < last)
                    compute(odd, t0 + kStep);
                request(odd, e1, t0 + 3 * kStep);
                e1 = entries(t0 + 5 * kStep);
            }
        }
        __syncthreads();                        // the list is read, its LDS goes to the join
        const int first_row = token;
        auto& o_lds = lds.joined.o;
        auto& m_lds = lds.joined.m;
        auto& l_lds = lds.joined.l;
#define ROWS run * group
#define FIRST first_row
#define WRITE_SPLIT(row, m, l) write_split(a, D, split, row, m, l)
#include "join_waves.inc"
    }
}

// How the work is cut: tokens that a workgroup takes together, its query rows, and
// splits of the listed tokens where there are too few workgroups for the card.
struct SparsePlan {
    int together, block, row_blocks, splits;
};

SparsePlan sparse_plan(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t head_dim, int32_t page_size,
                       int64_t num_seqs, int64_t list_len)
{
    using serving::ceil_div;
    SparsePlan p;
    const int group = heads / kv_heads;
    const int64_t pitch = ceil_div(list_len, (int64_t)4) * 4;
    // by the batch's average: 512 tokens of one request beside 255 single ones take 370 us,
    // the two apart 318
    const int64_t average = tokens / (num_seqs < 1 ? 1 : num_seqs);
    p.together = 1;
    while (p.together < average && (p.together + 1) * group <= 16 && (p.together + 1) * pitch <= 1024 &&
           (p.together + 1) * list_len * page_size <= (1 << 30))
        ++p.together;
    const int rows = p.together * group;
    const int64_t range = list_len * page_size, units = ceil_div(tokens, (int64_t)p.together) * kv_heads;
    // More rows share a tile's conversion, but take the registers of other waves: 512
    // tokens of 64 heads on one of 128, 64 pages of 32: 112 us in blocks of 16, 83 of 32,
    // 144 of 64; 48 such tokens 28, 27 and 62 us. Of 64 dimensions 512 tokens take 87, 67 and
    // 51 us, 48 of them 23, 21 and 27.
    const int most = head_dim > 128 ? 16 : head_dim > 64 || units < 512 ? 32 : 64;
    p.block = rows <= 16 || most == 16 ? 16 : rows <= 32 || most == 32 ? 32 : 64;
    p.row_blocks = ceil_div(rows, p.block);
    const int64_t items = units * p.row_blocks;
    // two workgroups a compute unit in all (three or four: up to 1.2 or 1.6 times the time
    // where the join is then needed; 64 requests of 8 heads 64 us instead of 58)
    int64_t splits = items < 1 ? 1 : 512 / items;
    if (splits > ceil_div(range, (int64_t)128))
        splits = ceil_div(range, (int64_t)128);
    if (splits > 256)
        splits = 256;
    if (splits < 1 || tokens * heads > (1 << 22))
        splits = 1;
    p.splits = (int)splits;
    return p;
}

// Pages of whole 16 tokens are read a half tile at a time, scales also where there is
// nothing to see; so there must be a page.
template <int D, int RT>
void launch_rows(const Sparse& s, dim3 grid, hipStream_t stream)
{
    if (s.a.page % 16 == 0 && s.a.num_pages > 0)
        hipLaunchKernelGGL((sparse_rows_kernel<D, RT, true>), grid, dim3(kThreads), 0, stream, s);
    else
        hipLaunchKernelGGL((sparse_rows_kernel<D, RT, false>), grid, dim3(kThreads), 0, stream, s);
}

template <int D>
void launch(const Sparse& s, int block, hipStream_t stream)
{
    const Attn& a = s.a;
    const int64_t groups = (a.tokens + (int64_t)s.together - 1) / s.together;
    const int64_t units = (groups * a.row_blocks * a.splits + 7) / 8 * 8 * a.kv_heads;
    const dim3 grid((unsigned)units);
    if (block == 16) {
        launch_rows<D, 1>(s, grid, stream);
    } else if constexpr (D <= 128) {
        if (block == 32) {
            launch_rows<D, 2>(s, grid, stream);
        } else if constexpr (D == 64) {
            launch_rows<D, 4>(s, grid, stream);
        }
    }
    if (a.splits > 16)
        hipLaunchKernelGGL((attn_join_kernel<D, 4, true>), dim3((unsigned)(a.tokens * a.heads)), dim3(256), 0, stream, a);
    else if (a.splits > 1)
        hipLaunchKernelGGL((attn_join_kernel<D, 1, true>), dim3((unsigned)(a.tokens * a.heads + 3) / 4), dim3(256), 0, stream, a);
}

bool sizes_ok(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t page_size, int64_t list_len)
{
    return tokens >= 0 && heads >= 1 && kv_heads >= 1 && heads % kv_heads == 0 && page_size >= 1 && list_len >= 0;
}

bool sizes_supported(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t head_dim, int32_t page_size, int64_t num_seqs,
                     int64_t list_len)
{
    return (head_dim == 64 || head_dim == 128 || head_dim == 256) && heads <= 1024 && tokens <= (1 << 23) / heads &&
           num_seqs <= 65535 && num_seqs * kv_heads <= (1 << 22) && list_len <= kMostListed &&
           list_len <= (1 << 30) / page_size;
}

}  // namespace

extern "C" int64_t nvfp4_sparse_attention_workspace(int64_t tokens, int32_t heads, int32_t kv_heads,
                                                    int32_t head_dim, int32_t page_size, int64_t num_seqs,
                                                    int64_t list_len)
{
    if (num_seqs < 0 || !sizes_ok(tokens, heads, kv_heads, page_size, list_len) ||
        !sizes_supported(tokens, heads, kv_heads, head_dim, page_size, num_seqs, list_len))
        return -1;
    const SparsePlan p = sparse_plan(tokens, heads, kv_heads, head_dim, page_size, num_seqs, list_len);
    return p.splits > 1 ? tokens * heads * 4 * ((head_dim + 2) * p.splits + 1) : 0;
}

extern "C" nvfp4_status_t nvfp4_sparse_attention(
    const uint16_t* q, int64_t tokens, int64_t ld_q, int32_t heads, int32_t kv_heads, int32_t head_dim,
    const uint8_t* k_packed, const uint8_t* k_scales, const uint8_t* v_packed, const uint8_t* v_scales,
    int64_t num_slots, int32_t page_size, const int32_t* block_table, int64_t ld_table, int64_t max_pages,
    const int32_t* seq_lens, const int32_t* query_offsets, int64_t num_seqs, const int32_t* pages, int64_t list_len,
    float scale, const float* k_gs, const float* v_gs, uint16_t* out, int64_t ld_out, float* lse, void* workspace,
    int64_t workspace_bytes, hipStream_t stream)
{
    using namespace serving;
    if (!sizes_ok(tokens, heads, kv_heads, page_size, list_len) || num_slots < 0 || num_slots % page_size != 0 ||
        max_pages < 0 || ld_table < max_pages || num_seqs < 0 || !extent_ok(num_seqs, ld_table, 4) || ld_q < 0 ||
        ld_out < 0 || workspace_bytes < 0 || !(scale - scale == 0.0f))
        return NVFP4_ERROR_INVALID_VALUE;
    if (!sizes_supported(tokens, heads, kv_heads, head_dim, page_size, num_seqs, list_len) || num_slots > INT32_MAX ||
        max_pages > (1 << 30) / page_size)
        return NVFP4_ERROR_UNSUPPORTED_SHAPE;
    const int64_t cols = (int64_t)heads * head_dim;
    if (ld_q < cols || ld_out < cols || !extent_ok(tokens, ld_q, 2) || !extent_ok(tokens, ld_out, 2))
        return NVFP4_ERROR_INVALID_VALUE;
    if (tokens == 0 || num_seqs == 0)
        return NVFP4_SUCCESS;
    if (!q || !out || !seq_lens || !query_offsets || (max_pages > 0 && !block_table) || (list_len > 0 && !pages) ||
        (num_slots > 0 && (!k_packed || !k_scales || !v_packed || !v_scales)))
        return NVFP4_ERROR_INVALID_VALUE;
    const uintptr_t sa = head_dim / 16;
    if (!aligned(q, 16) || !aligned(out, 16) || ld_q % 8 != 0 || ld_out % 8 != 0 || !aligned(k_packed, 16) ||
        !aligned(v_packed, 16) || !aligned(k_scales, sa) || !aligned(v_scales, sa) || !aligned(block_table, 4) ||
        !aligned(seq_lens, 4) || !aligned(query_offsets, 4) || !aligned(pages, 4) || !aligned(k_gs, 4) ||
        !aligned(v_gs, 4) || !aligned(lse, 4) || !aligned(workspace, 16))
        return NVFP4_ERROR_MISALIGNED;
    const int64_t need = nvfp4_sparse_attention_workspace(tokens, heads, kv_heads, head_dim, page_size, num_seqs,
                                                          list_len);
    if (workspace_bytes < need || (need > 0 && !workspace))
        return NVFP4_ERROR_INVALID_VALUE;
    const SparsePlan p = sparse_plan(tokens, heads, kv_heads, head_dim, page_size, num_seqs, list_len);
    Sparse s = {};
    Attn& a = s.a;
    a.q = q;
    a.kp = k_packed;
    a.ks = k_scales;
    a.vp = v_packed;
    a.vs = v_scales;
    a.table = block_table;
    a.lens = seq_lens;
    a.offsets = query_offsets;
    a.k_gs = k_gs;
    a.v_gs = v_gs;
    a.out = out;
    a.lse = lse;
    a.part = (float*)workspace;
    a.ld_q = ld_q;
    a.ld_out = ld_out;
    a.ld_table = ld_table;
    a.tokens = (int)tokens;
    a.heads = heads;
    a.kv_heads = kv_heads;
    a.page = page_size;
    a.num_pages = (int)(num_slots / page_size);
    a.max_pages = (int)max_pages;
    a.num_seqs = (int)num_seqs;
    a.causal = 1;
    a.scale = scale;
    int shift = 0;
    while (((int64_t)1 << shift) < page_size)
        ++shift;
    a.page_shift = 31 + shift;
    a.page_magic = (uint32_t)((((uint64_t)1 << a.page_shift) + page_size - 1) / page_size);
    a.splits = p.splits;
    a.row_blocks = p.row_blocks;
    s.together = p.together;
    s.pages = pages;
    s.list_len = (int)list_len;
    if (head_dim == 64)
        launch<64>(s, p.block, stream);
    else if (head_dim == 128)
        launch<128>(s, p.block, stream);
    else
        launch<256>(s, p.block, stream);
    return launched();
}
