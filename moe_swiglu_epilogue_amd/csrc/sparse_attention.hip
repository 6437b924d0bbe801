// Attention over listed pages of the paged NVFP4 cache (include/nvfp4_sparse.h).
//
// A token's listed pages, one behind the other, are a range of list_len *
// page_size tokens, which a workgroup walks in tiles of 32 as the rows kernel of
// paged_attention.hip does with a request's tokens (attention_rows.hpp): the same
// arithmetic, one (token, key/value head) a workgroup, whose query rows are the
// heads that share the key/value head. The workgroup first looks the list up: for
// each entry the page in the cache and how many of its tokens the query sees.
#include "attention_rows.hpp"
#include "nvfp4_sparse.h"

namespace {

constexpr int kMostListed = 2048;

struct Sparse {
    Attn a;
    const int32_t* pages;
    int list_len;
};

// The request of token t, -1 if it is none's: the last b with offsets[b] <= t.
__device__ __forceinline__ int request_of(const Attn& a, int t, int lane)
{
    int b = -1;
    for (int base = 0; base <= a.num_seqs; base += 64) {
        const int i = base + lane;
        b += __popcll(__ballot(i <= a.num_seqs && a.offsets[min(i, a.num_seqs)] <= t));
    }
    return b >= a.num_seqs ? -1 : b;
}

// The listed pages of a workgroup's range: the page in the cache, -1 where the
// query sees nothing of it, and the number of its tokens that it sees.
struct Listed {
    int page[kMostListed], seen[kMostListed];
};

template <int D>
union Shared {
    Joined<D> joined;
    Listed list;
};

template <int D, int RT, bool kPaged16>
__global__ __launch_bounds__(256, (D * RT <= 256 ? 2 : 1)) void sparse_rows_kernel(Sparse s)
{
    using T = Tile<D>;
    constexpr int C = T::C, KF = D / 32, VM = T::VM;
    __shared__ Shared<D> lds;
    __shared__ int ends[4];
    const Attn& a = s.a;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, n = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = a.heads / a.kv_heads;
    const float k_scale = a.scale * (a.k_gs ? a.k_gs[0] : 1.0f) * kLog2e;

    // As in the rows kernel: all key/value heads of a token go to one XCD
    const int64_t per_split = (int64_t)a.tokens * a.row_blocks;
    const int64_t units = (per_split * a.splits + 7) / 8 * 8 * a.kv_heads;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t j = unit >> 3, work = j / a.kv_heads * 8 + (unit & 7);
        const int h = (int)(j % a.kv_heads);
        if (work >= per_split * a.splits)
            continue;
        const int split = (int)(work / per_split);
        const int64_t item = work % per_split;
        const int token = (int)(item / a.row_blocks), row0 = (int)(item % a.row_blocks) * 16 * RT;
        const int b = request_of(a, token, lane);
        if (b < 0)
            continue;
        const int len = a.num_pages > 0 ? min(max(a.lens[b], 0), a.max_pages * a.page) : 0;
        const int position = min(len - a.offsets[b + 1] + token, len - 1);

        // the list of this split
        const int first = split * a.chunk;
        const int most = min(first + a.chunk, s.list_len * a.page);
        const int page0 = (int)page_of(a, first), pages = most > first ? (int)page_of(a, most - 1) - page0 + 1 : 0;
        const int32_t* list = s.pages + ((int64_t)token * a.kv_heads + h) * s.list_len + page0;
        int used = 0;
        __syncthreads();                        // the LDS of the item before is read
        for (int i = tid; i < pages; i += 256) {
            const int p = list[i];
            int entry = -1, seen = 0;
            if (p >= 0 && p < a.max_pages) {
                entry = a.table[b * a.ld_table + p];
                // a page behind the token's own: nothing
                seen = (int)min(max((int64_t)position + 1 - (int64_t)p * a.page, (int64_t)0), (int64_t)a.page);
            }
            const bool in = entry >= 0 && entry < a.num_pages && seen > 0;
            lds.list.page[i] = in ? entry : -1;
            lds.list.seen[i] = in ? seen : 0;
            used = in ? i + 1 : used;
        }
        for (int d = 32; d; d >>= 1)
            used = max(used, __shfl_xor(used, d));
        if (lane == 0)
            ends[wave] = used;
        __syncthreads();
        used = max(max(ends[0], ends[1]), max(ends[2], ends[3]));
        const int last = __builtin_amdgcn_readfirstlane((int)min((int64_t)most, ((int64_t)page0 + used) * a.page));

        auto entries = [&](int t0) {
            Entries r = {{-1, -1}};
            if (kPaged16)
                for (int hh = 0; hh < 2; ++hh)
                    if (t0 + 16 * hh < last)
                        r.e[hh] = __builtin_amdgcn_readfirstlane(lds.list.page[(int)page_of(a, t0 + 16 * hh) - page0]);
            return r;
        };
        auto request = [&](Tile<D>& t, int t0) {
            if (t0 >= last)
                return;
            load_tile<D, kPaged16>(t, a, lds.list.page - page0, entries(t0), h, t0, first, last, lane);
            const int at = min(t0 + (lane & 31), last - 1), p = (int)page_of(a, at);
            t.shown = t.shown && at - p * a.page < lds.list.seen[p - page0];
            __builtin_amdgcn_sched_barrier(0);
        };

        half8v q[RT][KF];
        float factor[RT];
        int lo[RT], hi[RT];
        for (int rt = 0; rt < RT; ++rt) {
            const int r = row0 + 16 * rt + n;
            lo[rt] = 0;
            hi[rt] = r < group ? INT32_MAX : 0;
            const uint16_t* src = a.q + token * a.ld_q + (h * group + min(r, group - 1)) * D;
            uint4v w[KF];
            uint32_t top = 0;
            for (int f = 0; f < KF; ++f) {
                w[f] = *(const uint4v*)(src + (D > 64 ? 128 * (f / 4) + 32 * g + 8 * (f % 4) : 16 * g + 8 * f));
                top = largest_bits(w[f], top);
            }
            top = max(top, (uint32_t)__shfl_xor((int)top, 16));
            top = max(top, (uint32_t)__shfl_xor((int)top, 32));
            const int e = fp16_exponent(top);
            for (int f = 0; f < KF; ++f)
                q[rt][f] = scaled_half8(w[f], e, k_scale < 0);
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
        for (int t0 = first + 32 * wave; t0 < last; t0 += 128) {
            Tile<D> tile;
            request(tile, t0);
            attend<D, RT>(tile, t0, lane, q, factor, lo, hi, 0, INT32_MAX, m, l, o);
        }
        __syncthreads();                        // the list is read, its LDS goes to the join
        join_waves<D, RT>(a, lds.joined, split, a.splits, token, group, row0, h, m, l, o);
    }
}

// How the work is cut: 16 RT query rows a workgroup, and splits of the listed
// tokens where there are too few workgroups for the card.
struct SparsePlan {
    int block, row_blocks, splits, chunk;
};

SparsePlan sparse_plan(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t head_dim, int32_t page_size,
                       int64_t list_len)
{
    using serving::ceil_div;
    SparsePlan p;
    const int group = heads / kv_heads;
    p.block = head_dim > 128 ? 16 : group <= 64 ? ceil_div(group, 16) * 16 : 64;
    p.row_blocks = ceil_div(group, p.block);
    const int64_t range = list_len * page_size, items = tokens * kv_heads * p.row_blocks;
    const int64_t slots = 512;
    int64_t splits = items < 1 ? 1 : slots / items;
    if (splits > ceil_div(range, (int64_t)128))
        splits = ceil_div(range, (int64_t)128);
    if (splits > 256)
        splits = 256;
    if (splits < 1 || tokens * heads > (1 << 22))
        splits = 1;
    const int64_t chunk = ceil_div(ceil_div(range, splits), (int64_t)128) * 128;
    p.chunk = (int)(chunk < 128 ? 128 : chunk);
    p.splits = (int)ceil_div(range < 1 ? 1 : range, (int64_t)p.chunk);
    return p;
}

template <int D, int RT>
void launch_rows(const Sparse& s, dim3 grid, hipStream_t stream)
{
    if (s.a.page % 16 == 0)
        hipLaunchKernelGGL((sparse_rows_kernel<D, RT, true>), grid, dim3(256), 0, stream, s);
    else
        hipLaunchKernelGGL((sparse_rows_kernel<D, RT, false>), grid, dim3(256), 0, stream, s);
}

template <int D>
void launch(const Sparse& s, int block, hipStream_t stream)
{
    const Attn& a = s.a;
    const int64_t work = (int64_t)a.tokens * a.row_blocks * a.splits;
    const int64_t units = (work + 7) / 8 * 8 * a.kv_heads;
    // a grid holds less than 2^32 threads; workgroups take several items beyond 2^22
    const dim3 grid((unsigned)(units < (1 << 22) ? units : 1 << 22));
    if (block == 16) {
        launch_rows<D, 1>(s, grid, stream);
    } else if constexpr (D <= 128) {
        if (block == 32)
            launch_rows<D, 2>(s, grid, stream);
        else if (block == 48)
            launch_rows<D, 3>(s, grid, stream);
        else
            launch_rows<D, 4>(s, grid, stream);
    }
    if (a.splits > 16)
        hipLaunchKernelGGL((attn_join_kernel<D, 4>), dim3((unsigned)(a.tokens * a.heads)), dim3(256), 0, stream, a);
    else if (a.splits > 1)
        hipLaunchKernelGGL((attn_join_kernel<D, 1>), dim3((unsigned)(a.tokens * a.heads + 3) / 4), dim3(256), 0, stream, a);
}

bool sizes_ok(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t page_size, int64_t list_len)
{
    return tokens >= 0 && heads >= 1 && kv_heads >= 1 && heads % kv_heads == 0 && page_size >= 1 && list_len >= 0;
}

bool sizes_supported(int64_t tokens, int32_t heads, int32_t head_dim, int32_t page_size, int64_t list_len)
{
    return (head_dim == 64 || head_dim == 128 || head_dim == 256) && heads <= 1024 && tokens <= (1 << 30) / heads &&
           list_len <= kMostListed && list_len <= (1 << 30) / page_size;
}

}  // namespace

extern "C" int64_t nvfp4_sparse_attention_workspace(int64_t tokens, int32_t heads, int32_t kv_heads,
                                                    int32_t head_dim, int32_t page_size, int64_t list_len)
{
    if (!sizes_ok(tokens, heads, kv_heads, page_size, list_len) ||
        !sizes_supported(tokens, heads, head_dim, page_size, list_len))
        return -1;
    const SparsePlan p = sparse_plan(tokens, heads, kv_heads, head_dim, page_size, list_len);
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
    if (!sizes_supported(tokens, heads, head_dim, page_size, list_len) || num_slots > INT32_MAX || num_seqs > 65535 ||
        num_seqs * kv_heads > (1 << 22) || max_pages > (1 << 30) / page_size)
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
    const int64_t need = nvfp4_sparse_attention_workspace(tokens, heads, kv_heads, head_dim, page_size, list_len);
    if (workspace_bytes < need || (need > 0 && !workspace))
        return NVFP4_ERROR_INVALID_VALUE;
    const SparsePlan p = sparse_plan(tokens, heads, kv_heads, head_dim, page_size, list_len);
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
    a.chunk = p.chunk;
    a.row_blocks = p.row_blocks;
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
