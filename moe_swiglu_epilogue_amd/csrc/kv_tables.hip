// Block tables and slot maps of a paged cache (include/nvfp4_serving.h).
//
// The whole of it is two prefix sums over the requests (new tokens, new
// pages) and a map: token i belongs to the last request whose offset is <= i,
// new page j to the last request whose page base is <= j. One launch, no
// workgroup waits for another: each workgroup scans all lengths itself (at
// most 4096 of them, out of L2) into LDS and then maps its own share of the
// tokens, pages and requests with binary searches there. Bound by latency:
// a launch, two rounds of dependent loads (lengths; table or free list) and
// the stores. 256 requests of one new token take 5.2 us, 48 prompts of up to
// 8192 tokens 8.3 us on the GPU, where a launch of nothing takes about 3; a
// call from Python about 10.6, most of it the host's.
#include "serving_common.hpp"

namespace {

constexpr int kThreads = 256;
constexpr int kMaxSeqs = 4096;
constexpr int kTokensPerGroup = 1024;

struct Tables {
    const int32_t* context;
    const int32_t* query;
    const int32_t* free_pages;
    const int32_t* free_begin;
    int32_t* table;
    int32_t* offsets;
    int32_t* lens;
    int64_t* slots;
    int32_t* free_end;
    int64_t ld_table;
    int num_seqs, page, num_free, max_pages, max_tokens;   // num_free < 0: no list
};

struct Request {
    int64_t context, total;   // tokens before and after
    int held, want;           // table entries there already, and after
};

__device__ __forceinline__ Request request(const Tables& a, int b)
{
    Request r;
    r.context = a.context ? max(a.context[b], 0) : 0;
    // at most 2^31 - 1, so that total + page - 1 stays below 2^32
    r.total = min(r.context + max(a.query[b], 0), (int64_t)INT32_MAX);
    r.want = (int)min((uint32_t)(r.total + a.page - 1) / (uint32_t)a.page, (uint32_t)a.max_pages);
    r.held = a.num_free >= 0
                 ? min((int)((uint32_t)(r.context + a.page - 1) / (uint32_t)a.page), r.want)
                 : r.want;
    return r;
}

__device__ __forceinline__ int saturate(int64_t v) { return (int)min(v, (int64_t)INT32_MAX); }

// Index of the last entry of v[0..n] (v[0] == 0, non-decreasing) that is <= i.
__device__ __forceinline__ int last_at_most(const int* v, int n, int i)
{
    int lo = 0, hi = n + 1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= i)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(kThreads) void kv_tables_kernel(Tables a)
{
    __shared__ int offset[kMaxSeqs + 1], base[kMaxSeqs + 1];
    __shared__ int64_t wave_tokens[kThreads / 64], wave_pages[kThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = a.num_seqs;

    // Exclusive sums: each thread adds up a run of requests, the runs' sums
    // are scanned over the workgroup, then each thread walks its run again.
    const int run = (n + kThreads - 1) / kThreads;
    const int first = min(tid * run, n), last = min(first + run, n);
    int64_t tokens = 0, pages = 0;
    for (int b = first; b < last; ++b) {
        const Request r = request(a, b);
        tokens += r.total - r.context;
        pages += r.want - r.held;
    }
    int64_t t = tokens, p = pages;
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t t2 = __shfl_up(t, d), p2 = __shfl_up(p, d);
        if (lane >= d) {
            t += t2;
            p += p2;
        }
    }
    if (lane == 63) {
        wave_tokens[wave] = t;
        wave_pages[wave] = p;
    }
    __syncthreads();
    int64_t before_t = t - tokens, before_p = p - pages, all_t = 0, all_p = 0;
    for (int w = 0; w < kThreads / 64; ++w) {
        if (w < wave) {
            before_t += wave_tokens[w];
            before_p += wave_pages[w];
        }
        all_t += wave_tokens[w];
        all_p += wave_pages[w];
    }
    for (int b = first; b < last; ++b) {
        const Request r = request(a, b);
        offset[b] = saturate(before_t);
        base[b] = saturate(before_p);
        before_t += r.total - r.context;
        before_p += r.want - r.held;
    }
    if (tid == 0) {
        offset[n] = saturate(all_t);
        base[n] = saturate(all_p);
    }
    __syncthreads();

    int begin = a.free_begin ? a.free_begin[0] : 0;
    int left = max(a.num_free, 0) - begin;      // pages left in the list
    if (begin < 0 || left < 0) {
        begin = 0;
        left = 0;
    }
    const int step = gridDim.x * kThreads, at = blockIdx.x * kThreads + tid;
    for (int b = at; b < n; b += step) {
        a.offsets[b] = offset[b];
        a.lens[b] = (int)request(a, b).total;
    }
    if (at == 0) {
        a.offsets[n] = offset[n];
        a.free_end[0] = saturate((int64_t)begin + base[n]);
    }
    // new pages into the table
    const int new_pages = base[n];
    for (int64_t j = at; j < new_pages; j += step) {
        const int b = last_at_most(base, n, (int)j);
        const int col = request(a, b).held + (int)j - base[b];
        a.table[b * a.ld_table + col] = j < left ? a.free_pages[begin + j] : -1;
    }
    // slots of the new tokens; no new table entry is read back from memory
    const int real = offset[n];
    for (int64_t i = at; i < a.max_tokens; i += step) {
        int64_t slot = -1;
        if (i < real) {
            const int b = last_at_most(offset, n, (int)i);
            const Request r = request(a, b);
            const uint32_t pos = (uint32_t)(r.context + (i - offset[b]));
            const uint32_t col = pos / (uint32_t)a.page;
            int page = -1;
            if (col < (uint32_t)r.held) {
                page = a.table[b * a.ld_table + col];
            } else if (col < (uint32_t)r.want) {
                const int64_t j = (int64_t)base[b] + (col - r.held);
                page = j < left ? a.free_pages[begin + j] : -1;
            }
            if (page >= 0)
                slot = (int64_t)page * a.page + (pos - col * (uint32_t)a.page);
        }
        a.slots[i] = slot;
    }
}

// `rows` rows of `bytes` bytes, `pitch` bytes apart; one row for a vector.
struct Memory {
    uintptr_t at;
    int64_t rows, pitch, bytes;
};

Memory vector(const void* p, int64_t bytes) { return {(uintptr_t)p, 1, bytes, p ? bytes : 0}; }

// Whether a vector touches some row of m.
bool shared(const Memory& v, const Memory& m)
{
    if (v.bytes == 0 || m.rows == 0 || m.bytes == 0)
        return false;
    if (v.at < m.at)
        return m.at - v.at < (uintptr_t)v.bytes;
    const uintptr_t off = v.at - m.at;       // in row off / pitch, or in the gap behind it
    const int64_t row = off / (uintptr_t)m.pitch < (uintptr_t)m.rows ? (int64_t)(off / (uintptr_t)m.pitch) : m.rows - 1;
    const uintptr_t in_row = off - (uintptr_t)row * m.pitch;
    return in_row < (uintptr_t)m.bytes || (row + 1 < m.rows && m.pitch - in_row < (uintptr_t)v.bytes);
}

}  // namespace

extern "C" nvfp4_status_t kv_block_tables(const int32_t* context_lens, const int32_t* query_lens,
                                          int64_t num_seqs, int32_t page_size,
                                          const int32_t* free_pages, int64_t num_free,
                                          const int32_t* free_begin, int32_t* block_table,
                                          int64_t ld_table, int64_t max_pages,
                                          int32_t* query_offsets, int32_t* seq_lens,
                                          int64_t* slots, int64_t max_tokens, int32_t* free_end,
                                          hipStream_t stream)
{
    using namespace serving;
    if (num_seqs < 0 || page_size < 1 || num_free < -1 || max_pages < 0 || max_tokens < 0 ||
        ld_table < max_pages || !extent_ok(num_seqs, ld_table, 4))
        return NVFP4_ERROR_INVALID_VALUE;
    if (num_seqs > kMaxSeqs || num_free > INT32_MAX || max_pages > INT32_MAX ||
        max_tokens > INT32_MAX)
        return NVFP4_ERROR_UNSUPPORTED_SHAPE;
    if ((num_seqs > 0 && (!query_lens || !seq_lens || (max_pages > 0 && !block_table))) ||
        !query_offsets || !free_end || (max_tokens > 0 && !slots) || (num_free > 0 && !free_pages))
        return NVFP4_ERROR_INVALID_VALUE;
    if (!aligned(context_lens, 4) || !aligned(query_lens, 4) || !aligned(free_pages, 4) ||
        !aligned(free_begin, 4) || !aligned(block_table, 4) || !aligned(query_offsets, 4) ||
        !aligned(seq_lens, 4) || !aligned(slots, 8) || !aligned(free_end, 4))
        return NVFP4_ERROR_MISALIGNED;
    // Every workgroup reads all lengths and what it needs of the lists, and none
    // waits for another: a written value must not be one that is read.
    const Memory in[] = {vector(context_lens, 4 * num_seqs), vector(query_lens, 4 * num_seqs),
                         vector(free_pages, num_free > 0 ? 4 * num_free : 0), vector(free_begin, 4)};
    const Memory out[] = {vector(query_offsets, 4 * num_seqs + 4), vector(seq_lens, 4 * num_seqs),
                          vector(slots, 8 * max_tokens), vector(free_end, 4)};
    const Memory table = {(uintptr_t)block_table, num_seqs, 4 * ld_table, 4 * max_pages};
    for (int i = 0; num_seqs > 0 && i < 4; ++i) {
        if (shared(out[i], table) || shared(in[i], table))
            return NVFP4_ERROR_INVALID_VALUE;
        for (int j = 0; j < 4; ++j)
            if (shared(out[i], in[j]) || (j < i && shared(out[i], out[j])))
                return NVFP4_ERROR_INVALID_VALUE;
    }
    Tables a = {context_lens, query_lens, free_pages, free_begin, block_table, query_offsets,
                seq_lens, slots, free_end, ld_table, (int)num_seqs, page_size, (int)num_free,
                (int)max_pages, (int)max_tokens};
    int64_t groups = ceil_div(max_tokens, (int64_t)kTokensPerGroup);
    groups = groups < 1 ? 1 : groups > 1024 ? 1024 : groups;
    hipLaunchKernelGGL(kv_tables_kernel, dim3((unsigned)groups), dim3(kThreads), 0, stream, a);
    return launched();
}
