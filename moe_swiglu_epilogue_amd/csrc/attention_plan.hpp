// How nvfp4_paged_attention cuts its work: the host's plan, and the split of a
// range of tokens that its kernels take from it. Sizes and integers alone.
//
// All positions are below kMostTokens = 2^30, the most that a block table may
// cover. A plan keeps splits * chunk below kMostTokens + chunk, so that a
// split's first token, at most begin + (splits - 1) * chunk, stays below 2^31.
#pragma once

#include "serving_common.hpp"

namespace attention {

constexpr int64_t kMostTokens = 1 << 30;

struct Plan {
    int block;         // query rows of a workgroup: 16, 32, 48, 64, or 256 (the prompt kernel)
    int row_blocks;    // workgroups over a request's rows
    int splits, chunk; // of the tokens
};

inline Plan make_plan(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t head_dim, int64_t num_seqs,
                      int64_t max_query_len, int64_t max_seq_len, int64_t window)
{
    using serving::ceil_div;
    Plan p;
    const int64_t group = heads / kv_heads;
    const int64_t rows = (max_query_len < 1 ? 1 : max_query_len > (1 << 20) ? 1 << 20 : max_query_len) * group;
    // Few rows go to the rows kernel in one or two equal blocks of whole 16 (24
    // requests of 5 tokens, 40 rows, head_dim 64: 21 us with a block of 48, 24 with
    // one of 64), for head_dim 256 in one or two of 16, as its registers hold no
    // more.
    if (head_dim > 128)
        p.block = rows <= 32 ? 16 : 256;
    else
        p.block = rows <= 64 ? (int)ceil_div(rows, (int64_t)16) * 16
                  : rows <= 128 ? (int)ceil_div(rows, (int64_t)32) * 16 : 256;
    int64_t blocks = ceil_div(rows, (int64_t)p.block);
    p.row_blocks = (int)(blocks > 4096 ? 4096 : blocks);
    int64_t range = max_seq_len > kMostTokens ? kMostTokens : max_seq_len;
    if (window > 0 && window < range && window + rows / group + 32 < range)
        range = window + rows / group + 32;
    const int64_t items = (num_seqs < 1 ? 1 : num_seqs) * kv_heads * p.row_blocks;
    // One round of workgroups on the card's 256 compute units, as many on each
    // as its registers hold, by splits of at least `shortest` tokens; for few rows
    // also splits short enough that ragged requests balance (prompt kernel: half
    // as many workgroups again, as most blocks see less than the longest).
    const bool prompt = p.block == 256;
    const int64_t slots = prompt ? 384 : 256 * (p.block == 16 && head_dim <= 128 ? 3 : head_dim * p.block <= 4096 ? 2 : 1);
    const int64_t shortest = prompt ? 1024 : 128;
    int64_t splits = slots / items < 1 ? 1 : slots / items;
    if (!prompt && splits < ceil_div(range, (int64_t)2048))
        splits = ceil_div(range, (int64_t)2048);
    if (splits > ceil_div(range < 1 ? 1 : range, shortest))
        splits = ceil_div(range < 1 ? 1 : range, shortest);
    if (splits > 256)
        splits = 256;
    // grids stay below 2^32 work-items, 2^23 workgroups of 512 (rows and splits left
    // out are looped over; 8 kv_heads for the rounding in launch)
    if (tokens * heads > (1 << 22))
        splits = 1;
    const int64_t most = ((1 << 23) - 8 * 1024 - 1) / ((num_seqs < 1 ? 1 : num_seqs) * kv_heads);
    if (splits * p.row_blocks > most) {
        splits = 1;
        if (p.row_blocks > most)
            p.row_blocks = (int)(most < 1 ? 1 : most);
    }
    const int64_t chunk = ceil_div(ceil_div(range, splits), (int64_t)128) * 128;
    p.chunk = (int)(chunk < 128 ? 128 : chunk);
    p.splits = (int)ceil_div(range < 1 ? 1 : range, (int64_t)p.chunk);
    return p;
}

// Tokens of a split of a range of `total`: more than planned where the range is
// longer than promised.
__host__ __device__ inline int chunk_of(int planned, int splits, int total)
{
    const int even = ((total + splits - 1) / splits + 127) & ~127;
    return planned > even ? planned : even;
}

// The end of the split that begins at `first`, not behind the range's (which a
// split past the last one begins behind).
__host__ __device__ inline int last_of(int first, int chunk, int end)
{
    return end - first < chunk ? end : first + chunk;
}

}  // namespace attention
