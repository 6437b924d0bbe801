// What the sparse-attention kernels share: whose token is whose.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sparse {

// The request b of token t, offsets[b] <= t < offsets[b + 1], -1 if it is none's. The
// t-th request (single tokens) or the last one (a chunk) is tried first, which takes
// one round of loads; a wave then counts 64 offsets at a time. Offsets that fall
// may give -1, but never a request that ends in front of the token, which a loop over
// tokens could not leave.
__device__ __forceinline__ int request_of(const int32_t* offsets, int num_seqs, int t)
{
    const int guess = min(t, num_seqs - 1);
    if (offsets[guess] <= t && t < offsets[guess + 1])
        return guess;
    const int lane = threadIdx.x & 63;
    int b = -1;
#pragma unroll 1
    for (int base = 0; base <= num_seqs; base += 64) {
        const int i = base + lane;
        b += __popcll(__ballot(i <= num_seqs && offsets[min(i, num_seqs)] <= t));
    }
    return b < 0 || b >= num_seqs || offsets[b] > t || offsets[b + 1] <= t ? -1 : b;
}

}  // namespace sparse
