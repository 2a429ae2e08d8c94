// paged.cuh -- device helpers shared by the paged key/value cache kernels.
#pragma once

#include "common.cuh"

namespace fp8fg {

// The sequence that owns new token t: the number of offsets <= t, less one
// (offsets[0 .. seqs] non-decreasing; the whole warp calls with one t).  -1 or
// seqs: t belongs to none.  The offsets are read side by side, 32 a step, so
// the latency is one load's for up to 32 sequences rather than a search's.
__device__ __forceinline__ int seq_of_token(const int32_t *__restrict__ offsets, int seqs, int64_t t, int lane)
{
    int n = 0;
    for (int i = lane; i - lane <= seqs; i += 32) {
        const bool le = i <= seqs && offsets[i] <= t;
        n += __popc(__ballot_sync(0xffffffffu, le));
    }
    return n - 1;
}

}  // namespace fp8fg
