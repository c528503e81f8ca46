// What the prompt attention kernels share: the blocks of rows of a packed batch.
#pragma once
#include "common.cuh"
#include "launchers.h"

namespace dsa {

// First row and length of a prompt; bounds that lie outside the rows are
// reported and leave it empty.
__device__ __forceinline__ void prompt_bounds(const PromptArgs& a, int seq, int& start, int& len) {
    start = a.cu_seqlens[seq];
    len = a.cu_seqlens[seq + 1] - start;
    if (start < 0 || len < 0 || (int64_t)start + len > a.total) {
        record_error(a.err, DEV_ERR_BAD_INDEX);
        start = len = 0;
    }
}

// Up to 32 prompts, one per lane of a warp, and their blocks of rows in falling
// order of their number within their prompt, which is their work.
constexpr int LANE_SEQS = 32;
struct PromptLanes {
    int start, len, blocks;         // of prompt `lane`

    __device__ __forceinline__ void init(const PromptArgs& a, int rows_per_block) {
        const int lane = threadIdx.x & 31;
        start = len = 0;
        if (lane < a.n_seqs) prompt_bounds(a, lane, start, len);
        blocks = (len + rows_per_block - 1) / rows_per_block;
    }
    // row blocks whose number (from 1) within their prompt is at least v
    __device__ __forceinline__ int at_least(int v) const {
        return (int)__reduce_add_sync(0xffffffffu, (unsigned)max(0, blocks - v + 1));
    }
    // Block e, 0 <= e < at_least(1): its prompt's first row and length, its number (from 0).
    __device__ __forceinline__ void get(int e, int& first, int& n, int& block) const {
        int lo = 1, hi = (int)__reduce_max_sync(0xffffffffu, (unsigned)blocks) + 1;
        while (hi - lo > 1) {                   // at_least(lo) > e >= at_least(hi)
            const int mid = (lo + hi) >> 1;
            if (at_least(mid) > e) lo = mid;
            else hi = mid;
        }
        const unsigned have = __ballot_sync(0xffffffffu, blocks >= lo);
        const int seq = (int)__fns(have, 0, e - at_least(lo + 1) + 1);
        first = __shfl_sync(0xffffffffu, start, seq);
        n = __shfl_sync(0xffffffffu, len, seq);
        block = lo - 1;
    }
};

}  // namespace dsa
