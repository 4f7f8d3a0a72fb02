// tree.cuh -- trees of drafted tokens (include/spec_tree.h): parents and ancestors of
// the up to 32 rows of a request, one lane of a warp each.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "spec_tree.h"

namespace specv {

// The parent of node `lane` of the request whose first row is `lo`, -1 for none.  A warp
// calls it; `status`: where to report a parent that is not before its node, or null.
__device__ __forceinline__ int tree_parent(const int32_t *parent, int lo, int n, uint32_t *status)
{
    const int lane = threadIdx.x & 31;
    if (lane == 0 || lane >= n) return -1;
    const int p = parent ? __ldg(parent + lo + lane) : lane - 1;
    if (p >= lane || p < -1) {
        set_status(status, SPEC_STATUS_BAD_TREE);
        return -1;
    }
    return p;
}

// The node's ancestors and itself, a bit each: after step s those up to 2^s above it.  All
// 32 lanes of the warp have to call it.
__device__ __forceinline__ uint32_t tree_ancestors(int parent)
{
    const int lane = threadIdx.x & 31;
    uint32_t anc = 1u << lane;
    int p = parent;
#pragma unroll
    for (int s = 0; s < 5; ++s) {
        const int from = p >= 0 ? p : lane;
        const uint32_t a = __shfl_sync(0xFFFFFFFFu, anc, from);
        const int q = __shfl_sync(0xFFFFFFFFu, p, from);
        if (p >= 0) {
            anc |= a;
            p = q;
        }
    }
    return anc;
}

}  // namespace specv
