// tree.cuh -- the nodes of a tree of drafted tokens.
//
// parents[j] (j < K <= 64) is the place of node j's parent, a place before j; -1: the node follows the last
// cached token; below -1: the place holds no node.  A parent that is not before its child, or holds no node
// itself, makes the child none too, and is reported.
#pragma once
#include <cstdint>
#include "common.cuh"

namespace kda {

constexpr int kTreeMax = 64;

// The tree as one warp sees it: lane l has nodes l and l + 32, each as the set of itself and its ancestors (bit i:
// node i; 0 where there is no node).  A set reaches up to `far`; each round takes over the set of that ancestor and
// what it reaches up to, so a tree of depth d takes log2 d rounds.  Returns whether a parent has to be reported.
__device__ __forceinline__ bool tree_sets(const int32_t* __restrict__ parents, int K, int lane, uint64_t (&set)[2]) {
    int far[2];                                 // -1: complete; -2: no node
    bool given[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int j = lane + 32 * s;
        const int p = j < K ? __ldg(parents + j) : -2;
        given[s] = p >= -1;
        far[s] = p < -1 || p >= j ? -2 : p;
        set[s] = 1ull << j;
    }
    while (__any_sync(0xffffffffu, far[0] >= 0 || far[1] >= 0)) {
        uint64_t up[2];
        int next[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int from = far[s] & 31;
            const uint64_t s0 = __shfl_sync(0xffffffffu, set[0], from), s1 = __shfl_sync(0xffffffffu, set[1], from);
            const int f0 = __shfl_sync(0xffffffffu, far[0], from), f1 = __shfl_sync(0xffffffffu, far[1], from);
            up[s] = far[s] >= 32 ? s1 : s0;
            next[s] = far[s] >= 32 ? f1 : f0;
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (far[s] >= 0) {
                set[s] |= up[s];
                far[s] = next[s];
            }
    }
    bool report = false;
#pragma unroll
    for (int s = 0; s < 2; ++s)
        if (far[s] == -2) {
            set[s] = 0;
            report |= given[s];
        }
    return __any_sync(0xffffffffu, report);
}
// The set of node j (the same for every lane, or one a lane).
__device__ __forceinline__ uint64_t tree_set_of(const uint64_t (&set)[2], int j) {
    const uint64_t s0 = __shfl_sync(0xffffffffu, set[0], j & 31), s1 = __shfl_sync(0xffffffffu, set[1], j & 31);
    return j >= 32 ? s1 : s0;
}

}  // namespace kda
