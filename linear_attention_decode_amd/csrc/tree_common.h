// tree_common.h -- the tree of a sequence's drafted tokens, as the tree calls
// (conv.hip, tree.hip) read it: node w follows node parent[w] < w, or, where
// that is -1, the sequence's newest token.
#pragma once

#include "device_common.h"
#include "prompt.h"

namespace replay {

// In every wavefront of 64: lane w has node w.
struct Tree {
    int parent;   // -1 too for the lanes past the nodes
    int n;        // nodes; 0 where the tree is none
    bool ok;      // 0 <= n <= W, -1 <= parent[w] < w
    __device__ __forceinline__ void load(const int32_t *parents, const int32_t *n_nodes, int b, int W, int lane) {
        n = n_nodes ? n_nodes[b] : W;
        const int p = lane < W ? parents[(size_t)b * W + lane] : -1;
        ok = n >= 0 && n <= W && !__any(lane < n && (p < -1 || p >= lane));
        n = __builtin_amdgcn_readfirstlane(ok ? n : 0);
        parent = lane < n ? p : -1;
    }
    // of count nodes, 0 <= count <= W, p loaded already
    __device__ __forceinline__ void set(int p, int count, int lane) {
        ok = !__any(lane < count && (p < -1 || p >= lane));
        n = count;
        parent = lane < count ? p : -1;
    }
    // one step up from x: a node, or -s for the s-th token before the tree
    __device__ __forceinline__ int up(int x) const {
        const int p = __shfl(parent, x < 0 ? 0 : x);
        return x < 0 ? x - 1 : p;
    }
};

}  // namespace replay
