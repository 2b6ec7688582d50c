// tree.h -- private declarations of the tree calls (tree.hip, tree_*.hip).
#pragma once

#include "internal.h"

namespace replay {

// Most values in a node's rows of q, k or v: 64 of them then stay within 31-bit byte offsets.
constexpr int64_t kMaxTreeRow = 1 << 23;

// Outputs of a tree of W nodes a sequence, and its accepted path's append.
struct TreeArgs {
    RingView r;
    const void *S, *scale;             // as DecodeArgs
    const int32_t *parent, *n_nodes;   // [B][W]; [B] or null
    const void *q, *k, *v;             // [B][W][G][N] x2, [B][W][H][P]
    const float *dt, *a;               // [B][W][H]
    float *y;                          // [B][W][H][P]
    int32_t W;
};

hipError_t launch_tree_mamba2_bf16(int P, int N, int st, const TreeArgs &a, hipStream_t s);
hipError_t launch_tree_mamba2_f32(int P, int N, int st, const TreeArgs &a, hipStream_t s);
hipError_t launch_tree_delta_bf16(int P, int N, int st, const TreeArgs &a, hipStream_t s);
hipError_t launch_tree_delta_f32(int P, int N, int st, const TreeArgs &a, hipStream_t s);
// path [B][W], n_keep [B]: nodes path[b][0 .. n_keep[b]) appended to the ring
hipError_t launch_append_path(int P, int N, const TreeArgs &t, const int32_t *path, const int32_t *n_keep, void *ring_q,
                              void *ring_k, void *ring_v, float *ring_dt, float *ring_a, int32_t *pos, int32_t *sync,
                              hipStream_t s);

}  // namespace replay
