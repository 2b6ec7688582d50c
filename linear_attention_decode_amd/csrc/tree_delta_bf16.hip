// tree_delta_bf16.hip -- the tree kernels of Gated DeltaNet layers with bf16 io.
#include "tree_impl.h"

namespace replay {
hipError_t launch_tree_delta_bf16(int P, int N, int st, const TreeArgs &a, hipStream_t s) {
    return launch_tree<true, true>(P, N, st, a, s);
}
}  // namespace replay
