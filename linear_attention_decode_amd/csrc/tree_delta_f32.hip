// tree_delta_f32.hip -- the tree kernels of Gated DeltaNet layers with float32 io.
#include "tree_impl.h"

namespace replay {
hipError_t launch_tree_delta_f32(int P, int N, int st, const TreeArgs &a, hipStream_t s) {
    return launch_tree<false, true>(P, N, st, a, s);
}
}  // namespace replay
