// tree_mamba2_bf16.hip -- the tree kernels of Mamba-2 layers with bf16 io.
#include "tree_impl.h"

namespace replay {
hipError_t launch_tree_mamba2_bf16(int P, int N, int st, const TreeArgs &a, hipStream_t s) {
    return launch_tree<true, false>(P, N, st, a, s);
}
}  // namespace replay
