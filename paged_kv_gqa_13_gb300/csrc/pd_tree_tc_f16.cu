// Tensor-core tree decode with f16 q over pools of the same type.
#include "pd_tree_tc.cuh"

namespace pd {
bool tree_tc_f16(int D, bool wide, TreeKernels* k) { return tree_tc_lookup<__half, false>(D, wide, k); }
}  // namespace pd
