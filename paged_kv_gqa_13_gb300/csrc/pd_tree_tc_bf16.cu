// Tensor-core tree decode with bf16 q over pools of the same type.
#include "pd_tree_tc.cuh"

namespace pd {
bool tree_tc_bf16(int D, bool wide, TreeKernels* k) { return tree_tc_lookup<__nv_bfloat16, false>(D, wide, k); }
}  // namespace pd
