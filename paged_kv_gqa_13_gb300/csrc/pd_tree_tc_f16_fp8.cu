// Tensor-core tree decode with f16 q over E4M3 pools.
#include "pd_tree_tc.cuh"

namespace pd {
bool tree_tc_f16_fp8(int D, bool wide, TreeKernels* k) { return tree_tc_lookup<__half, true>(D, wide, k); }
}  // namespace pd
