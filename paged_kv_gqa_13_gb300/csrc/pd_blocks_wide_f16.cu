// Attention of many rows over block-scaled E4M3 pools, f16 q and o.
#include "pd_tree_tc.cuh"

namespace pd {
bool blocks_wide_f16(int head_dim, TreeKernels* k) { return blocks_wide_lookup<__half, kPoolBlocks>(head_dim, k); }
}  // namespace pd
