// Attention of many rows over block-scaled E4M3 pools, bf16 q and o.
#include "pd_tree_tc.cuh"

namespace pd {
bool blocks_wide_bf16(int head_dim, TreeKernels* k) { return blocks_wide_lookup<__nv_bfloat16, kPoolBlocks>(head_dim, k); }
}  // namespace pd
