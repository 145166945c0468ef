// Attention of many rows over E4M3 pools scaled by blocks of 16 rows or a multiple, f16 q and o.
#include "pd_tree_tc.cuh"

namespace pd {
bool blocks_wide16_f16(int head_dim, TreeKernels* k) { return blocks_wide_lookup<__half, kPoolBlocks16>(head_dim, k); }
}  // namespace pd
