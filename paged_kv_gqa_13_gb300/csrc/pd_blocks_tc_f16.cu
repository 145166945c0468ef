// Attention over block-scaled E4M3 pools, f16 q and o.
#include "pd_blocks_tc.cuh"

namespace pd {
bool blocks_tc_f16(int head_dim, TreeKernels* k) { return blocks_tc_lookup<__half, 16>(head_dim, k); }
}  // namespace pd
