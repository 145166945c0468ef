// Attention over block-scaled E4M3 pools, bf16 q and o.
#include "pd_blocks_tc.cuh"

namespace pd {
bool blocks_tc_bf16(int head_dim, int rows, TreeKernels* k) { return blocks_tc_by_rows<__nv_bfloat16>(head_dim, rows, k); }
}  // namespace pd
