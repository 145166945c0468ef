// Attention over block-scaled E4M3 pools, bf16 q and o.
#include "pd_blocks_tc.cuh"

namespace pd {
bool blocks_tc_bf16(int head_dim, int rows, TreeKernels* k) {
    return rows > 16 ? blocks_tc_lookup<__nv_bfloat16, 32>(head_dim, k) : blocks_tc_lookup<__nv_bfloat16, 16>(head_dim, k);
}
}  // namespace pd
