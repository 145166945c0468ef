// Tensor-core tree decode with f16 q.
#include "pd_tree_kernels.h"
#include "pd_tree_tc.cuh"

namespace pd {

template <int D, bool kWide>
static TreeKernels tc_kernels() {
    using C = CfgTree<D, kWide>;
    TreeKernels k{};
    k.main = reinterpret_cast<const void*>(tree_tc_kernel<__half, D, kWide>);
    k.merge = reinterpret_cast<const void*>(tree_merge_kernel<__half, D>);
    k.threads = C::kThreads;
    k.smem = C::kBytes;
    k.per_sm = 1;
    k.tile_rows = C::kRows;
    k.tiles = C::kPipes;
    k.workers = C::kLines;
    k.block_tokens = C::kKeys;
    k.tensor = true;
    return k;
}

bool tree_tc_f16(int D, bool wide, TreeKernels* k) {
    switch (D) {
        case 64: *k = wide ? tc_kernels<64, true>() : tc_kernels<64, false>(); return true;
        case 128: *k = wide ? tc_kernels<128, true>() : tc_kernels<128, false>(); return true;
        case 256: *k = tc_kernels<256, false>(); return true;
    }
    return false;
}

}  // namespace pd
