// The tree decode's kernel variants, looked up by its host code.
#pragma once

namespace pd {

struct TreeKernels {
    const void* main;
    const void* merge;
    int threads, smem, per_sm;  // of main
    int tile_rows, tiles;       // rows of a row tile, row tiles per segment
    int workers;                // independent ranges of work per CTA
    int block_tokens;           // tokens of a key block
    int seg_cost;               // TreeArgs::seg_cost
    bool tensor;                // main runs on the tensor cores and takes tensor maps
    bool codes;                 // its operands are codes as they lie: maps of K and V alone
};

bool tree_tc_f16(int head_dim, bool wide, TreeKernels* k);
bool tree_tc_bf16(int head_dim, bool wide, TreeKernels* k);
bool tree_tc_f16_fp8(int head_dim, bool wide, TreeKernels* k);
bool tree_tc_bf16_fp8(int head_dim, bool wide, TreeKernels* k);
// over block-scaled E4M3 pools: up to 16 or 32 rows a row tile; many rows, with any blocks or (16) blocks of a multiple of
// 16 rows
bool blocks_tc_f16(int head_dim, TreeKernels* k);
bool blocks_tc_bf16(int head_dim, int rows, TreeKernels* k);
bool blocks_wide_f16(int head_dim, TreeKernels* k);
bool blocks_wide_bf16(int head_dim, TreeKernels* k);
bool blocks_wide16_f16(int head_dim, TreeKernels* k);
bool blocks_wide16_bf16(int head_dim, TreeKernels* k);

}  // namespace pd
