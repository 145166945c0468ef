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
};

bool tree_tc_f16(int head_dim, bool wide, TreeKernels* k);
bool tree_tc_bf16(int head_dim, bool wide, TreeKernels* k);
bool tree_tc_f16_fp8(int head_dim, bool wide, TreeKernels* k);
bool tree_tc_bf16_fp8(int head_dim, bool wide, TreeKernels* k);
// over block-scaled E4M3 pools; rows: of a request
bool blocks_tc_f16(int head_dim, int rows, TreeKernels* k);
bool blocks_tc_bf16(int head_dim, int rows, TreeKernels* k);

}  // namespace pd
