// Host-side helpers of the C ABI shared by its translation units: the
// thread's error message, argument checks and per-device facts (pd_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <cudaTypedefs.h>

#include "pagedecode.h"

namespace pd {
namespace host {

pd_status fail(pd_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
pd_status ok();
pd_status cuda_fail(cudaError_t e, const char* what);
pd_status check_workspace(void* ws, size_t have, size_t need);
pd_status sm_count(int* sms);
pd_status allow_smem(const void* fn, int bytes);
// A block of block_tokens rows divides a page (pd_norm_rope.cu).
pd_status check_block(int block_tokens, int page_size);
// Checks of a rotation's arguments, shared by the calls that rotate (pd_rope.cu).
pd_status check_rotation(int tokens, int head_dim, int rot_dim, int layout, float rope_scale, const uint64_t* freqs, pd_dtype dt);
// pd_paged_decode_fp8_blocks on the kernels of the tree decode (pd_tree.cu).
pd_status blocks_one_node(const void* q, const void* k_data, const void* v_data, const float* k_scale, const float* v_scale,
                          const int32_t* indices, const int32_t* indptr, const int32_t* last_page_len, void* o, float* lse,
                          int batch, int num_qo_heads, int num_kv_heads, int head_dim, int page_size, int num_total_pages,
                          int num_indices, int block_tokens, float sm_scale, pd_dtype dt, void* workspace,
                          size_t workspace_bytes, void* stream);
// pd_test_inject_wait_timeout's extra bytes (0: off).
int test_extra_tx();
// The driver's tensor-map encoder; null when the driver does not offer it.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool known_dtype(pd_dtype dt) { return dt == PD_F32 || dt == PD_F16 || dt == PD_BF16; }
inline size_t elem_size(pd_dtype dt) { return dt == PD_F32 ? 4 : 2; }

}  // namespace host
}  // namespace pd
