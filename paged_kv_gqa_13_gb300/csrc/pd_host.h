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
// pd_test_inject_wait_timeout's extra bytes (0: off).
int test_extra_tx();
// The driver's tensor-map encoder; null when the driver does not offer it.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool known_dtype(pd_dtype dt) { return dt == PD_F32 || dt == PD_F16 || dt == PD_BF16; }
inline size_t elem_size(pd_dtype dt) { return dt == PD_F32 ? 4 : 2; }

}  // namespace host
}  // namespace pd
