/*
 * pagedecode: batched single-query (decode-phase) grouped-query attention over
 * a paged KV cache, for NVIDIA sm_103a (GB300).
 *
 * The problem statement followed here is the module documentation of
 * baracuda-kernels 0.0.1-alpha.68, src/attention/batch_paged_decode.rs,
 * sections "Layout" and "Constraints", and its descriptor and argument types
 * (PagedKvCacheDescriptor, BatchPagedDecodeDescriptor, BatchPagedDecodeArgs):
 *
 *   k_data, v_data  [num_total_pages, num_kv_heads, page_size, head_dim]  T, HND
 *   indices         [num_indices]  int32  physical page ids
 *   indptr          [batch + 1]    int32  request b owns indices[indptr[b] .. indptr[b+1])
 *   last_page_len   [batch]        int32  valid rows in request b's last page, 0..page_size
 *   q, o            [batch, num_qo_heads, head_dim]  T
 *   lse             [batch, num_qo_heads]  float32 (whatever T is)
 *
 * For request b with np = indptr[b+1] - indptr[b] pages, kv_len = (np - 1) *
 * page_size + last_page_len[b] (0 when np = 0); token t is row t % page_size of
 * page indices[indptr[b] + t / page_size]. Query head h reads kv head
 * h / (num_qo_heads / num_kv_heads) (ferrox-cuda 0.15.2, src/attn.rs,
 * gqa_decode). With s_t = sm_scale * q[b,h,:] . k_t:
 *
 *   o[b,h,:]  = sum_t exp(s_t - lse) * v_t        lse[b,h] = ln sum_t exp(s_t)
 *
 * An empty request (kv_len = 0) gets o = 0 and lse = -infinity.
 *
 * Conventions shared by every call:
 *  - Pointers marked "device" are CUDA device pointers (or managed memory) on
 *    the current device; host pointers are marked "host". The caller owns
 *    every buffer, including the page table and its allocator; the library
 *    allocates no memory on any call.
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL is the legacy default
 *    stream). No call blocks the host except the two marked "synchronizes".
 *  - T is given by `dtype`: PD_F32 float, PD_F16 IEEE half, PD_BF16 bfloat16.
 *    Accumulation is float32 for every T. Results are bit-identical across
 *    repeated calls with the same arguments on the same device.
 *  - Arguments are checked on the host before anything is enqueued; a failed
 *    check returns an error status, enqueues nothing and sets the message
 *    returned by pd_last_error_string(). Values that live in device memory
 *    (page ids, indptr, last_page_len) are checked by the kernels: a bad
 *    value sets a bit of the sticky status word in the workspace header (see
 *    PD_FLAG_*), the offending page or request is treated as empty, and the
 *    kernel carries on. No kernel traps. A malformed indptr (decreasing,
 *    negative or past num_indices: PD_FLAG_BAD_INDPTR) makes request ranges
 *    overlap or run off the table, so it leaves every output of that call
 *    undefined, not only the flagged request's; the kernels still finish,
 *    and later calls with a good table are unaffected.
 *  - Status codes: PD_ERR_INVALID for malformed extents or null pointers,
 *    PD_ERR_UNSUPPORTED for a head_dim, dtype or pointer alignment this
 *    library does not handle, PD_ERR_WORKSPACE for a missing or small
 *    workspace, PD_ERR_CUDA when the CUDA runtime reports an error.
 */
#ifndef PAGEDECODE_H
#define PAGEDECODE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PD_VERSION 1

typedef enum { PD_F32 = 0, PD_F16 = 1, PD_BF16 = 2 } pd_dtype;

typedef enum {
    PD_OK = 0,
    PD_ERR_INVALID = 1,
    PD_ERR_UNSUPPORTED = 2,
    PD_ERR_WORKSPACE = 3,
    PD_ERR_CUDA = 4
} pd_status;

/* Bits of the sticky device status word (first int32 of every workspace). */
#define PD_FLAG_BAD_PAGE_ID 0x1       /* a page id outside [0, num_total_pages): page treated as empty */
#define PD_FLAG_BAD_LAST_PAGE_LEN 0x2 /* last_page_len outside [0, page_size]: clamped to that range */
#define PD_FLAG_BAD_INDPTR 0x4        /* indptr decreasing, negative or past num_indices: all outputs invalid */
#define PD_FLAG_WAIT_TIMEOUT 0x8      /* a copy pipeline wait passed its time limit; outputs invalid */
#define PD_FLAG_BAD_NEW_ROWS 0x10     /* new_indptr decreasing, outside [0, total_new], or more new rows than kv_len */
#define PD_FLAG_BAD_PATH 0x20         /* a path that does not increase, leaves the new rows or passes max_path */

/* Bytes at the start of every workspace that hold the status word and the
 * decode's work-distribution counters (zero between calls). */
#define PD_WORKSPACE_HEADER_BYTES 256

/*
 * Workspace bytes pd_paged_decode needs for this shape on the current device
 * (the split-KV partial results and the status word). Depends on the
 * device's SM count, so query it on the device that will run the call.
 * Returns 0 on a bad shape or when no device is present (see
 * pd_last_error_string()).
 */
size_t pd_paged_decode_workspace_bytes(int batch, int num_qo_heads, int num_kv_heads, int head_dim,
                                       pd_dtype dtype);

/*
 * Which decode kernel a call of this shape runs: one of PD_KERNEL_*. With
 * fp8_pool nonzero the question is about pd_paged_decode_fp8 (dtype is then
 * the type of q and o); otherwise about pd_paged_decode and the contiguous
 * calls, which share their kernels. The group g = num_qo_heads / num_kv_heads
 * is served in tiles of at most 8 q heads, padded to 1, 2, 4 or 8. 16-bit
 * tiles of 4 or 8 run on tensor cores; f32 and 16-bit tiles of 1 or 2 run on
 * CUDA cores. Over E4M3 pools, tiles of 4 or 8 at head_dim 128 or 256 run on
 * the mma.sync E4M3 tensor-core kernel, or, when pd_select_fp8_kernel chose
 * it and the shape allows it (bf16 q, groups of exactly 4 q heads, an even
 * number of kv heads, head_dim 128), on the tcgen05 kernel; the rest run on
 * CUDA cores. This is a host-side
 * lookup: it needs no device, enqueues nothing and returns PD_KERNEL_NONE for
 * a shape that no call accepts.
 */
#define PD_KERNEL_NONE 0
#define PD_KERNEL_CUDA_CORES 1
#define PD_KERNEL_TENSOR_CORES 2
#define PD_KERNEL_FP8_TENSOR_CORES 3
#define PD_KERNEL_FP8_TCGEN05 4
int pd_decode_kernel_kind(int num_qo_heads, int num_kv_heads, int head_dim, pd_dtype dtype, int fp8_pool);

/*
 * Which tensor-core kernel decodes over E4M3 pools where both apply (bf16 q,
 * groups of exactly 4 q heads, an even number of kv heads, head_dim 128):
 * PD_KERNEL_FP8_TENSOR_CORES (mma.sync over codes widened in registers; the
 * default, and the faster on the measured shapes) or PD_KERNEL_FP8_TCGEN05
 * (tcgen05.mma on the codes in shared memory, accumulators in tensor memory).
 * Both give results within the same tolerances. Process-wide; it applies to
 * the calls made after it returns, and to pd_decode_kernel_kind and the
 * workspace sizes (which may differ between the two). PD_ERR_INVALID for any
 * other value.
 */
pd_status pd_select_fp8_kernel(int kind);

/*
 * Batched paged decode (batch_paged_decode.rs: BatchPagedDecodePlan::run and
 * the per-dtype FFI launch it makes, whose argument order this follows).
 *
 * q, k_data, v_data, o: device, 16-byte aligned, layouts above. o (and lse)
 *   may also be pinned host memory (cudaHostAlloc / cudaMallocHost), which
 *   kernels reach at its host address under unified addressing: the kernels
 *   then store the results straight into host memory, with no copy back.
 * indices (may be NULL only if num_indices == 0), indptr, last_page_len: device int32.
 * lse: device float32 [batch, num_qo_heads], natural log.
 * head_dim: 64, 128 or 256. num_qo_heads % num_kv_heads == 0.
 * num_total_pages: pages in k_data/v_data. num_indices: entries in indices
 *   (the host-side length of the array; indptr[batch] must not exceed it).
 * sm_scale: the score scale, used as given (typically 1/sqrt(head_dim)).
 * workspace: device, 256-byte aligned, at least
 *   pd_paged_decode_workspace_bytes(...) bytes, its header zeroed once by
 *   pd_workspace_init() before first use. Calls that share a workspace must
 *   be ordered on one stream.
 *
 * Long requests are split across warps in a load-balanced partition of all
 * (kv head, page) work; the last part of each warp's share (a quarter of
 * shares of up to 1,024 K/V rows, an eighth of longer ones) goes, at fixed
 * boundaries, to whichever warp finishes first (counters in the workspace
 * header, back at zero after every call). Partial (o, lse) pairs are combined
 * by a merge kernel in a fixed order, so results do not depend on timing.
 */
pd_status pd_paged_decode(const void* q, const void* k_data, const void* v_data,
                          const int32_t* indices, const int32_t* indptr,
                          const int32_t* last_page_len, void* o, float* lse, int batch,
                          int num_qo_heads, int num_kv_heads, int head_dim, int page_size,
                          int num_total_pages, int num_indices, float sm_scale, pd_dtype dtype,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * Paged append (batch_paged_decode.rs, module doc "Companion plans":
 * PagedKvAppendPlan writes the new K/V slices into the paged store at decode
 * time; the caller owns the page table and its allocator).
 *
 * The caller first updates the page table for the new token: if request b's
 * last page is full (or it has no page) it appends a free page to its list
 * and sets last_page_len[b] = 1, otherwise it adds 1 to last_page_len[b].
 * This call then copies, bit for bit, k_new[b, h, :] and v_new[b, h, :] into
 * row last_page_len[b] - 1 of page indices[indptr[b+1] - 1], kv head h.
 *
 * k_new, v_new: device [batch, num_kv_heads, head_dim] T, 16-byte aligned.
 * k_data, v_data: device, modified in place. indices/indptr/last_page_len:
 *   device int32, the table after the caller's update.
 * workspace: device, at least PD_WORKSPACE_HEADER_BYTES bytes (the status
 *   word); a decode workspace may be shared.
 * A request with no page, a page id out of range or a last_page_len outside
 * [1, page_size] is skipped and flagged.
 */
pd_status pd_paged_append(const void* k_new, const void* v_new, void* k_data, void* v_data,
                          const int32_t* indices, const int32_t* indptr,
                          const int32_t* last_page_len, int batch, int num_kv_heads, int head_dim,
                          int page_size, int num_total_pages, int num_indices, pd_dtype dtype,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * FP8 KV pools. This is an extension of this library, not a layout of the
 * pages above: K and V pages hold one-byte E4M3 codes, in the same HND layout
 * as pd_paged_decode ([max_num_pages, num_kv_heads, page_size, head_dim]), and
 * element value = E4M3 value of the code * k_scale[h] (v_scale[h] for V), h
 * its kv head. E4M3 is the format of the OCP 8-bit floating point
 * specification (bias 7, 3 mantissa bits, S.1111.111 NaN, largest finite 448).
 * The pool is half the bytes of an f16 pool, and this decode is bound by
 * those bytes.
 *
 * pd_paged_decode_fp8: the arguments of pd_paged_decode plus k_scale, v_scale
 *   (device f32 [num_kv_heads], 4-byte aligned); dtype (PD_F16 or PD_BF16) is
 *   the type of q and o. The workspace size comes from
 *   pd_paged_decode_fp8_workspace_bytes (the stage geometry differs from the
 *   16-bit pools). Results, lse and errors as pd_paged_decode.
 * pd_paged_append_fp8: the slot of pd_paged_append receives, for each element
 *   x of k_new (v_new), the code of x / k_scale[h] (v_scale[h]): x widened to
 *   f32, the division in f32, rounded to the nearest code with ties to even,
 *   saturating at +-448 (NaN stays NaN). dtype is the type of k_new / v_new
 *   (PD_F16 or PD_BF16). Table errors as pd_paged_append.
 */
size_t pd_paged_decode_fp8_workspace_bytes(int batch, int num_qo_heads, int num_kv_heads, int head_dim,
                                           pd_dtype dtype);
pd_status pd_paged_decode_fp8(const void* q, const void* k_data, const void* v_data, const float* k_scale,
                              const float* v_scale, const int32_t* indices, const int32_t* indptr,
                              const int32_t* last_page_len, void* o, float* lse, int batch,
                              int num_qo_heads, int num_kv_heads, int head_dim, int page_size,
                              int num_total_pages, int num_indices, float sm_scale, pd_dtype dtype,
                              void* workspace, size_t workspace_bytes, void* stream);
pd_status pd_paged_append_fp8(const void* k_new, const void* v_new, const float* k_scale,
                              const float* v_scale, void* k_data, void* v_data, const int32_t* indices,
                              const int32_t* indptr, const int32_t* last_page_len, int batch,
                              int num_kv_heads, int head_dim, int page_size, int num_total_pages,
                              int num_indices, pd_dtype dtype, void* workspace, size_t workspace_bytes,
                              void* stream);

/*
 * Append, then decode, in one kernel launch. The companion plans of
 * batch_paged_decode.rs (module doc "Companion plans": PagedKvAppendPlan, then
 * BatchPagedDecodePlan) run as two plans per decode step; this call gives
 * exactly the result of pd_paged_append followed by pd_paged_decode on the
 * same arguments. That is, the K/V pool after the call is bit for bit the one
 * pd_paged_append leaves, and o / lse are those pd_paged_decode returns on it.
 *
 * Each decode warp whose chunk holds a request's new row (row
 * last_page_len[b] - 1 of its last page) first stores that row, then reads
 * the chunk. No other launch is made for the append, and no grid-wide barrier
 * is taken.
 *
 * Arguments are those of pd_paged_decode plus k_new, v_new (device
 * [batch, num_kv_heads, head_dim] T, 16-byte aligned); k_data and v_data are
 * modified in place, and the table must already describe the new token (as for
 * pd_paged_append). A request with no page, a bad last page id or a
 * last_page_len outside [1, page_size] is not appended to and is flagged in
 * the status word; the decode of the other requests is unaffected.
 */
pd_status pd_paged_append_decode(const void* q, const void* k_new, const void* v_new, void* k_data,
                                 void* v_data, const int32_t* indices, const int32_t* indptr,
                                 const int32_t* last_page_len, void* o, float* lse, int batch,
                                 int num_qo_heads, int num_kv_heads, int head_dim, int page_size,
                                 int num_total_pages, int num_indices, float sm_scale, pd_dtype dtype,
                                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * Append to a contiguous cache (batch_paged_decode.rs, module doc "Companion
 * plans": KvCacheAppendPlan, the append to a rank-4 cache with no page
 * table). For every request b and kv head h, row `position` of
 * k_cache[b, h, :, :] becomes k_new[b, h, :], bit for bit; the same for v.
 * With the cache holding `position` valid rows before the call, a decode
 * with valid_kv_len = position + 1 then sees the new token last.
 *
 * k_new, v_new: device [batch, num_kv_heads, head_dim] T, 16-byte aligned.
 * k_cache, v_cache: device [batch, num_kv_heads, max_kv_len, head_dim] T,
 *   modified in place. 0 <= position < max_kv_len (PD_ERR_INVALID otherwise).
 */
pd_status pd_contiguous_append(const void* k_new, const void* v_new, void* k_cache, void* v_cache, int batch,
                               int num_kv_heads, int head_dim, int max_kv_len, int position, pd_dtype dtype,
                               void* stream);

/*
 * pd_contiguous_append at `position`, then pd_contiguous_decode with
 * valid_kv_len = position + 1, in one launch (the contiguous-cache form of
 * pd_paged_append_decode). 0 <= position < max_kv_len (PD_ERR_INVALID
 * otherwise); k_cache, v_cache are modified in place; the workspace is that of
 * pd_contiguous_decode.
 */
pd_status pd_contiguous_append_decode(const void* q, const void* k_new, const void* v_new, void* k_cache,
                                      void* v_cache, void* o, float* lse, int batch, int num_qo_heads,
                                      int num_kv_heads, int head_dim, int max_kv_len, int position,
                                      float sm_scale, pd_dtype dtype, void* workspace,
                                      size_t workspace_bytes, void* stream);

/*
 * The token-major (NHD) contiguous cache. ferrox-cuda 0.15.2, src/attn.rs
 * (gqa_decode) stores one sequence as [seq_len, n_kv_heads, head_dim]: token t
 * of kv head h starts at element (t * n_kv_heads + h) * head_dim. These three
 * calls take that layout with a batch dimension in front,
 * k_cache / v_cache [batch, max_kv_len, num_kv_heads, head_dim], and are
 * otherwise the calls of the same name without _nhd: the same arguments,
 * results, workspace (pd_contiguous_decode_workspace_bytes) and errors.
 */
pd_status pd_contiguous_decode_nhd(const void* q, const void* k_cache, const void* v_cache, void* o,
                                   float* lse, int batch, int num_qo_heads, int num_kv_heads,
                                   int head_dim, int max_kv_len, int valid_kv_len, float sm_scale,
                                   pd_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);
pd_status pd_contiguous_append_nhd(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                                   int batch, int num_kv_heads, int head_dim, int max_kv_len,
                                   int position, pd_dtype dtype, void* stream);
pd_status pd_contiguous_append_decode_nhd(const void* q, const void* k_new, const void* v_new,
                                          void* k_cache, void* v_cache, void* o, float* lse, int batch,
                                          int num_qo_heads, int num_kv_heads, int head_dim,
                                          int max_kv_len, int position, float sm_scale, pd_dtype dtype,
                                          void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes pd_contiguous_decode needs (same rules as above). */
size_t pd_contiguous_decode_workspace_bytes(int batch, int num_qo_heads, int num_kv_heads,
                                            int head_dim, pd_dtype dtype);

/*
 * Decode over a contiguous cache (ferrum-kernels 0.7.7,
 * src/backend/cuda/decode_attention.rs, decode_attention: q [num_q_heads,
 * head_dim], k_cache/v_cache [num_kv_heads, max_kv_len, head_dim], rows
 * [0, valid_kv_len) valid, scale), with a leading batch dimension:
 *
 * q, o: device [batch, num_qo_heads, head_dim] T, 16-byte aligned.
 * k_cache, v_cache: device [batch, num_kv_heads, max_kv_len, head_dim] T.
 * lse: device float32 [batch, num_qo_heads] or NULL to skip it.
 * 0 <= valid_kv_len <= max_kv_len; valid_kv_len = 0 gives o = 0, lse = -inf.
 * The same kernels as pd_paged_decode run with each request's rows taken as
 * consecutive pages of one contiguous block.
 */
pd_status pd_contiguous_decode(const void* q, const void* k_cache, const void* v_cache, void* o,
                               float* lse, int batch, int num_qo_heads, int num_kv_heads,
                               int head_dim, int max_kv_len, int valid_kv_len, float sm_scale,
                               pd_dtype dtype, void* workspace, size_t workspace_bytes,
                               void* stream);

/*
 * Merge attention states computed over disjoint key sets of the same query
 * rows into the state over their union: lse = ln sum_c exp(lse_c),
 * o = sum_c exp(lse_c - lse) * o_c, parts taken in index order. This is the
 * combine step of the split-KV mode, exposed so that callers holding partial
 * results from elsewhere (another device, another cache tier) can use it.
 *
 * o_parts: device float32 [num_parts, num_rows, head_dim] (each part already
 *   normalised). lse_parts: device float32 [num_parts, num_rows], natural
 *   log, -inf for an empty part. o: device [num_rows, head_dim] T, 16-byte
 *   aligned. lse: device float32 [num_rows] or NULL. All parts empty gives
 *   o = 0, lse = -inf.
 */
pd_status pd_merge_states(const float* o_parts, const float* lse_parts, int num_parts,
                          int num_rows, int head_dim, void* o, float* lse, pd_dtype dtype,
                          void* stream);

/* Zero the status header of a workspace (enqueued on stream). */
pd_status pd_workspace_init(void* workspace, size_t workspace_bytes, void* stream);

/*
 * Read the sticky status word of a workspace into *flags (host). Synchronizes
 * `stream`. The word is not cleared; pd_workspace_init() clears it.
 */
pd_status pd_read_device_flags(const void* workspace, int32_t* flags, void* stream);

/*
 * Plain copy kernel (16-byte vector loads and stores, grid sized to the SM
 * count), used to measure the achievable HBM bandwidth in the same process as
 * the decode, and to bring a step's small inputs in from pinned host memory.
 * dst and src: device memory or pinned host memory (cudaHostAlloc /
 * cudaMallocHost, which kernels reach at its host address under unified
 * addressing), 16-byte aligned, not overlapping; bytes a multiple of 16.
 * Enqueued on stream; the caller keeps both buffers alive until it is done.
 */
pd_status pd_copy_bytes(void* dst, const void* src, size_t bytes, void* stream);

/*
 * Kernel timing for measurement. While enabled, every call records CUDA
 * events on its stream around each kernel it launches (decode, merge,
 * append). pd_profile_read() synchronizes on those events, returns the
 * summed milliseconds and launch counts per kind since the last read (host
 * pointers; any may be NULL), and starts a new count. Enabling costs two
 * event records per kernel; it is off by default.
 */
pd_status pd_profile_enable(int enable);

/*
 * Test-only failure injection for the bounded waits. While extra_bytes is
 * nonzero (a multiple of 16, at most 1 MiB), every decode call's first warp
 * waits, for its first pipeline stage, for extra_bytes more than its copies
 * deliver (the tensor-core tree decode: its first CTA, for its first copy). Its wait gives up after its limit (2 s), sets
 * PD_FLAG_WAIT_TIMEOUT in the status word, lets its other stages' copies
 * land, and returns; the outputs of the requests it held are then undefined,
 * and the GPU context stays usable. 0 (the default) turns it off.
 * Process-wide; not for use alongside other decode calls.
 */
pd_status pd_test_inject_wait_timeout(int extra_bytes);
pd_status pd_profile_read(double* decode_ms, int* decode_launches, double* merge_ms,
                          int* merge_launches, double* append_ms, int* append_launches);

/*
 * pd_paged_decode for callers that cannot allocate device memory at call
 * time (no counterpart on the pages: it is a deployment variant of the call
 * above). Typical callers: a plugin inside a host engine that owns all
 * device memory and passes its ops no scratch, or a serving loop that may
 * not call cudaMalloc on its hot path. Arguments are those of
 * pd_paged_decode without the workspace.
 *
 * The split-KV scratch lives in a 16 MiB static device array inside this
 * library, which every device that loads the library holds until the
 * process exits. A shape whose scratch (pd_paged_decode_workspace_bytes)
 * exceeds 16 MiB is rejected with PD_ERR_WORKSPACE before anything is
 * enqueued; the bundled workload shapes need at most ~13 MiB on a 148-SM
 * GB300. This call allocates nothing: no cudaMalloc, no cudaFree, no
 * allocating library routine.
 *
 * The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current; make that first call
 * before any stream capture. Each call that passes its argument checks
 * clears the array's status word and then runs the decode; a call rejected
 * by a check enqueues nothing. The kernels' device-side table checks set
 * PD_FLAG_* bits in that word, which pd_paged_decode_noalloc_flags reads.
 * All calls share one array, so calls whose kernels overlap on the GPU
 * (different streams, or different host threads) race on it: order them on
 * one stream.
 */
pd_status pd_paged_decode_noalloc(const void* q, const void* k_data, const void* v_data,
                                  const int32_t* indices, const int32_t* indptr,
                                  const int32_t* last_page_len, void* o, float* lse, int batch,
                                  int num_qo_heads, int num_kv_heads, int head_dim, int page_size,
                                  int num_total_pages, int num_indices, float sm_scale,
                                  pd_dtype dtype, void* stream);

/*
 * The status word of pd_paged_decode_noalloc's built-in scratch on the
 * current device, read into *flags (host): the PD_FLAG_* bits that the last
 * pd_paged_decode_noalloc call enqueued before this one set (a bad page id,
 * last_page_len or indptr; a wait that ran out, after which the outputs are
 * invalid). Synchronizes `stream`: enqueue it after that call, on the same
 * stream. Allocates nothing. The word is cleared by the next noalloc call.
 */
pd_status pd_paged_decode_noalloc_flags(int32_t* flags, void* stream);

/*
 * Speculative decoding. The four groups of calls below are an extension of
 * this library, not calls of the pages above. A step with drafted tokens
 * rotates q and k and appends k and v (pd_paged_rope_append), attends for all
 * drafted tokens at once (pd_paged_tree_decode), and keeps the accepted ones
 * (pd_paged_tree_commit). A prompt, or a piece of one, goes through the first
 * two as a chain.
 *
 * New rows. Request b's new tokens are rows new_indptr[b] .. new_indptr[b+1]
 * of the ragged tensors (new_indptr: device int32 [batch + 1], increasing from
 * 0 to total_new), n_b of them, and are the LAST n_b tokens of its cache: the
 * page table already describes them (the caller's update for n_b tokens).
 * n_b may be 0, and total_new too (the rows' pointers may then be NULL). A
 * malformed new_indptr, or n_b > kv_len, is flagged with PD_FLAG_BAD_NEW_ROWS
 * and that request's rows are not written to the pool. last_page_len may be 0
 * (an allocated page that is still empty; the new tokens end in the page
 * before it). Outside [0, page_size] it is flagged with
 * PD_FLAG_BAD_LAST_PAGE_LEN: the append and the commit, which write, skip the
 * request; the tree decode clamps it, as the decode does.
 */

/*
 * Rotary positions. Pair i of a head at position p turns by the angle p f_i:
 *
 *   (a, b)  ->  rope_scale * (a cos - b sin, b cos + a sin)
 *
 * for the pairs of the leading rot_dim elements: (i, i + rot_dim / 2) with
 * PD_ROPE_HALF, (2i, 2i + 1) with PD_ROPE_PAIRS. Elements from rot_dim on are
 * copied. Arithmetic is f32, rounded once to T. Positions are int32 and may be
 * negative: rotating by -p undoes rotating by p, and is also the gradient of
 * pd_rope (of the same rope_scale).
 *
 * freqs: device uint64 [rot_dim / 2], 8-byte aligned: f_i in turns (2 pi
 * radians) per position, as a binary fraction, floor(f_i / (2 pi) * 2^64) for
 * f_i in radians. The angle modulo one turn is then exact at any position.
 */
#define PD_ROPE_HALF 0
#define PD_ROPE_PAIRS 1

/*
 * Fill freqs (HOST memory, rot_dim / 2 entries; the caller copies it to the
 * device) and *rope_scale (host). With f_i = theta^(-2i / rot_dim):
 *  PD_ROPE_PLAIN   f_i
 *  PD_ROPE_LINEAR  f_i / factor
 *  PD_ROPE_BASE    theta replaced by theta * factor^(rot_dim / (rot_dim - 2))
 *  PD_ROPE_BANDED  k f_i + (1 - k) f_i / factor, k = clamp((turns - low) /
 *                  (high - low), 0, 1), turns = original_positions f_i / 2 pi
 *  PD_ROPE_YARN    the same with k falling linearly over the pair index, from
 *                  1 at the (floored) index that makes `high` turns over
 *                  original_positions to 0 at the (ceiled) one that makes
 *                  `low`; rope_scale = 0.1 ln(factor) + 1 (1 for the others)
 * factor >= 1 (ignored by PLAIN); 0 < low < high and original_positions > 0
 * for BANDED and YARN (ignored by the others). Needs no device.
 */
#define PD_ROPE_PLAIN 0
#define PD_ROPE_LINEAR 1
#define PD_ROPE_BASE 2
#define PD_ROPE_BANDED 3
#define PD_ROPE_YARN 4
pd_status pd_rope_frequencies(uint64_t* freqs, float* rope_scale, int rot_dim, double theta, int scaling,
                              double factor, double low, double high, int original_positions);

/*
 * Rotate num_tokens tokens. x, out: device T; head h of token t is the
 * head_dim elements at t * stride + h * head_dim (strides in elements, at
 * least num_heads * head_dim: a token's heads are contiguous, tokens may be
 * slices of a wider row). out may be x (the same stride), and must not
 * otherwise overlap it. Elements between the tokens of out are left alone.
 * positions: device int32 [num_tokens]. rot_dim even, 0 .. head_dim; head_dim
 * up to 4096. 16-byte accesses where x, out and their strides allow it and
 * rot_dim is a multiple of 16 (f32: 8); single elements otherwise.
 */
pd_status pd_rope(const void* x, const int32_t* positions, const uint64_t* freqs, void* out, int num_tokens,
                  int num_heads, int head_dim, int rot_dim, int64_t x_stride, int64_t out_stride, int layout,
                  float rope_scale, pd_dtype dtype, void* stream);

/*
 * Append n_b new tokens to every request, with the rotation on the way: row
 * kv_len - n_b + j of request b's cache becomes the rotated k_new row (K pool)
 * and, bit for bit, the v_new row (V pool) of its new token j; q_out receives
 * the rotated q rows.
 *
 * q: device [total_new] tokens of num_qo_heads heads, q_stride elements apart;
 *   q_out: device [total_new, num_qo_heads, head_dim], may be q if q is laid
 *   out so (refused otherwise), and must not otherwise overlap it.
 *   num_qo_heads = 0 leaves q out (q, q_out may be NULL).
 * k_new, v_new: device [total_new] tokens of num_kv_heads heads, k_stride and
 *   v_stride elements apart. q, k_new and v_new may be views of one tensor.
 * positions: device int32 [total_new], or NULL for each token's index in its
 *   cache. A tree's nodes sit at positions given by their depth, not by their
 *   row: give them.
 * rot_dim = 0 (freqs may be NULL) appends without rotation.
 * k_data, v_data: device, 16-byte aligned, modified in place. No two requests
 *   may own the page that a new row falls in.
 * workspace: at least PD_WORKSPACE_HEADER_BYTES (the status word).
 * A new row whose request or page is bad is flagged and not written; its q
 * row is still rotated when positions are given, and undefined otherwise.
 *
 * The _fp8 form writes E4M3 codes of the rotated k / k_scale[h] and of v /
 * v_scale[h] (the f32 values, divided in f32, rounded once to the nearest
 * code, ties to even, saturating at +-448). dtype PD_F16 or PD_BF16.
 */
pd_status pd_paged_rope_append(const void* q, const void* k_new, const void* v_new, const int32_t* positions,
                               const uint64_t* freqs, void* q_out, void* k_data, void* v_data, const int32_t* indices,
                               const int32_t* indptr, const int32_t* last_page_len, const int32_t* new_indptr,
                               int batch, int total_new, int num_qo_heads, int num_kv_heads, int head_dim, int rot_dim,
                               int page_size, int num_total_pages, int num_indices, int64_t q_stride, int64_t k_stride,
                               int64_t v_stride, int layout, float rope_scale, pd_dtype dtype, void* workspace,
                               size_t workspace_bytes, void* stream);
pd_status pd_paged_rope_append_fp8(const void* q, const void* k_new, const void* v_new, const int32_t* positions,
                                   const uint64_t* freqs, void* q_out, const float* k_scale, const float* v_scale,
                                   void* k_data, void* v_data, const int32_t* indices, const int32_t* indptr,
                                   const int32_t* last_page_len, const int32_t* new_indptr, int batch, int total_new,
                                   int num_qo_heads, int num_kv_heads, int head_dim, int rot_dim, int page_size,
                                   int num_total_pages, int num_indices, int64_t q_stride, int64_t k_stride,
                                   int64_t v_stride, int layout, float rope_scale, pd_dtype dtype, void* workspace,
                                   size_t workspace_bytes, void* stream);

/*
 * Attention of every request's new tokens (its nodes) over its cache, their
 * own rows among it. Node j of request b attends every one of the first
 * kv_len - n_b tokens, and node i of the request iff bit i % 32 of
 * tree_mask[new_indptr[b] + j][i / 32] is set (a node sees itself only if its
 * own bit is set; bits from 32 * mask_words on count as clear). tree_mask =
 * NULL is a chain: node j attends nodes 0 .. j. With s_t = sm_scale * q . k_t
 * over the attended tokens,
 *
 *   o = sum_t exp(s_t - lse) v_t        lse = ln sum_t exp(s_t)
 *
 * and a node that attends nothing gets o = 0, lse = -infinity. Tokens that a
 * node does not attend have no part in its result, whatever they hold (NaN and
 * infinities included). A NaN among a node's scores makes its o and lse NaN.
 *
 * q, o: device [total_new, num_qo_heads, head_dim] T, 16-byte aligned.
 * tree_mask: device uint32 [total_new, mask_words], or NULL.
 * lse: device float32 [total_new, num_qo_heads].
 * The rest is as for pd_paged_decode. workspace: at least
 * pd_paged_tree_decode_workspace_bytes(...) bytes, header zeroed once; it may
 * be shared with the other calls on the same stream. Results do not depend on
 * timing: the work is cut at fixed places and merged in a fixed order.
 * A node of a bad request (bad indptr, or n_b > kv_len) attends nothing.
 *
 * 16-bit q runs on the tensor cores (tcgen05) for groups of up to 128 q heads;
 * f32, and larger groups, on CUDA cores. Weights are rounded to T before they
 * meet V, sums are f32.
 * The _fp8 form reads E4M3 pools as pd_paged_decode_fp8 does (dtype PD_F16 or
 * PD_BF16 is the type of q and o).
 */
size_t pd_paged_tree_decode_workspace_bytes(int num_qo_heads, int num_kv_heads, int head_dim, pd_dtype dtype);
pd_status pd_paged_tree_decode(const void* q, const void* k_data, const void* v_data, const int32_t* indices,
                               const int32_t* indptr, const int32_t* last_page_len, const int32_t* new_indptr,
                               const uint32_t* tree_mask, void* o, float* lse, int batch, int total_new,
                               int mask_words, int num_qo_heads, int num_kv_heads, int head_dim, int page_size,
                               int num_total_pages, int num_indices, float sm_scale, pd_dtype dtype, void* workspace,
                               size_t workspace_bytes, void* stream);
pd_status pd_paged_tree_decode_fp8(const void* q, const void* k_data, const void* v_data, const float* k_scale,
                                   const float* v_scale, const int32_t* indices, const int32_t* indptr,
                                   const int32_t* last_page_len, const int32_t* new_indptr, const uint32_t* tree_mask,
                                   void* o, float* lse, int batch, int total_new, int mask_words, int num_qo_heads,
                                   int num_kv_heads, int head_dim, int page_size, int num_total_pages, int num_indices,
                                   float sm_scale, pd_dtype dtype, void* workspace, size_t workspace_bytes,
                                   void* stream);

/*
 * Keep the accepted nodes: for i < path_len[b], the K and V rows of node
 * path[b][i] move, bit for bit, to the place of node i. A path increases
 * strictly (a parent comes before its child); node i = path[b][i] stays where
 * it is. The caller then shortens the request to kv_len - n_b + path_len[b]
 * tokens. Rows of the new tokens past path_len[b] are left as they fall.
 *
 * path: device int32 [batch, max_path]; path_len: device int32 [batch], 0 ..
 * max_path. elem_bytes: 1 (E4M3 pools), 2 or 4. workspace as for
 * pd_paged_rope_append. The table is the one of the tree decode. A request
 * with a bad path or table is flagged and left as it is. Not for block-scaled
 * pools (below), which this call cannot tell from other E4M3 pools: a code is
 * another value under another block's scale. There the accepted nodes' rows are
 * appended again (see pd_paged_rope_append_fp8_blocks).
 */
pd_status pd_paged_tree_commit(void* k_data, void* v_data, const int32_t* indices, const int32_t* indptr,
                               const int32_t* last_page_len, const int32_t* new_indptr, const int32_t* path,
                               const int32_t* path_len, int batch, int total_new, int max_path, int num_kv_heads,
                               int head_dim, int page_size, int num_total_pages, int num_indices, int elem_bytes,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * Norms of q and k heads with the rotation in the same pass. An extension of
 * this library, like the calls above. Each head x becomes
 *
 *   x / sqrt(mean(x^2) + eps) * w        (w: q_weight for q, k_weight for k)
 *
 * over its head_dim elements, and its leading rot_dim elements then turn as in
 * pd_rope. Arithmetic is f32, rounded once to T.
 *
 * q_weight, k_weight: device T [head_dim], or NULL for ones. eps > 0.
 *
 * pd_norm_rope: q, q_out: device T [num_tokens] tokens of num_qo_heads heads;
 *   k, k_out: the same of num_kv_heads heads (0 leaves k out: k, k_out may be
 *   NULL). Strides between tokens in elements, as in pd_rope; q_out may be q,
 *   and k_out k (the same stride); outputs must not otherwise overlap inputs
 *   or each other. positions: device int32 [num_tokens] (may be NULL where
 *   rot_dim is 0). head_dim even, up to 256. 16-byte accesses where every row
 *   and stride allows it and rot_dim and head_dim are multiples of 16 (f32: 8);
 *   single elements otherwise.
 * pd_paged_norm_rope_append, _fp8: pd_paged_rope_append and its _fp8 form with
 *   the norms in front. Arguments, results and errors as there.
 */
pd_status pd_norm_rope(const void* q, const void* k, const void* q_weight, const void* k_weight, const int32_t* positions,
                       const uint64_t* freqs, void* q_out, void* k_out, int num_tokens, int num_qo_heads,
                       int num_kv_heads, int head_dim, int rot_dim, int64_t q_stride, int64_t k_stride,
                       int64_t q_out_stride, int64_t k_out_stride, float eps, int layout, float rope_scale,
                       pd_dtype dtype, void* stream);
pd_status pd_paged_norm_rope_append(const void* q, const void* k_new, const void* v_new, const void* q_weight,
                                    const void* k_weight, const int32_t* positions, const uint64_t* freqs, void* q_out,
                                    void* k_data, void* v_data, const int32_t* indices, const int32_t* indptr,
                                    const int32_t* last_page_len, const int32_t* new_indptr, int batch, int total_new,
                                    int num_qo_heads, int num_kv_heads, int head_dim, int rot_dim, int page_size,
                                    int num_total_pages, int num_indices, int64_t q_stride, int64_t k_stride,
                                    int64_t v_stride, float eps, int layout, float rope_scale, pd_dtype dtype,
                                    void* workspace, size_t workspace_bytes, void* stream);
pd_status pd_paged_norm_rope_append_fp8(const void* q, const void* k_new, const void* v_new, const void* q_weight,
                                        const void* k_weight, const int32_t* positions, const uint64_t* freqs,
                                        void* q_out, const float* k_scale, const float* v_scale, void* k_data,
                                        void* v_data, const int32_t* indices, const int32_t* indptr,
                                        const int32_t* last_page_len, const int32_t* new_indptr, int batch,
                                        int total_new, int num_qo_heads, int num_kv_heads, int head_dim, int rot_dim,
                                        int page_size, int num_total_pages, int num_indices, int64_t q_stride,
                                        int64_t k_stride, int64_t v_stride, float eps, int layout, float rope_scale,
                                        pd_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Block-scaled pools. E4M3 codes in the layout of the E4M3 pools above, with
 * one f32 scale for each block of block_tokens consecutive rows of a page and
 * kv head instead of one per kv head:
 *
 *   k_data, v_data    [num_total_pages, num_kv_heads, page_size, head_dim]  codes
 *   k_scale, v_scale  [num_total_pages, num_kv_heads, page_size / block_tokens]  f32
 *   element value = E4M3 value of the code * the scale of its row's block
 *
 * block_tokens in [1, PD_MAX_BLOCK_TOKENS], a divisor of page_size: a scale for
 * each token (1), or one per page and head (page_size). The scales follow the
 * data: the append chooses them. They are finite and not negative. Scales of rows
 * past a request's end are not read.
 *
 * pd_paged_rope_append_fp8_blocks: pd_paged_rope_append (its arguments,
 *   results, and errors) into such pools, with the norms of pd_norm_rope in
 *   front where eps > 0; eps = 0 leaves them out (q_weight and
 *   k_weight are then NULL). dtype PD_F16 or PD_BF16. Let a be the largest
 *   finite magnitude, after norm and rotation in f32, of the new elements of a
 *   block. A new_indptr that does not run from 0 to total_new without decreasing
 *   is flagged (PD_FLAG_BAD_NEW_ROWS).
 *    - A block whose first row is new gets the scale a / 448, at least 2^-126.
 *    - A block that also holds older rows of the request keeps its scale s
 *      (at least 2^-126) if a <= 464 s (what still rounds to the largest code).
 *      Otherwise s doubles until that holds, and the codes of the older rows
 *      are rounded again, by that power of two: exactly, but for subnormals.
 *   A new element x is written as the code nearest to x * (1 / s), both
 *   operations in f32, ties to even, saturating at +-448 (infinities too; NaN
 *   stays NaN). Rows past the request's end keep their codes; a page may be
 *   shared with another request where no new row falls into it.
 *
 *   After a step with drafted tokens the accepted ones are kept by a second
 *   call: the table with the request's length shortened to its context and the
 *   accepted nodes, and the accepted nodes' rows of k_new and v_new as the new
 *   rows (num_qo_heads = 0), positions as before or NULL (a path's depths are
 *   its indices). An accepted prefix of a chain is kept by shortening alone.
 *   The scale of the block that the context ends in stays what the drafted rows
 *   made it.
 *
 * pd_paged_read_fp8_blocks: the values of tokens first[b] .. first[b] + n_b - 1
 *   of request b (f32 products, rounded to T) in rows out_indptr[b] .. of k_out and
 *   v_out (device T [total, num_kv_heads, head_dim], 16-byte aligned), n_b =
 *   out_indptr[b + 1] - out_indptr[b] (device int32 [batch + 1], not decreasing,
 *   within 0 .. total; n_b may be 0). Rows before out_indptr[0] and from
 *   out_indptr[batch] on stay as they are. first: device int32 [batch], or NULL
 *   for 0. dtype: any T. Tokens outside the request, or a malformed out_indptr:
 *   PD_FLAG_BAD_NEW_ROWS, and that request's rows are not written. Rows on a
 *   bad page are zero (PD_FLAG_BAD_PAGE_ID).
 *
 * pd_paged_decode_fp8_blocks: pd_paged_decode over such pools: one query row
 *   per request, which attends all of its cached tokens. An empty request gets
 *   o = 0, lse = -infinity. A NaN among a row's scores makes its o and lse NaN.
 * pd_paged_tree_decode_fp8_blocks: pd_paged_tree_decode over such pools.
 *   Both: dtype (PD_F16 or PD_BF16) is the type of q and o. Scores, maxima, sums
 *   and outputs are f32 until the last rounding; a weight times its V scale is
 *   rounded to f16 before it meets the codes, and for bf16 outputs of few rows to
 *   9 significant bits. An f16 output so has a fifth to a third more error than
 *   its own rounding. V scales below 2^-88 lose precision by how far they are below it.
 *   One kernel is chosen for the whole call, by the mean number of rows of a
 *   request: a prompt piece beside many single tokens runs faster in a call of
 *   its own.
 *   workspace: at least
 *   the bytes that the call's _workspace_bytes gives, which any other call on
 *   the same stream may share. The other arguments, results and errors
 *   are those of pd_paged_decode and pd_paged_tree_decode.
 */
#define PD_MAX_BLOCK_TOKENS 64
pd_status pd_paged_rope_append_fp8_blocks(const void* q, const void* k_new, const void* v_new, const void* q_weight,
                                          const void* k_weight, const int32_t* positions, const uint64_t* freqs,
                                          void* q_out, float* k_scale, float* v_scale, void* k_data, void* v_data,
                                          const int32_t* indices, const int32_t* indptr, const int32_t* last_page_len,
                                          const int32_t* new_indptr, int batch, int total_new, int num_qo_heads,
                                          int num_kv_heads, int head_dim, int rot_dim, int page_size,
                                          int num_total_pages, int num_indices, int block_tokens, int64_t q_stride,
                                          int64_t k_stride, int64_t v_stride, float eps, int layout, float rope_scale,
                                          pd_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);
pd_status pd_paged_read_fp8_blocks(const void* k_data, const void* v_data, const float* k_scale, const float* v_scale,
                                   const int32_t* indices, const int32_t* indptr, const int32_t* last_page_len,
                                   const int32_t* out_indptr, const int32_t* first, void* k_out, void* v_out, int batch,
                                   int total, int num_kv_heads, int head_dim, int page_size, int num_total_pages,
                                   int num_indices, int block_tokens, pd_dtype dtype, void* workspace,
                                   size_t workspace_bytes, void* stream);
size_t pd_paged_decode_fp8_blocks_workspace_bytes(int batch, int num_qo_heads, int num_kv_heads, int head_dim,
                                                  pd_dtype dtype);
size_t pd_paged_tree_decode_fp8_blocks_workspace_bytes(int num_qo_heads, int num_kv_heads, int head_dim, pd_dtype dtype);
pd_status pd_paged_decode_fp8_blocks(const void* q, const void* k_data, const void* v_data, const float* k_scale,
                                     const float* v_scale, const int32_t* indices, const int32_t* indptr,
                                     const int32_t* last_page_len, void* o, float* lse, int batch, int num_qo_heads,
                                     int num_kv_heads, int head_dim, int page_size, int num_total_pages,
                                     int num_indices, int block_tokens, float sm_scale, pd_dtype dtype, void* workspace,
                                     size_t workspace_bytes, void* stream);
pd_status pd_paged_tree_decode_fp8_blocks(const void* q, const void* k_data, const void* v_data, const float* k_scale,
                                          const float* v_scale, const int32_t* indices, const int32_t* indptr,
                                          const int32_t* last_page_len, const int32_t* new_indptr,
                                          const uint32_t* tree_mask, void* o, float* lse, int batch, int total_new,
                                          int mask_words, int num_qo_heads, int num_kv_heads, int head_dim,
                                          int page_size, int num_total_pages, int num_indices, int block_tokens,
                                          float sm_scale, pd_dtype dtype, void* workspace, size_t workspace_bytes,
                                          void* stream);

/* Message for the last error status returned on this host thread ("" if none). */
const char* pd_last_error_string(void);

/* PD_VERSION of the built library. */
int pd_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDECODE_H */
