// Tree decode: argument checks, the choice of kernel, launches.
#include <cmath>
#include <type_traits>

#include "pd_host.h"
#include "pd_tree.cuh"
#include "pd_tree_kernels.h"

namespace pd {
namespace {

template <typename T, typename KV, int D, int kCols>
TreeKernels cc_kernels() {
    using C = CfgTreeCc<D, kCols>;
    TreeKernels k{};
    k.main = reinterpret_cast<const void*>(tree_cc_kernel<T, KV, D, kCols>);
    k.merge = reinterpret_cast<const void*>(tree_merge_kernel<T, D>);
    k.threads = C::kThreads;
    k.smem = C::kBytes;
    k.per_sm = C::kBlocksPerSm;
    k.tile_rows = C::kRows;
    k.tiles = 1;
    k.workers = 1;
    k.block_tokens = C::kBlockTokens;
    return k;
}

template <typename T, typename KV, int kCols>
bool cc_by_dim(int D, TreeKernels* k) {
    switch (D) {
        case 64: *k = cc_kernels<T, KV, 64, (kCols < 16 ? kCols : 16)>(); return true;
        case 128: *k = cc_kernels<T, KV, 128, kCols>(); return true;
        case 256: *k = cc_kernels<T, KV, 256, kCols>(); return true;
    }
    return false;
}

// The rows of a request on average: up to 8, up to 16, up to half a row tile of the tensor cores, more.
enum Rows { kRows8, kRows16, kRows64, kRowsMany };

// 16-bit q of a group that fits a row tile runs on the tensor cores; f32 q,
// which no tensor-core type holds, and larger groups on CUDA cores.
bool pick(pd_dtype dt, bool fp8, int D, int group, Rows rows, TreeKernels* k) {
    if (dt != PD_F32 && group <= 128) {
        const bool wide = rows == kRowsMany;  // two row tiles per segment (where a kernel for it exists)
        if (fp8) return dt == PD_F16 ? tree_tc_f16_fp8(D, wide, k) : tree_tc_bf16_fp8(D, wide, k);
        return dt == PD_F16 ? tree_tc_f16(D, wide, k) : tree_tc_bf16(D, wide, k);
    }
    switch (dt) {
        case PD_F32:
            if (fp8) return false;
            return rows == kRows8    ? cc_by_dim<float, float, 32>(D, k)
                   : rows == kRows16 ? cc_by_dim<float, float, 16>(D, k)
                                     : cc_by_dim<float, float, 8>(D, k);
        case PD_F16: return fp8 ? cc_by_dim<__half, uint8_t, 8>(D, k) : cc_by_dim<__half, __half, 8>(D, k);
        case PD_BF16:
            return fp8 ? cc_by_dim<__nv_bfloat16, uint8_t, 8>(D, k) : cc_by_dim<__nv_bfloat16, __nv_bfloat16, 8>(D, k);
    }
    return false;
}

pd_status encode(CUtensorMap* map, CUtensorMapDataType ty, int rank, const void* base, const cuuint64_t* dims,
                 const cuuint64_t* strides, const cuuint32_t* box) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = host::tensor_map_encoder();
    if (enc == nullptr) return host::fail(PD_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    const CUtensorMapSwizzle swizzle = ty == CU_TENSOR_MAP_DATA_TYPE_UINT8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
    const CUresult r = enc(map, ty, cuuint32_t(rank), const_cast<void*>(base), dims, strides, box, ones,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PD_OK : host::fail(PD_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", int(r));
}

// Boxes: of q {64 columns, heads of a tile, nodes of a row tile}; of K and V {64
// columns, rows of a slot}, of codes {head_dim columns, rows of a slot}.
pd_status make_maps(const TreeArgs& a, pd_dtype dt, bool fp8, int D, CUtensorMap* q, CUtensorMap* k, CUtensorMap* v) {
    const CUtensorMapDataType qt = dt == PD_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUtensorMapDataType kt = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : qt;
    const cuuint64_t d = cuuint64_t(D), ps = cuuint64_t(a.page_size), hk = cuuint64_t(a.num_kv_heads),
                     hq = cuuint64_t(a.num_qo_heads), e = fp8 ? 1 : 2;
    const cuuint64_t kd[4] = {d, ps, hk, cuuint64_t(a.num_total_pages)}, ks[3] = {d * e, ps * d * e, hk * ps * d * e};
    const cuuint32_t kb[4] = {fp8 ? cuuint32_t(D) : 64u, 1u << a.slot_shift, 1, 1};
    pd_status st = encode(k, kt, 4, a.k, kd, ks, kb);
    if (st == PD_OK) st = encode(v, kt, 4, a.v, kd, ks, kb);
    if (st != PD_OK) return st;
    const cuuint64_t qd[3] = {d, hq, cuuint64_t(a.total_new)}, qs[2] = {d * 2, hq * d * 2};
    const cuuint32_t qb[3] = {64, cuuint32_t(a.hpt), cuuint32_t(a.npt)};
    return encode(q, qt, 3, a.q, qd, qs, qb);
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// Workspace: header | split descriptors | partial lse | partial o, for a grid of `ctas`.
constexpr size_t kClaimsOff = 128;  // of TreeArgs::claims in the workspace header

struct TreeSpace {
    size_t splits, lse, o, bytes;
};
TreeSpace space(const TreeKernels& k, int ctas, int D) {
    TreeSpace s;
    const size_t ranges = size_t(2) * ctas * k.workers, rows = 2 * ranges * k.tile_rows * k.tiles;
    s.splits = PD_WORKSPACE_HEADER_BYTES;
    s.lse = s.splits + round256((ranges + 1) * sizeof(TreeSplit));
    s.o = s.lse + round256(rows * 4);
    s.bytes = s.o + rows * D * 4;
    return s;
}

pd_status check_heads(int Hq, int Hk, int D, pd_dtype dt) {
    if (!host::known_dtype(dt)) return host::fail(PD_ERR_UNSUPPORTED, "dtype must be PD_F32, PD_F16 or PD_BF16");
    if (Hq <= 0 || Hk <= 0) return host::fail(PD_ERR_INVALID, "num_qo_heads and num_kv_heads must be positive");
    if (Hq % Hk != 0) return host::fail(PD_ERR_INVALID, "num_qo_heads (%d) must be a multiple of num_kv_heads (%d)", Hq, Hk);
    if (D != 64 && D != 128 && D != 256) return host::fail(PD_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256 (got %d)", D);
    return PD_OK;
}

pd_status tree_impl(const void* q, const void* k_data, const void* v_data, const float* k_scale, const float* v_scale,
                    const int32_t* indices, const int32_t* indptr, const int32_t* last_page_len,
                    const int32_t* new_indptr, const uint32_t* tree_mask, void* o, float* lse, int batch, int total_new,
                    int mask_words, int Hq, int Hk, int D, int page_size, int num_total_pages, int num_indices,
                    float sm_scale, pd_dtype dt, void* workspace, size_t workspace_bytes, void* stream, bool fp8) {
    pd_status st = check_heads(Hq, Hk, D, dt);
    if (st != PD_OK) return st;
    if (fp8 && dt == PD_F32) return host::fail(PD_ERR_UNSUPPORTED, "E4M3 pools take PD_F16 or PD_BF16 q and o");
    if (batch <= 0 || page_size <= 0 || num_total_pages <= 0)
        return host::fail(PD_ERR_INVALID, "batch, page_size and num_total_pages must be positive");
    if (total_new < 0 || num_indices < 0) return host::fail(PD_ERR_INVALID, "total_new and num_indices must not be negative");
    if (total_new > (1 << 30) || Hq > (1 << 20)) return host::fail(PD_ERR_INVALID, "at most 2^30 new rows and 2^20 heads");
    if (tree_mask ? mask_words <= 0 : mask_words < 0 || (mask_words != 0 && total_new > 0))
        return host::fail(PD_ERR_INVALID, "mask_words must be positive with a tree_mask and 0 without (got %d)", mask_words);
    if (!std::isfinite(sm_scale)) return host::fail(PD_ERR_INVALID, "sm_scale must be finite");
    if (!k_data || !v_data || !indptr || !last_page_len || !new_indptr || (num_indices > 0 && !indices) ||
        (total_new > 0 && (!q || !o || !lse)) || (fp8 && (!k_scale || !v_scale)))
        return host::fail(PD_ERR_INVALID, "null pointer argument");
    if (!host::aligned(q, 16) || !host::aligned(k_data, 16) || !host::aligned(v_data, 16) || !host::aligned(o, 16))
        return host::fail(PD_ERR_UNSUPPORTED, "q, k_data, v_data and o must be 16-byte aligned");
    if (!host::aligned(lse, 4) || !host::aligned(indices, 4) || !host::aligned(indptr, 4) ||
        !host::aligned(last_page_len, 4) || !host::aligned(new_indptr, 4) || !host::aligned(tree_mask, 4) ||
        !host::aligned(k_scale, 4) || !host::aligned(v_scale, 4))
        return host::fail(PD_ERR_UNSUPPORTED, "lse, the table, tree_mask and the scales must be 4-byte aligned");
    const int group = Hq / Hk;
    TreeKernels kn{};
    // On the tensor cores, more than half a row tile per request on average: segments of up to two row tiles, which
    // read K and V once for both (64 trees of 1 to 32 nodes, 8 heads a group: 191 us as two halves of a CTA, 162 so).
    // Fewer: two independent halves of each CTA (32 chains of 4, 4 heads a group: 93 us as two row tiles, 68 so). On
    // CUDA cores, row tiles of 32, of 16 or of 8 rows (16 requests, 16 rows of head_dim 64: 104 us in 32, 72 in 16).
    const long long all_rows = (long long)total_new * group;
    const Rows rows = all_rows > 64ll * batch   ? kRowsMany
                      : all_rows > 16ll * batch ? kRows64
                      : all_rows > 8ll * batch  ? kRows16
                                                : kRows8;
    if (!pick(dt, fp8, D, group, rows, &kn)) return host::fail(PD_ERR_UNSUPPORTED, "no kernel for this type and head_dim");
    int sms = 0;
    if ((st = host::sm_count(&sms)) != PD_OK) return st;
    const int most = sms * kn.per_sm;
    const TreeSpace sp = space(kn, most, D);
    if ((st = host::check_workspace(workspace, workspace_bytes, sp.bytes)) != PD_OK) return st;
    if (total_new == 0) return host::ok();

    uint8_t* ws = static_cast<uint8_t*>(workspace);
    TreeArgs a{};
    a.q = q;
    a.k = k_data;
    a.v = v_data;
    a.indices = indices;
    a.indptr = indptr;
    a.last_page_len = last_page_len;
    a.new_indptr = new_indptr;
    a.mask = tree_mask;
    a.o = o;
    a.lse = lse;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.splits = reinterpret_cast<TreeSplit*>(ws + sp.splits);
    a.part_lse = reinterpret_cast<float*>(ws + sp.lse);
    a.part_o = reinterpret_cast<float*>(ws + sp.o);
    a.flags = reinterpret_cast<int*>(ws);
    a.claims = reinterpret_cast<unsigned*>(ws + kClaimsOff);
    a.batch = batch;
    a.total_new = total_new;
    a.mask_words = mask_words;
    a.num_qo_heads = Hq;
    a.num_kv_heads = Hk;
    a.group = group;
    a.page_size = page_size;
    a.num_total_pages = num_total_pages;
    a.num_indices = num_indices;
    while ((1 << a.tile_shift) < kn.tile_rows) ++a.tile_shift;
    a.seg_rows = kn.tile_rows * kn.tiles;
    a.hs = (group + kn.tile_rows - 1) / kn.tile_rows;
    a.hpt = (group + a.hs - 1) / a.hs;
    a.npt = kn.tile_rows / a.hpt;
    a.nps = a.npt * kn.tiles;
    int slot_rows = 1;
    if (kn.tensor) {
        // a slot is one copy: the largest power of two that divides the page, from 8 rows (the swizzle's period) to a block
        slot_rows = 8;
        while (slot_rows < kn.block_tokens && page_size % (2 * slot_rows) == 0) slot_rows *= 2;
    }
    while ((1 << a.slot_shift) < slot_rows) ++a.slot_shift;
    while ((slot_rows << a.spb_shift) < kn.block_tokens) ++a.spb_shift;
    a.cpp = int(((long long)page_size + slot_rows - 1) / slot_rows);
    a.packed = page_size % slot_rows == 0;
    a.by_page = FastDiv::of(page_size);
    a.by_cpp = FastDiv::of(a.cpp);
    a.by_nps = FastDiv::of(a.nps);
    a.by_hpt = FastDiv::of(a.hpt);
    a.by_hs = FastDiv::of(a.hs);
    a.by_heads = FastDiv::of(a.hs * Hk);
    a.scale_log2 = sm_scale * kLog2e;
    a.test_extra_tx = host::test_extra_tx();

    // No more CTAs than there can be units: segments x key blocks of the longest possible request.
    const long long segs = ((long long)total_new / a.nps + batch) * a.hs * Hk;
    const long long blocks = (((long long)num_indices * a.cpp - 1) >> a.spb_shift) + 1;
    const long long bound = segs * (blocks < 1 ? 1 : blocks);
    const long long ctas = (bound + kn.workers - 1) / kn.workers;
    const int grid = int(ctas < most ? ctas : most);
    const int workers = grid * kn.workers;
    // Requests of a few blocks are not cut: a worker streams them in less time than a merge takes (tensor
    // cores, one request of 100 tokens: 12.8 us with the merge, 10.4 without; of 250: 12.9 and 12.8. CUDA cores
    // take longer per block).
    const bool merge = workers > 1 && blocks > (kn.tensor ? 3 : 1);
    a.whole = !merge;
    a.seg_cost = kn.seg_cost;
    a.tails = merge && !(rows == kRowsMany && kn.tensor && !fp8);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if ((st = host::allow_smem(kn.main, kn.smem)) != PD_OK) return st;
    CUtensorMap maps[3]{};
    if (kn.tensor && (st = make_maps(a, dt, fp8, D, &maps[0], &maps[1], &maps[2])) != PD_OK) return st;
    void* args[] = {&a, &maps[0], &maps[1], &maps[2]};
    cudaError_t e = cudaLaunchKernel(kn.main, dim3(grid), dim3(kn.threads), args, kn.smem, cs);
    if (e != cudaSuccess) return host::cuda_fail(e, "tree decode launch");
    if (merge) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(((a.tails ? 2 : 1) * workers - 1) * kMergeBlocks);
        cfg.blockDim = dim3(256);
        cfg.stream = cs;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelExC(&cfg, kn.merge, args);
        if (e != cudaSuccess) return host::cuda_fail(e, "tree merge launch");
    }
    return host::ok();
}

}  // namespace
}  // namespace pd

using namespace pd;

extern "C" {

size_t pd_paged_tree_decode_workspace_bytes(int num_qo_heads, int num_kv_heads, int head_dim, pd_dtype dtype) {
    if (check_heads(num_qo_heads, num_kv_heads, head_dim, dtype) != PD_OK) return 0;
    int sms = 0;
    if (host::sm_count(&sms) != PD_OK) return 0;
    size_t most = 0;  // of the kernels that take this type, with either pool
    for (int form = 0; form < 8; ++form) {
        TreeKernels k{};
        if (!pick(dtype, form % 2 != 0, head_dim, num_qo_heads / num_kv_heads, Rows(form / 2), &k)) continue;
        const size_t n = space(k, sms * k.per_sm, head_dim).bytes;
        if (n > most) most = n;
    }
    host::ok();
    return most;
}

pd_status pd_paged_tree_decode(const void* q, const void* k_data, const void* v_data, const int32_t* indices,
                               const int32_t* indptr, const int32_t* last_page_len, const int32_t* new_indptr,
                               const uint32_t* tree_mask, void* o, float* lse, int batch, int total_new,
                               int mask_words, int num_qo_heads, int num_kv_heads, int head_dim, int page_size,
                               int num_total_pages, int num_indices, float sm_scale, pd_dtype dtype, void* workspace,
                               size_t workspace_bytes, void* stream) {
    return tree_impl(q, k_data, v_data, nullptr, nullptr, indices, indptr, last_page_len, new_indptr, tree_mask, o, lse,
                     batch, total_new, mask_words, num_qo_heads, num_kv_heads, head_dim, page_size, num_total_pages,
                     num_indices, sm_scale, dtype, workspace, workspace_bytes, stream, false);
}

pd_status pd_paged_tree_decode_fp8(const void* q, const void* k_data, const void* v_data, const float* k_scale,
                                   const float* v_scale, const int32_t* indices, const int32_t* indptr,
                                   const int32_t* last_page_len, const int32_t* new_indptr, const uint32_t* tree_mask,
                                   void* o, float* lse, int batch, int total_new, int mask_words, int num_qo_heads,
                                   int num_kv_heads, int head_dim, int page_size, int num_total_pages, int num_indices,
                                   float sm_scale, pd_dtype dtype, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    return tree_impl(q, k_data, v_data, k_scale, v_scale, indices, indptr, last_page_len, new_indptr, tree_mask, o, lse,
                     batch, total_new, mask_words, num_qo_heads, num_kv_heads, head_dim, page_size, num_total_pages,
                     num_indices, sm_scale, dtype, workspace, workspace_bytes, stream, true);
}

}  // extern "C"
