// Reading tokens of a block-scaled E4M3 cache back as rows of T: kernel and C
// entry point. An element is its code's value times its block's scale, one f32
// product rounded once to T.
//
// Bound by its bytes: one in and sizeof(T) out for each element. One CTA takes
// 16 rows of output of one request (tiles as in the appends, see pd_norm_rope.cu)
// and a thread 16 bytes of codes at a time: 8 threads read a 128-byte row, whose
// neighbours in the page follow, and write a head's row of the output. 16 requests,
// 53,000 tokens of 8 heads of 128 to bf16: 58 us between events, 51 of them the
// kernel's against 48 for the bytes; 2 or 8 loads at once, 128 threads and tiles of
// 32 rows read 58 to 62.
#include "pd_host.h"
#include "pd_rows.cuh"

namespace pd {
namespace {

constexpr int kFlagBadNewRows = PD_FLAG_BAD_NEW_ROWS;
constexpr int kThreads = 256, kTile = 16;

struct ReadArgs {
    const uint8_t* k;
    const uint8_t* v;
    const float* k_scale;
    const float* v_scale;
    const int32_t* indices;
    const int32_t* indptr;
    const int32_t* last_page_len;
    const int32_t* out_indptr;
    const int32_t* first;  // null: 0
    void* k_out;
    void* v_out;
    int batch, total, hk, page_size, num_total_pages, num_indices, block, slices;
    int* flags;
};

// 16 elements, in stores of whole 32-byte sectors where the rows lie so: a warp's 16-byte stores, two to a sector and 32
// bytes apart, take 68 us where these take 58 (16 requests, 53,000 tokens of 8 heads of 128 to bf16).
template <bool kSectors, typename T>
__device__ __forceinline__ void store16(T* p, const float (&f)[16]) {
    constexpr int kVec = Elt<T>::kVec;
#pragma unroll
    for (int i = 0; i < 16; i += 2 * kVec) {
        const uint4 x = Elt<T>::from_f32(f + i), y = Elt<T>::from_f32(f + i + kVec);
        if constexpr (kSectors) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + i), "r"(x.x), "r"(x.y), "r"(x.z),
                         "r"(x.w), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w)
                         : "memory");
        } else {
            *reinterpret_cast<uint4*>(p + i) = x;
            *reinterpret_cast<uint4*>(p + i + kVec) = y;
        }
    }
}

// kSectors: k_out and v_out are 32-byte aligned
template <typename T, int D, bool kSectors>
__global__ void __launch_bounds__(kThreads) blocks_read_kernel(const ReadArgs a) {
    constexpr int kPieces = D / 16, kAhead = 4;  // 16-byte pieces of a row; loads in flight
    __shared__ int s_count, s_first;
    __shared__ long long s_row[kTile];    // pool row of kv head 0; -1: a bad page
    __shared__ long long s_scale[kTile];  // scale of kv head 0
    const int tid = threadIdx.x, lane = tid & 31;
    const int c = int(blockIdx.x) / a.slices, slice = int(blockIdx.x) - c * a.slices;
    const int per = a.page_size / a.block;
    // Each request's range is checked by a tile of its number (there are as many and more).
    if (tid == 32 && slice == 0 && c < a.batch) {
        const int s = __ldg(a.out_indptr + c), e = __ldg(a.out_indptr + c + 1);
        if (s < 0 || e < s || e > a.total) atomicOr(a.flags, kFlagBadNewRows);
    }
    if (tid < 32) {
        // request b's tiles start at out_indptr[b] / kTile + b
        int lo_b = 0, hi_b = a.batch;
        while (hi_b - lo_b > 1) {
            const int step = (hi_b - lo_b + 31) / 32;
            const long long at = lo_b + (long long)(lane + 1) * step;
            const bool below = at < hi_b && max(0, __ldg(a.out_indptr + at)) / kTile + at <= c;
            lo_b += __popc(__ballot_sync(kFull, below)) * step;
            hi_b = min(hi_b, lo_b + step);
        }
        const int b = lo_b;
        const int s = __ldg(a.out_indptr + b), e = __ldg(a.out_indptr + b + 1);
        const int lo = __ldg(a.indptr + b), hi = __ldg(a.indptr + b + 1), last = __ldg(a.last_page_len + b);
        const int from = a.first != nullptr ? __ldg(a.first + b) : 0;
        int bad = 0, count = 0, row0 = 0;
        if (s < 0 || e < s || e > a.total) {
            bad = kFlagBadNewRows;
        } else if (e > s) {
            if (lo < 0 || hi < lo || hi > a.num_indices)
                bad = kFlagBadIndptr;
            else if (hi > lo && (last < 0 || last > a.page_size))
                bad = kFlagBadLastPageLen;
            else if (from < 0 || (long long)from + (e - s) > 0x7fffffffll ||
                     (long long)from + (e - s) > (hi > lo ? (long long)(hi - lo - 1) * a.page_size + last : 0ll))
                bad = kFlagBadNewRows;
            else {
                row0 = (c - (s / kTile + b)) * kTile;  // of the request's rows
                count = max(0, min(kTile, e - s - row0));
            }
        }
        if (bad != 0 && lane == 0 && slice == 0) atomicOr(a.flags, bad);
        if (lane < count) {
            const int t = from + row0 + lane, nth = t / a.page_size, row = t - nth * a.page_size;
            const int page = __ldg(a.indices + lo + nth);
            const bool fine = page >= 0 && page < a.num_total_pages;
            if (!fine && slice == 0) atomicOr(a.flags, kFlagBadPage);
            s_row[lane] = fine ? (long long)page * a.hk * a.page_size + row : -1;
            s_scale[lane] = (long long)page * a.hk * per + row / a.block;
        }
        if (lane == 0) {
            s_count = count;
            s_first = s + row0;
        }
    }
    __syncthreads();
    const int count = s_count;
    if (count == 0) return;
    // pieces in the order head, K or V, row, place: i / kPieces is a row of a head
    const int h0 = int((long long)a.hk * slice / a.slices), h1 = int((long long)a.hk * (slice + 1) / a.slices);
    const int n = (h1 - h0) * 2 * count * kPieces;
    for (int i0 = tid; i0 < n; i0 += kThreads * kAhead) {
        uint4 w[kAhead];
        float s[kAhead];
        T* to[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j * kThreads;
            if (i >= n) break;
            const int piece = i % kPieces, x = i / kPieces, y = x / count, r = x - y * count, h = h0 + (y >> 1);
            const bool is_v = (y & 1) != 0;
            const long long row = s_row[r];
            w[j] = make_uint4(0u, 0u, 0u, 0u);
            s[j] = 0.f;
            if (row >= 0) {
                w[j] = __ldg(reinterpret_cast<const uint4*>((is_v ? a.v : a.k) + (size_t(row) + size_t(h) * a.page_size) * D + piece * 16));
                s[j] = __ldg((is_v ? a.v_scale : a.k_scale) + s_scale[r] + (long long)h * per);
            }
            to[j] = static_cast<T*>(is_v ? a.v_out : a.k_out) + ((size_t(s_first) + r) * a.hk + h) * D + piece * 16;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (i0 + j * kThreads >= n) break;
            float f[16];
            e4m3x8_to_f32(make_uint2(w[j].x, w[j].y), f);
            e4m3x8_to_f32(make_uint2(w[j].z, w[j].w), f + 8);
#pragma unroll
            for (int x = 0; x < 16; ++x) f[x] *= s[j];
            store16<kSectors>(to[j], f);
        }
    }
}

template <typename T, bool kSectors>
const void* by_dim(int D) {
    return D == 64    ? reinterpret_cast<const void*>(blocks_read_kernel<T, 64, kSectors>)
           : D == 128 ? reinterpret_cast<const void*>(blocks_read_kernel<T, 128, kSectors>)
                      : reinterpret_cast<const void*>(blocks_read_kernel<T, 256, kSectors>);
}

template <bool kSectors>
const void* by_type(pd_dtype dtype, int D) {
    return dtype == PD_F32   ? by_dim<float, kSectors>(D)
           : dtype == PD_F16 ? by_dim<__half, kSectors>(D)
                             : by_dim<__nv_bfloat16, kSectors>(D);
}

}  // namespace
}  // namespace pd

using namespace pd;

extern "C" {

pd_status pd_paged_read_fp8_blocks(const void* k_data, const void* v_data, const float* k_scale, const float* v_scale,
                                   const int32_t* indices, const int32_t* indptr, const int32_t* last_page_len,
                                   const int32_t* out_indptr, const int32_t* first, void* k_out, void* v_out, int batch,
                                   int total, int num_kv_heads, int head_dim, int page_size, int num_total_pages,
                                   int num_indices, int block_tokens, pd_dtype dtype, void* workspace,
                                   size_t workspace_bytes, void* stream) {
    if (!host::known_dtype(dtype)) return host::fail(PD_ERR_UNSUPPORTED, "dtype must be PD_F32, PD_F16 or PD_BF16");
    if (batch <= 0 || num_kv_heads <= 0 || page_size <= 0 || num_total_pages <= 0)
        return host::fail(PD_ERR_INVALID, "batch, num_kv_heads, page_size and num_total_pages must be positive");
    if (total < 0 || num_indices < 0 || num_kv_heads > (1 << 20) || batch > (1 << 28))
        return host::fail(PD_ERR_INVALID, "total and num_indices must not be negative, heads at most 2^20, batch at most 2^28");
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return host::fail(PD_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256 (got %d)", head_dim);
    pd_status st = host::check_block(block_tokens, page_size);
    if (st != PD_OK) return st;
    if (!k_data || !v_data || !k_scale || !v_scale || !indptr || !last_page_len || !out_indptr || (num_indices > 0 && !indices) ||
        (total > 0 && (!k_out || !v_out)))
        return host::fail(PD_ERR_INVALID, "null pointer argument");
    if (!host::aligned(k_data, 16) || !host::aligned(v_data, 16) || !host::aligned(k_out, 16) || !host::aligned(v_out, 16))
        return host::fail(PD_ERR_UNSUPPORTED, "k_data, v_data, k_out and v_out must be 16-byte aligned");
    if (!host::aligned(k_scale, 4) || !host::aligned(v_scale, 4) || !host::aligned(indices, 4) || !host::aligned(indptr, 4) ||
        !host::aligned(last_page_len, 4) || !host::aligned(out_indptr, 4) || !host::aligned(first, 4))
        return host::fail(PD_ERR_UNSUPPORTED, "the table and the scales must be 4-byte aligned");
    if ((st = host::check_workspace(workspace, workspace_bytes, PD_WORKSPACE_HEADER_BYTES)) != PD_OK) return st;
    if (total == 0) return host::ok();
    int sms = 0;
    if ((st = host::sm_count(&sms)) != PD_OK) return st;
    // Few rows: the heads of a tile in slices, so that the card has about 8 CTAs per SM.
    const long long tiles = (long long)total / kTile + batch;
    const long long want = ((long long)sms * 8 + tiles - 1) / tiles;
    ReadArgs a{static_cast<const uint8_t*>(k_data), static_cast<const uint8_t*>(v_data), k_scale, v_scale, indices, indptr,
               last_page_len, out_indptr, first, k_out, v_out, batch, total, num_kv_heads, page_size, num_total_pages,
               num_indices, block_tokens, int(want > num_kv_heads ? num_kv_heads : want), static_cast<int*>(workspace)};
    if (tiles * a.slices > 0x7fffffff) return host::fail(PD_ERR_INVALID, "batch and the number of tokens are too large");
    const bool sectors = host::aligned(k_out, 32) && host::aligned(v_out, 32);
    const void* fn = sectors ? by_type<true>(dtype, head_dim) : by_type<false>(dtype, head_dim);
    void* args[] = {&a};
    const cudaError_t e = cudaLaunchKernel(fn, dim3(unsigned(tiles * a.slices)), dim3(kThreads), args, 0, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? host::ok() : host::cuda_fail(e, "block-scaled read launch");
}

}  // extern "C"
