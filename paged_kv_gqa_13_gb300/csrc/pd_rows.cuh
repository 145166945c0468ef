// What the kernels that read and write whole rows of heads share: accesses of
// 16 bytes or of one element, E4M3 codes, and the request of a ragged row.
#pragma once

#include <type_traits>

#include "pd_device.cuh"

namespace pd {

// V elements of a row: one 16-byte access, or one element (V = 1).
template <typename T, int V>
using Raw = typename std::conditional<V == 1, T, uint4>::type;

template <typename T, int V>
__device__ __forceinline__ void widen(const Raw<T, V>& w, float (&f)[V]) {
    if constexpr (V == 1)
        f[0] = float(w);
    else
        Elt<T>::to_f32(w, f);
}

template <typename T, int V>
__device__ __forceinline__ void store_elems(T* p, const float (&f)[V]) {
    if constexpr (V == 1)
        *p = T(f[0]);
    else
        *reinterpret_cast<uint4*>(p) = Elt<T>::from_f32(f);
}

// The E4M3 codes of f[i] / scale: the division in f32 (IEEE), then rounded to
// the nearest code, ties to even, saturating at +-448 (NaN stays NaN).
template <int V>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&f)[V], float scale) {
    if constexpr (V == 1) {
        *p = __nv_cvt_float_to_fp8(__fdiv_rn(f[0], scale), __NV_SATFINITE, __NV_E4M3);
    } else {
        uint32_t w[V / 4] = {};
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float2 x = make_float2(__fdiv_rn(f[i], scale), __fdiv_rn(f[i + 1], scale));
            w[i / 4] |= uint32_t(__nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3)) << (8 * (i % 4));
        }
        if constexpr (V == 8)
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t*>(p) = w[0];
    }
}

// The request b whose range [new_indptr[b], new_indptr[b + 1]) holds token t,
// by a 32-way search of the whole warp (one round for up to 32 requests). On a
// malformed table it still ends, with some b in [0, batch).
__device__ __forceinline__ int request_of(const int32_t* new_indptr, int batch, int t, int lane) {
    int lo = 0, hi = batch;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const long long at = lo + (long long)(lane + 1) * step;
        const bool below = at < hi && __ldg(new_indptr + at) <= t;
        lo += __popc(__ballot_sync(kFull, below)) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

}  // namespace pd
