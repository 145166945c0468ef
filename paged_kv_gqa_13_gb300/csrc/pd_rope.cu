// Rotary positions, the paged append with the rotation on the way, and the
// commit of accepted drafted tokens: kernels and C entry points.
//
// Rotation. Pair i of a head at position p turns by p f_i: (a, b) becomes
// scale (a cos - b sin, b cos + a sin). f_i is given in turns per position as
// a 64-bit binary fraction, so the angle modulo one turn is one wrapping
// 64-bit multiply, exact at every position: its top 32 bits, as a signed
// integer, are the angle in [-1/2, 1/2) turns, which goes to sincospif. An f32
// angle would lose p 2^-24 radians (0.008 at position 131,072).
//
// All three kernels move bytes: at most 4 flops and 1/heads of a sincospif per
// element against 2 element sizes of traffic. One warp takes one token (or a
// slice of its heads when there are few tokens), so a lane computes the sines
// of its pairs once and uses them for every head.
//
// Measured: 8191 tokens of 64 f16 heads in 45.1 us, 88% of the copy rate (the
// last wave of warps is short of work); 7000 tokens of 80 f16 heads, 16 of them
// into an E4M3 pool, in 53.7 us, 74% (lookups and codes); one token in 2.7 us,
// which is a launch and two dependent reads. A prefetch of a token's rows into
// L2 before its lookup made both large calls 4 us longer.
#include <cmath>
#include <type_traits>

#include "pd_host.h"
#include "pd_rows.cuh"

namespace pd {
namespace {

constexpr int kFlagBadNewRows = PD_FLAG_BAD_NEW_ROWS;
constexpr int kFlagBadPath = PD_FLAG_BAD_PATH;

struct RopeArgs {
    // q section (hq heads): rows read at q + token * q_stride, written at q_out + token * q_out_stride
    const void* q;
    void* q_out;
    long long q_stride, q_out_stride;  // elements
    int hq;
    // k / v section (hk heads; 0: none)
    const void* k;
    const void* v;
    long long k_stride, v_stride;
    int hk;
    void* k_data;
    void* v_data;
    const float* k_scale;  // E4M3 pools
    const float* v_scale;
    const int32_t* indices;
    const int32_t* indptr;
    const int32_t* last_page_len;
    const int32_t* new_indptr;
    int batch, page_size, num_total_pages, num_indices;
    int* flags;
    // rotation
    const int32_t* positions;  // null: the token's index in its request's cache
    const uint64_t* freqs;
    float scale;
    int head_dim, rot_dim;
    int tokens, slices;
    FastDiv by_rest, by_chunks;  // by the accesses of a head's elements past rot_dim, and of a whole head
};

// Pools that a call writes: none, of q's type, or of E4M3 codes.
constexpr int kNoPool = 0, kPlainPool = 1, kCodePool = 2;

// One warp per (token, slice of the token's hq + 2 hk heads: q, k, then v).
// Unit u of a rotated head is its elements u V .. and rot/2 + u V .., V of
// each: V pairs (half layout), or V / 2 pairs in each half (pairs layout; V =
// 1: elements 2 u and 2 u + 1), so that neighbouring lanes read neighbouring
// 16 bytes in both layouts. A lane keeps one unit at a time and takes heads in
// rounds of kRound, whose loads are all issued before the first store (out may
// be x) and kept as they come. What decides is bytes in flight per SM against
// registers: without a pool 20 warps of up to 4 KB each (8191 tokens of 64 f16
// heads 45.1 us; 24 warps 47.1), into pools of the same type 24 of 4 KB (7000
// tokens of 48 bf16 heads 34.9 us; 2 KB 37.0), into E4M3 pools, whose codes
// take registers, 24 of 2 KB (7000 tokens of 80 f16 heads 53.7 us; 4 KB 61.4).
template <typename T, int kPool, int V, bool kPairs>
__global__ void __launch_bounds__(128, kPool == kNoPool ? 5 : 6) rope_kernel(const RopeArgs a) {
    constexpr int kRound = kPool == kCodePool ? 2 : 4, kCopies = kPool == kCodePool ? 4 : 8;
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (w >= (long long)a.tokens * a.slices) return;
    const int t = int(w / a.slices), slice = int(w % a.slices);
    const int D = a.head_dim, rot = a.rot_dim;
    const int items = a.hq + 2 * a.hk;
    const int i0 = int((long long)items * slice / a.slices), i1 = int((long long)items * (slice + 1) / a.slices);
    const bool wants_kv = kPool != kNoPool && i1 > a.hq;

    // ---- where this token's k and v rows go (row offset in elements of kv head 0), and its position
    int pos = 0;
    bool write_kv = false;
    size_t dst = 0;
    const size_t head_step = size_t(a.page_size) * D;
    if (kPool != kNoPool && (wants_kv || a.positions == nullptr)) {
        const int b = request_of(a.new_indptr, a.batch, t, lane);
        const int s = __ldg(a.new_indptr + b), e = __ldg(a.new_indptr + b + 1);
        const int lo = __ldg(a.indptr + b), hi = __ldg(a.indptr + b + 1);
        const int last = __ldg(a.last_page_len + b);
        int bad = 0;
        long long at = 0;
        if (s < 0 || t < s || t >= e || e > a.tokens)
            bad = kFlagBadNewRows;
        else if (lo < 0 || hi <= lo || hi > a.num_indices)
            bad = kFlagBadIndptr;
        else if (last < 0 || last > a.page_size)
            bad = kFlagBadLastPageLen;
        else {
            const long long kv = ((long long)hi - lo - 1) * a.page_size + last;
            at = kv - (e - t);  // the request's new rows are its last e - s
            if (kv < e - s) bad = kFlagBadNewRows;
        }
        if (bad == 0) {
            pos = int(at);
            if (wants_kv) {
                const int page = __ldg(a.indices + lo + int(at / a.page_size));
                if (page < 0 || page >= a.num_total_pages)
                    bad = kFlagBadPage;
                else
                    dst = size_t(page) * a.hk * head_step + size_t(at % a.page_size) * D;
            }
        }
        write_kv = bad == 0;
        if (bad != 0 && lane == 0) atomicOr(a.flags, bad);
    }
    if (a.positions != nullptr) pos = __ldg(a.positions + t);

    const T* qr = static_cast<const T*>(a.q) + (long long)t * a.q_stride;
    T* qo = static_cast<T*>(a.q_out) + (long long)t * a.q_out_stride;
    const T* kr = static_cast<const T*>(a.k) + (long long)t * a.k_stride;
    auto source = [&](int h) { return kPool == kNoPool || h < a.hq ? qr + (long long)h * D : kr + (long long)(h - a.hq) * D; };
    // V elements of rotated head h (q or k) at element e
    auto store = [&](int h, int e, const float(&f)[V]) {
        if (kPool == kNoPool || h < a.hq) {
            store_elems<T, V>(qo + (long long)h * D + e, f);
        } else if (write_kv) {
            const int kh = h - a.hq;
            const size_t at = dst + size_t(kh) * head_step + e;
            if constexpr (kPool == kCodePool)
                store_codes<V>(static_cast<uint8_t*>(a.k_data) + at, f, __ldg(a.k_scale + kh));
            else
                store_elems<T, V>(static_cast<T*>(a.k_data) + at, f);
        }
    };
    // The same of elements that are not rotated: w as they came, every bit of them, f as f32. E4M3 calls take f for q
    // too: a NaN of q stays one, its payload does not (raw stores of q there cost registers, and 7000 tokens of 80
    // heads 56.5 us instead of 53.7).
    auto store_raw = [&](int h, int e, const Raw<T, V>& w, const float(&f)[V]) {
        if constexpr (kPool == kCodePool)
            store(h, e, f);
        else if (kPool == kNoPool || h < a.hq)
            *reinterpret_cast<Raw<T, V>*>(qo + (long long)h * D + e) = w;
        else if (write_kv)
            *reinterpret_cast<Raw<T, V>*>(static_cast<T*>(a.k_data) + dst + size_t(h - a.hq) * head_step + e) = w;
    };
    const int h_end = min(i1, a.hq + a.hk);

    // ---- rotated elements of the q and k heads
    const int units = rot / (2 * V);
    if (units > 0 && i0 < h_end) {
        const int across = min(units, 32), heads = 32 / across;
        for (int u = lane % across; u < units && lane < across * heads; u += across) {
            float c[V], s[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int pair = !kPairs || V == 1 ? u * V + i : i % (V > 1 ? V / 2 : 1) + u * (V / 2) + (2 * i < V ? 0 : rot / 4);
                const uint64_t turns = uint64_t(int64_t(pos)) * __ldg(a.freqs + pair);
                // int32 -> f32 rounds the phase by at most 2^-25 of half a turn
                sincospif(float(int32_t(uint32_t(turns >> 32))) * 4.656612873077393e-10f, &s[i], &c[i]);
                s[i] *= a.scale;
                c[i] *= a.scale;
            }
            const int e0 = kPairs && V == 1 ? 2 * u : u * V, e1 = kPairs && V == 1 ? e0 + 1 : rot / 2 + u * V;
            for (int h = i0 + lane / across; h < h_end; h += heads * kRound) {
                Raw<T, V> xs[kRound], ys[kRound];
#pragma unroll
                for (int r = 0; r < kRound; ++r) {
                    if (h + r * heads < h_end) {
                        const T* row = source(h + r * heads);
                        xs[r] = *reinterpret_cast<const Raw<T, V>*>(row + e0);
                        ys[r] = *reinterpret_cast<const Raw<T, V>*>(row + e1);
                    }
                }
#pragma unroll
                for (int r = 0; r < kRound; ++r) {
                    if (h + r * heads >= h_end) continue;
                    float x[V], y[V];
                    widen<T, V>(xs[r], x);
                    widen<T, V>(ys[r], y);
                    float lo[V], hi[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        // pair i: (x[i], y[i]) in the half layout; neighbours of x, then of y, in the pairs layout
                        const float p = kPairs && V > 1 ? (2 * i < V ? x[2 * i % V] : y[2 * i % V]) : x[i];
                        const float q = kPairs && V > 1 ? (2 * i < V ? x[(2 * i + 1) % V] : y[(2 * i + 1) % V]) : y[i];
                        const float pr = p * c[i] - q * s[i], qr2 = q * c[i] + p * s[i];
                        if (kPairs && V > 1) {
                            (2 * i < V ? lo : hi)[2 * i % V] = pr;
                            (2 * i < V ? lo : hi)[(2 * i + 1) % V] = qr2;
                        } else {
                            lo[i] = pr;
                            hi[i] = qr2;
                        }
                    }
                    store(h + r * heads, e0, lo);
                    store(h + r * heads, e1, hi);
                }
            }
        }
    }
    // ---- elements past rot_dim of the q and k heads (q in place: nothing to do), then the v heads: plain copies
    const int rest = (D - rot) / V;
    const int q_from = (a.q_out == a.q && a.q_stride == a.q_out_stride) ? max(i0, a.hq) : i0;
    // n chunks of V elements, `at` giving a chunk's head and element; loads of a round before its stores
    auto copy = [&](int n, auto at, auto from, auto to) {
        for (int x = lane; x < n; x += 32 * kCopies) {
            Raw<T, V> w[kCopies];
#pragma unroll
            for (int r = 0; r < kCopies; ++r)
                if (x + 32 * r < n) {
                    const int2 c = at(x + 32 * r);
                    w[r] = *reinterpret_cast<const Raw<T, V>*>(from(c.x) + c.y);
                }
#pragma unroll
            for (int r = 0; r < kCopies; ++r)
                if (x + 32 * r < n) {
                    const int2 c = at(x + 32 * r);
                    float f[V];
                    widen<T, V>(w[r], f);
                    to(c.x, c.y, w[r], f);
                }
        }
    };
    copy(
        rest * (h_end - q_from),
        [&](int x) {
            const int h = a.by_rest.div(x);
            return make_int2(q_from + h, rot + (x - h * rest) * V);
        },
        source, store_raw);
    if (!write_kv) return;
    const int v0 = max(i0 - a.hq - a.hk, 0), v1 = i1 - a.hq - a.hk;
    const T* vr = static_cast<const T*>(a.v) + (long long)t * a.v_stride;
    copy(
        D / V * (v1 - v0),
        [&](int x) {
            const int h = a.by_chunks.div(x);
            return make_int2(v0 + h, (x - h * (D / V)) * V);
        },
        [&](int h) { return vr + (long long)h * D; },
        [&](int h, int e, const Raw<T, V>& w, const float(&f)[V]) {
            const size_t at = dst + size_t(h) * head_step + e;
            if constexpr (kPool == kCodePool)
                store_codes<V>(static_cast<uint8_t*>(a.v_data) + at, f, __ldg(a.v_scale + h));
            else
                *reinterpret_cast<Raw<T, V>*>(static_cast<T*>(a.v_data) + at) = w;
        });
}

template <typename T, int kPool, int V>
const void* pick_layout(int layout) {
    return layout == PD_ROPE_PAIRS ? reinterpret_cast<const void*>(rope_kernel<T, kPool, V, true>)
                                   : reinterpret_cast<const void*>(rope_kernel<T, kPool, V, false>);
}

// The kernel that moves 16 bytes per access where every row allows it: the
// rotated part a whole number of units, rows 16-byte aligned. Otherwise one
// element per access (odd rotary sizes, unaligned views): 8191 tokens of 64 bf16
// heads 80 to 85 us from rows off their 16 bytes and 128 us with rot_dim 100,
// against 50 (with 5 us of events each).
template <typename T, int kPool>
const void* pick_kernel(int layout, bool wide) {
    return wide ? pick_layout<T, kPool, Elt<T>::kVec>(layout) : pick_layout<T, kPool, 1>(layout);
}

template <typename T>
const void* pick_pool(int pool, int layout, bool wide) {
    if constexpr (sizeof(T) == 2)
        if (pool == kCodePool) return pick_kernel<T, kCodePool>(layout, wide);
    return pool == kNoPool ? pick_kernel<T, kNoPool>(layout, wide) : pick_kernel<T, kPlainPool>(layout, wide);
}

pd_status launch(RopeArgs& a, pd_dtype dt, bool fp8, int layout, cudaStream_t stream) {
    const int vec = dt == PD_F32 ? 4 : 8;
    const auto fits = [&](const void* p, long long stride) {
        return p == nullptr || (host::aligned(p, 16) && stride % vec == 0);
    };
    const bool wide = a.rot_dim % (2 * vec) == 0 && a.head_dim % vec == 0 && fits(a.q, a.q_stride) &&
                      fits(a.q_out, a.q_out_stride) && fits(a.k, a.k_stride) && fits(a.v, a.v_stride);
    int sms = 0;
    pd_status st = host::sm_count(&sms);
    if (st != PD_OK) return st;
    // Few tokens: cut each token's heads into slices so that the card has about 8 warps per SM. More slices make
    // a shorter last wave and more sines and lookups: with 64 warps per SM, 8191 tokens of 64 f16 heads took 47.9
    // instead of 49.7 us, but 9000 of 8 bf16 heads 22.5 instead of 16.4, and 7000 of 80 heads into an E4M3 pool
    // 68.2 instead of 64.9.
    const int items = a.hq + 2 * a.hk;
    const long long want = ((long long)sms * 8 + a.tokens - 1) / a.tokens;
    a.slices = int(want < 1 ? 1 : want > (items + 3) / 4 ? (items + 3) / 4 : want);
    const int per = wide ? vec : 1;
    if (a.head_dim > a.rot_dim) a.by_rest = FastDiv::of((a.head_dim - a.rot_dim) / per);
    a.by_chunks = FastDiv::of(a.head_dim / per);
    const long long warps = (long long)a.tokens * a.slices;
    const int pool = a.hk == 0 ? kNoPool : fp8 ? kCodePool : kPlainPool;
    const void* fn = dt == PD_F32   ? pick_pool<float>(pool, layout, wide)
                     : dt == PD_F16 ? pick_pool<__half>(pool, layout, wide)
                                    : pick_pool<__nv_bfloat16>(pool, layout, wide);
    void* args[] = {&a};
    const cudaError_t e = cudaLaunchKernel(fn, dim3(unsigned((warps + 3) / 4)), dim3(128), args, 0, stream);
    return e == cudaSuccess ? host::ok() : host::cuda_fail(e, "rope launch");
}

// ---------------------------------------------------------------- commit

struct CommitArgs {
    uint8_t* k_data;
    uint8_t* v_data;
    const int32_t* indices;
    const int32_t* indptr;
    const int32_t* last_page_len;
    const int32_t* new_indptr;
    const int32_t* path;
    const int32_t* path_len;
    int* flags;
    int batch, total_new, max_path, hk, row_bytes, page_size, num_total_pages, num_indices;
};

// One warp per (request, kv head): row first + path[i] moves to row first + i,
// first the request's first new row, for K (chunks 0 .. n - 1 of 16 bytes) and
// V (the next n). Lane i finds the places of the path's node i, 32 at a time;
// then a lane owns whole columns of chunks and walks them in order, kRound rows
// at a time, loads before stores. A path increases, so path[i] >= i: no row is
// written before it has been read; no row moves where one of the pages is bad.
// Bound by a chain of four dependent reads (lengths, path, page, row): 3.2 us for 32 requests, 4.3 for 256 that keep up
// to 12 of 64 nodes (places found one after another: 8.1).
__global__ void __launch_bounds__(128) commit_kernel(const CommitArgs a) {
    constexpr int kRound = 8;
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (w >= (long long)a.batch * a.hk) return;
    const int b = int(w / a.hk), kh = int(w % a.hk);
    const int len = __ldg(a.path_len + b);
    const int s = __ldg(a.new_indptr + b), e = __ldg(a.new_indptr + b + 1);
    const int lo = __ldg(a.indptr + b), hi = __ldg(a.indptr + b + 1);
    const int last = __ldg(a.last_page_len + b);
    const int32_t* path = a.path + (long long)b * a.max_path;
    int mine = lane < a.max_path ? __ldg(path + lane) : 0;  // this lane's node of the first 32
    if (len == 0) return;
    int bad = 0;
    const long long kv = ((long long)hi - lo - 1) * a.page_size + last;
    if (s < 0 || e < s || e > a.total_new)
        bad = kFlagBadNewRows;
    else if (lo < 0 || hi <= lo || hi > a.num_indices)
        bad = kFlagBadIndptr;
    else if (last < 0 || last > a.page_size)
        bad = kFlagBadLastPageLen;
    else if (kv < e - s)
        bad = kFlagBadNewRows;
    else if (len < 0 || len > a.max_path)
        bad = kFlagBadPath;
    if (bad == 0) {
        bool wrong = false;
        int before = -1;  // the last node of the 32 before
        for (int i0 = 0; i0 < len; i0 += 32) {
            const int node = i0 == 0 ? mine : i0 + lane < len ? __ldg(path + i0 + lane) : 0;
            int prev = __shfl_up_sync(kFull, node, 1);
            if (lane == 0) prev = before;
            before = __shfl_sync(kFull, node, 31);
            wrong |= i0 + lane < len && (node <= prev || node >= e - s);
        }
        if (__any_sync(kFull, wrong)) bad = kFlagBadPath;
    }
    if (bad != 0) {
        if (lane == 0 && kh == 0) atomicOr(a.flags, bad);
        return;
    }
    const long long first = kv - (e - s);
    const int chunks = a.row_bytes / 16;
    // byte offset of the request's row `at` of this kv head; false: a bad page
    auto locate = [&](long long at, size_t* off) {
        const int nth = int(at / a.page_size), page = __ldg(a.indices + lo + nth);
        *off = ((size_t(page) * a.hk + kh) * a.page_size + size_t(at - (long long)nth * a.page_size)) * a.row_bytes;
        return page >= 0 && page < a.num_total_pages;
    };
    size_t from = 0, to = 0;
    bool go = false;
    // the places of node i0 + lane of the path; false: a bad page
    auto find = [&](int i0) {
        if (i0 > 0) mine = i0 + lane < len ? __ldg(path + i0 + lane) : 0;
        go = i0 + lane < len && mine != i0 + lane;
        return !go || (locate(first + mine, &from) & locate(first + i0 + lane, &to));
    };
    // every page is looked at before the first row moves
    bool fine = true;
    for (int i0 = (len - 1) / 32 * 32; i0 > 0; i0 -= 32) fine &= find(i0);
    if (len > 32) mine = __ldg(path + lane);
    fine &= find(0);
    if (!__all_sync(kFull, fine)) {
        if (lane == 0 && kh == 0) atomicOr(a.flags, kFlagBadPage);
        return;
    }
    for (int i0 = 0; i0 < len; i0 += 32) {
        if (i0 > 0) find(i0);
        const unsigned moves = __ballot_sync(kFull, go);
        for (unsigned rest = moves; rest != 0u;) {
            size_t src[kRound], dst[kRound];
            int n = 0;
#pragma unroll
            for (int r = 0; r < kRound; ++r) {
                if (rest != 0u) {
                    const int x = __ffs(rest) - 1;
                    rest &= rest - 1u;
                    src[r] = __shfl_sync(kFull, from, x);
                    dst[r] = __shfl_sync(kFull, to, x);
                    n = r + 1;
                }
            }
            for (int c = lane; c < 2 * chunks; c += 32) {
                uint8_t* pool = c < chunks ? a.k_data : a.v_data;
                const size_t at = size_t(c < chunks ? c : c - chunks) * 16;
                uint4 x[kRound];
#pragma unroll
                for (int r = 0; r < kRound; ++r)
                    if (r < n) x[r] = *reinterpret_cast<const uint4*>(pool + src[r] + at);
#pragma unroll
                for (int r = 0; r < kRound; ++r)
                    if (r < n) *reinterpret_cast<uint4*>(pool + dst[r] + at) = x[r];
            }
        }
    }
}

pd_status append_impl(const void* q, const void* k_new, const void* v_new, const int32_t* positions,
                      const uint64_t* freqs, void* q_out, const float* k_scale, const float* v_scale, void* k_data,
                      void* v_data, const int32_t* indices, const int32_t* indptr, const int32_t* last_page_len,
                      const int32_t* new_indptr, int batch, int total_new, int Hq, int Hk, int D, int rot_dim,
                      int page_size, int num_total_pages, int num_indices, long long q_stride, long long k_stride,
                      long long v_stride, int layout, float rope_scale, pd_dtype dt, void* workspace,
                      size_t workspace_bytes, void* stream, bool fp8) {
    if (D != 64 && D != 128 && D != 256) return host::fail(PD_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256 (got %d)", D);
    pd_status st = host::check_rotation(total_new, D, rot_dim, layout, rope_scale, freqs, dt);
    if (st != PD_OK) return st;
    if (batch <= 0 || Hk <= 0 || page_size <= 0 || num_total_pages <= 0)
        return host::fail(PD_ERR_INVALID, "batch, num_kv_heads, page_size and num_total_pages must be positive");
    if (num_indices < 0 || Hq < 0 || Hq > (1 << 20) || Hk > (1 << 20))
        return host::fail(PD_ERR_INVALID, "num_indices and num_qo_heads must not be negative, heads at most 2^20");
    if (!k_data || !v_data || !indptr || !last_page_len || !new_indptr || (num_indices > 0 && !indices) ||
        (total_new > 0 && (!k_new || !v_new || (Hq > 0 && (!q || !q_out)))) || (fp8 && (!k_scale || !v_scale)))
        return host::fail(PD_ERR_INVALID, "null pointer argument");
    if (k_stride < (long long)Hk * D || v_stride < (long long)Hk * D || (Hq > 0 && q_stride < (long long)Hq * D))
        return host::fail(PD_ERR_INVALID, "a token's stride must hold its heads");
    // (one token lies where it lies whatever its stride)
    if (Hq > 0 && total_new > 1 && q == q_out && q_stride != (long long)Hq * D)
        return host::fail(PD_ERR_INVALID, "q_out may be q only where q_stride is num_qo_heads * head_dim");
    const size_t e = host::elem_size(dt);
    if (!host::aligned(k_data, 16) || !host::aligned(v_data, 16))
        return host::fail(PD_ERR_UNSUPPORTED, "k_data and v_data must be 16-byte aligned");
    if (!host::aligned(q, e) || !host::aligned(q_out, e) || !host::aligned(k_new, e) || !host::aligned(v_new, e))
        return host::fail(PD_ERR_UNSUPPORTED, "q, q_out, k_new and v_new must be aligned to their element");
    if (!host::aligned(positions, 4) || !host::aligned(indices, 4) || !host::aligned(indptr, 4) ||
        !host::aligned(last_page_len, 4) || !host::aligned(new_indptr, 4) || !host::aligned(k_scale, 4) ||
        !host::aligned(v_scale, 4))
        return host::fail(PD_ERR_UNSUPPORTED, "positions, the table and the scales must be 4-byte aligned");
    if ((st = host::check_workspace(workspace, workspace_bytes, PD_WORKSPACE_HEADER_BYTES)) != PD_OK) return st;
    if (total_new == 0) return host::ok();
    RopeArgs a{};
    a.q = Hq > 0 ? q : nullptr;
    a.q_out = Hq > 0 ? q_out : nullptr;
    a.q_stride = Hq > 0 ? q_stride : 0;
    a.q_out_stride = (long long)Hq * D;
    a.hq = Hq;
    a.k = k_new;
    a.v = v_new;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.hk = Hk;
    a.k_data = k_data;
    a.v_data = v_data;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.indices = indices;
    a.indptr = indptr;
    a.last_page_len = last_page_len;
    a.new_indptr = new_indptr;
    a.batch = batch;
    a.page_size = page_size;
    a.num_total_pages = num_total_pages;
    a.num_indices = num_indices;
    a.flags = static_cast<int*>(workspace);
    a.positions = positions;
    a.freqs = freqs;
    a.scale = rope_scale;
    a.head_dim = D;
    a.rot_dim = rot_dim;
    a.tokens = total_new;
    return launch(a, dt, fp8, layout, static_cast<cudaStream_t>(stream));
}

}  // namespace
}  // namespace pd

namespace pd {
namespace host {

pd_status check_rotation(int tokens, int head_dim, int rot_dim, int layout, float rope_scale, const uint64_t* freqs,
                         pd_dtype dt) {
    if (!known_dtype(dt)) return fail(PD_ERR_UNSUPPORTED, "dtype must be PD_F32, PD_F16 or PD_BF16");
    if (tokens < 0) return fail(PD_ERR_INVALID, "the number of tokens must not be negative");
    if (rot_dim < 0 || rot_dim % 2 != 0 || rot_dim > head_dim)
        return fail(PD_ERR_INVALID, "rot_dim must be even and in [0, head_dim] (got %d of %d)", rot_dim, head_dim);
    if (layout != PD_ROPE_HALF && layout != PD_ROPE_PAIRS)
        return fail(PD_ERR_INVALID, "layout must be PD_ROPE_HALF or PD_ROPE_PAIRS");
    if (!std::isfinite(rope_scale)) return fail(PD_ERR_INVALID, "rope_scale must be finite");
    if (rot_dim > 0 && !freqs) return fail(PD_ERR_INVALID, "null pointer argument");
    if (!aligned(freqs, 8)) return fail(PD_ERR_UNSUPPORTED, "freqs must be 8-byte aligned");
    return PD_OK;
}

}  // namespace host
}  // namespace pd

using namespace pd;

extern "C" {

pd_status pd_rope_frequencies(uint64_t* freqs, float* rope_scale, int rot_dim, double theta, int scaling,
                              double factor, double low, double high, int original_positions) {
    const double kTwoPi = 6.283185307179586476925286766559;
    if (!freqs || !rope_scale) return host::fail(PD_ERR_INVALID, "null pointer argument");
    if (rot_dim <= 0 || rot_dim % 2 != 0) return host::fail(PD_ERR_INVALID, "rot_dim must be positive and even (got %d)", rot_dim);
    if (!(theta > 1.0) || !std::isfinite(theta)) return host::fail(PD_ERR_INVALID, "theta must be finite and above 1");
    if (scaling < PD_ROPE_PLAIN || scaling > PD_ROPE_YARN) return host::fail(PD_ERR_INVALID, "unknown rope scaling %d", scaling);
    if (scaling != PD_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
        return host::fail(PD_ERR_INVALID, "factor must be finite and at least 1");
    const bool ranged = scaling == PD_ROPE_BANDED || scaling == PD_ROPE_YARN;
    if (ranged && (!(low > 0.0) || !(high > low) || !std::isfinite(high) || original_positions <= 0))
        return host::fail(PD_ERR_INVALID, "banded and yarn scaling need 0 < low < high and original_positions > 0");
    if (scaling == PD_ROPE_BASE) {
        if (rot_dim < 4) return host::fail(PD_ERR_INVALID, "base scaling needs rot_dim of at least 4");
        theta *= std::pow(factor, double(rot_dim) / (rot_dim - 2));
    }
    // yarn: the pair index at which a pair makes n turns over the original context
    const auto index_of = [&](double n) { return rot_dim * std::log(original_positions / (n * kTwoPi)) / (2.0 * std::log(theta)); };
    double from = 0.0, to = 0.0;
    if (scaling == PD_ROPE_YARN) {
        from = std::fmax(std::floor(index_of(high)), 0.0);
        to = std::fmin(std::ceil(index_of(low)), double(rot_dim - 1));
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / rot_dim);
        if (scaling == PD_ROPE_LINEAR) {
            f /= factor;
        } else if (ranged) {
            // keep: the share of the unstretched frequency
            double keep = scaling == PD_ROPE_BANDED ? (original_positions * f / kTwoPi - low) / (high - low)
                                                    : 1.0 - (i - from) / std::fmax(to - from, 0.001);
            keep = std::fmin(std::fmax(keep, 0.0), 1.0);
            f = (1.0 - keep) * f / factor + keep * f;
        }
        freqs[i] = uint64_t(std::ldexp(f / kTwoPi, 64));  // f <= 1: below 2^62
    }
    *rope_scale = scaling == PD_ROPE_YARN ? float(0.1 * std::log(factor) + 1.0) : 1.f;
    return host::ok();
}

pd_status pd_rope(const void* x, const int32_t* positions, const uint64_t* freqs, void* out, int num_tokens,
                  int num_heads, int head_dim, int rot_dim, int64_t x_stride, int64_t out_stride, int layout,
                  float rope_scale, pd_dtype dtype, void* stream) {
    if (num_heads <= 0 || num_heads > (1 << 20) || head_dim <= 0 || head_dim > 4096)
        return host::fail(PD_ERR_INVALID, "num_heads must be in [1, 2^20] and head_dim in [1, 4096]");
    const pd_status st = host::check_rotation(num_tokens, head_dim, rot_dim, layout, rope_scale, freqs, dtype);
    if (st != PD_OK) return st;
    if (num_tokens > 0 && (!x || !out || !positions)) return host::fail(PD_ERR_INVALID, "null pointer argument");
    if (x_stride < (long long)num_heads * head_dim || out_stride < (long long)num_heads * head_dim)
        return host::fail(PD_ERR_INVALID, "a token's stride must hold its heads");
    if (num_tokens > 1 && x == out && x_stride != out_stride) return host::fail(PD_ERR_INVALID, "in place, both strides must be the same");
    const size_t e = host::elem_size(dtype);
    if (!host::aligned(x, e) || !host::aligned(out, e) || !host::aligned(positions, 4))
        return host::fail(PD_ERR_UNSUPPORTED, "x and out must be aligned to their element, positions to 4 bytes");
    if (num_tokens == 0) return host::ok();
    RopeArgs a{};
    a.q = x;
    a.q_out = out;
    a.q_stride = x_stride;
    a.q_out_stride = out_stride;
    a.hq = num_heads;
    a.positions = positions;
    a.freqs = freqs;
    a.scale = rope_scale;
    a.head_dim = head_dim;
    a.rot_dim = rot_dim;
    a.tokens = num_tokens;
    return launch(a, dtype, false, layout, static_cast<cudaStream_t>(stream));
}

pd_status pd_paged_rope_append(const void* q, const void* k_new, const void* v_new, const int32_t* positions,
                               const uint64_t* freqs, void* q_out, void* k_data, void* v_data, const int32_t* indices,
                               const int32_t* indptr, const int32_t* last_page_len, const int32_t* new_indptr,
                               int batch, int total_new, int num_qo_heads, int num_kv_heads, int head_dim, int rot_dim,
                               int page_size, int num_total_pages, int num_indices, int64_t q_stride, int64_t k_stride,
                               int64_t v_stride, int layout, float rope_scale, pd_dtype dtype, void* workspace,
                               size_t workspace_bytes, void* stream) {
    return append_impl(q, k_new, v_new, positions, freqs, q_out, nullptr, nullptr, k_data, v_data, indices, indptr,
                       last_page_len, new_indptr, batch, total_new, num_qo_heads, num_kv_heads, head_dim, rot_dim,
                       page_size, num_total_pages, num_indices, q_stride, k_stride, v_stride, layout, rope_scale, dtype,
                       workspace, workspace_bytes, stream, false);
}

pd_status pd_paged_rope_append_fp8(const void* q, const void* k_new, const void* v_new, const int32_t* positions,
                                   const uint64_t* freqs, void* q_out, const float* k_scale, const float* v_scale,
                                   void* k_data, void* v_data, const int32_t* indices, const int32_t* indptr,
                                   const int32_t* last_page_len, const int32_t* new_indptr, int batch, int total_new,
                                   int num_qo_heads, int num_kv_heads, int head_dim, int rot_dim, int page_size,
                                   int num_total_pages, int num_indices, int64_t q_stride, int64_t k_stride,
                                   int64_t v_stride, int layout, float rope_scale, pd_dtype dtype, void* workspace,
                                   size_t workspace_bytes, void* stream) {
    if (dtype != PD_F16 && dtype != PD_BF16) return host::fail(PD_ERR_UNSUPPORTED, "E4M3 pools take PD_F16 or PD_BF16 rows");
    return append_impl(q, k_new, v_new, positions, freqs, q_out, k_scale, v_scale, k_data, v_data, indices, indptr,
                       last_page_len, new_indptr, batch, total_new, num_qo_heads, num_kv_heads, head_dim, rot_dim,
                       page_size, num_total_pages, num_indices, q_stride, k_stride, v_stride, layout, rope_scale, dtype,
                       workspace, workspace_bytes, stream, true);
}

pd_status pd_paged_tree_commit(void* k_data, void* v_data, const int32_t* indices, const int32_t* indptr,
                               const int32_t* last_page_len, const int32_t* new_indptr, const int32_t* path,
                               const int32_t* path_len, int batch, int total_new, int max_path, int num_kv_heads,
                               int head_dim, int page_size, int num_total_pages, int num_indices, int elem_bytes,
                               void* workspace, size_t workspace_bytes, void* stream) {
    if (batch <= 0 || num_kv_heads <= 0 || page_size <= 0 || num_total_pages <= 0)
        return host::fail(PD_ERR_INVALID, "batch, num_kv_heads, page_size and num_total_pages must be positive");
    if (total_new < 0 || max_path < 0 || num_indices < 0)
        return host::fail(PD_ERR_INVALID, "total_new, max_path and num_indices must not be negative");
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return host::fail(PD_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256 (got %d)", head_dim);
    if (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4)
        return host::fail(PD_ERR_UNSUPPORTED, "elem_bytes must be 1, 2 or 4 (got %d)", elem_bytes);
    if (!k_data || !v_data || !indptr || !last_page_len || !new_indptr || !path_len || (num_indices > 0 && !indices) ||
        (max_path > 0 && !path))
        return host::fail(PD_ERR_INVALID, "null pointer argument");
    if (!host::aligned(k_data, 16) || !host::aligned(v_data, 16))
        return host::fail(PD_ERR_UNSUPPORTED, "k_data and v_data must be 16-byte aligned");
    if (!host::aligned(indices, 4) || !host::aligned(indptr, 4) || !host::aligned(last_page_len, 4) ||
        !host::aligned(new_indptr, 4) || !host::aligned(path, 4) || !host::aligned(path_len, 4))
        return host::fail(PD_ERR_UNSUPPORTED, "the table and the path must be 4-byte aligned");
    const pd_status st = host::check_workspace(workspace, workspace_bytes, PD_WORKSPACE_HEADER_BYTES);
    if (st != PD_OK) return st;
    if (max_path == 0) return host::ok();
    CommitArgs a{static_cast<uint8_t*>(k_data), static_cast<uint8_t*>(v_data), indices, indptr, last_page_len,
                 new_indptr, path, path_len, static_cast<int*>(workspace), batch, total_new, max_path, num_kv_heads,
                 head_dim * elem_bytes, page_size, num_total_pages, num_indices};
    void* args[] = {&a};
    const long long warps = (long long)batch * num_kv_heads;
    if (warps > 4LL * 0x7fffffff) return host::fail(PD_ERR_INVALID, "batch * num_kv_heads is too large");
    const cudaError_t e = cudaLaunchKernel(reinterpret_cast<const void*>(commit_kernel), dim3(unsigned((warps + 3) / 4)),
                                           dim3(128), args, 0, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? host::ok() : host::cuda_fail(e, "commit launch");
}

}  // extern "C"
