// Norms of q and k heads with the rotary positions in the same pass, and the
// appends that do both on the way into a paged pool: rows of the pool's type,
// E4M3 codes with a scale per kv head, and E4M3 codes with a scale for each
// block of rows and kv head, which this kernel chooses.
//
// A head x becomes x / sqrt(mean(x^2) + eps) * w, then its pairs turn (see
// pd_rope.cu for the angles). f32 throughout, rounded once.
//
// Block scales. The rows of a block are new ones and, where a request's new
// rows start inside a block, older ones. A block of new rows gets s = a / 448, a
// its largest finite magnitude. A block with older rows keeps its scale unless a
// new element would round past the largest code (a > 464 s); the scale then
// doubles until it would not, and the older codes are rounded again by that
// power of two. A code is a floating-point number, so that this is exact unless
// it becomes a subnormal (or was one): rows that came one at a time are as good
// as rows that came together. (A scale of a / 448 anew each time would round
// older rows by a new factor each time.)
//
// Rows that pass through (q; k and v too where the pool's scales are given) go token by token, as in pd_rope.cu: a warp
// takes a token or a slice of its heads, a group of L lanes a head, V elements at two places a lane (a rotated element and
// its partner), whose sines a lane keeps for all heads. The groups share the work of the sines, and the first q heads are
// loaded before them (8191 tokens x 64 heads of 128: 60 us before both, 57 after). More slices of a token than the card
// needs repeat that start (two: 66 us, four: 76). Into pools, two heads of a group at once and 6 CTAs on an SM (7000 tokens,
// bf16: 39.6 us; four heads: 41.6 with 4 CTAs, 44 with 5); rotation alone, four heads and 5 CTAs (57 us; 60 to 62 so).
//
// k and v rows into blocks go head by head: a CTA takes a tile of T tokens of a request, T a whole number of blocks,
// aligned in the cache, so that all rows of a block are in one CTA. It computes the sines of the tile once for all heads,
// then each warp takes whole heads and goes over their rows twice, for the largest magnitudes and for the codes; rows of a
// tile that fits the registers are loaded once. Both kinds of work are CTAs of one launch.
#include <cmath>

#include "pd_host.h"
#include "pd_rows.cuh"

namespace pd {
namespace {

constexpr int kFlagBadNewRows = PD_FLAG_BAD_NEW_ROWS;
// Pools that a call writes: none (rotated k rows go to k_out), of the rows' type, E4M3 codes with a scale per kv head,
// E4M3 codes with a scale per block.
enum Pool { kNone, kPlain, kHeadScales, kBlockScales };

constexpr float kTop = 448.f, kEdge = 464.f;  // the largest code; the least magnitude that no longer rounds to it
constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126: the scale of a block of zeros
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kMaxTile = 64;   // tokens of a tile
constexpr int kMaxBlocks = 16;  // blocks of a tile

struct NormArgs {
    const void* q;
    const void* k;
    const void* v;
    void* q_out;
    void* k_out;  // kNone
    long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;  // elements between tokens
    int hq, hk;
    const void* q_weight;  // null: ones
    const void* k_weight;
    float eps;  // 0: no norms
    const int32_t* positions;  // null: the token's index in its request's cache
    const uint64_t* freqs;
    float scale;
    int head_dim, rot_dim;
    int tokens, slices;            // slices of a token's heads
    int tile, kv_slices, kv_ctas;  // block scales: tokens of a tile, slices of its k and v heads, CTAs that take them
    // the pool and its table
    void* k_data;
    void* v_data;
    float* k_scale;  // written with block scales
    float* v_scale;
    const int32_t* indices;
    const int32_t* indptr;
    const int32_t* last_page_len;
    const int32_t* new_indptr;
    int batch, page_size, num_total_pages, num_indices;
    int block;  // tokens of a block
    int* flags;
};

// The greatest b with new_indptr[b] / tile + 2 b <= c: request b's tiles lie from there on, n / tile + 2 of them at
// most. By a 32-way search; it ends with some b in [0, batch) on a malformed table too.
__device__ __forceinline__ int request_of_tile(const int32_t* new_indptr, int batch, int tile, int c, int lane) {
    int lo = 0, hi = batch;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const long long at = lo + (long long)(lane + 1) * step;
        const bool below = at < hi && max(0, __ldg(new_indptr + at)) / tile + 2 * at <= c;
        lo += __popc(__ballot_sync(kFull, below)) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

struct TileShared {
    int request, count, first;  // rows of the tile that are new; the first one's row in the ragged tensors
    int write, old_rows;        // whether rows go to the pool; rows of the tile's first block that were there before
    int pos[kMaxTile];
    long long dst[kMaxTile];    // pool row of kv head 0, in rows of head_dim; -1: a bad page
    long long old_dst;          // of the first old row
    unsigned most[kWarps][kMaxBlocks];  // largest magnitudes of a head's blocks, as the bits of an f32
    float inv[kWarps][kMaxBlocks];      // 1 / scale
};

// Codes of f[i] * inv.
template <int V>
__device__ __forceinline__ void store_codes_by(uint8_t* p, const float (&f)[V], float inv) {
    if constexpr (V == 1) {
        *p = __nv_cvt_float_to_fp8(f[0] * inv, __NV_SATFINITE, __NV_E4M3);
    } else {
        uint32_t w[V / 4] = {};
#pragma unroll
        for (int i = 0; i < V; i += 2)
            w[i / 4] |= uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(f[i] * inv, f[i + 1] * inv), __NV_SATFINITE, __NV_E4M3)) << (8 * (i % 4));
        if constexpr (V == 8)
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t*>(p) = w[0];
    }
}

// Where lanes are in a row of D elements: L lanes to a row (a power of two), units of V elements at e0 and V at e1.
// kUnits: units of a row per lane (V = 1 has more units than a warp has lanes).
template <int V, bool kPairs, int kUnits>
struct Places {
    int L, rows, lu, lr;  // lanes of a row, rows at once; this lane's place in its row, and its row
    int e0[kUnits], e1[kUnits];
    bool on[kUnits];
    __device__ __forceinline__ Places(int D, int rot, int lane) {
        const int units = D / (2 * V), rotated = rot / (2 * V);
        L = 1;
        while (L < min(units, 32)) L *= 2;
        rows = 32 / L, lu = lane & (L - 1), lr = lane / L;
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            const int u = lu + 32 * j;
            on[j] = u < units;
            if (u < rotated) {
                e0[j] = kPairs && V == 1 ? 2 * u : u * V;
                e1[j] = kPairs && V == 1 ? 2 * u + 1 : rot / 2 + u * V;
            } else {
                e0[j] = rot + (u - rotated) * 2 * V;
                e1[j] = e0[j] + V;
            }
        }
    }
};

// The pair that element i of unit u belongs to: (x[i], y[i]) in the half layout; neighbours of x, then of y, in the pairs
// layout.
template <int V, bool kPairs>
__device__ __forceinline__ int pair_of(int u, int i, int rot) {
    return !kPairs || V == 1 ? u * V + i : i % (V > 1 ? V / 2 : 1) + u * (V / 2) + (2 * i < V ? 0 : rot / 4);
}

__device__ __forceinline__ float2 turn_of(int pos, uint64_t freq, float scale) {
    const uint64_t turn = uint64_t(int64_t(pos)) * freq;
    float sn, cs;
    // int32 -> f32 rounds the phase by at most 2^-25 of half a turn
    sincospif(float(int32_t(uint32_t(turn >> 32))) * 4.656612873077393e-10f, &sn, &cs);
    return make_float2(cs * scale, sn * scale);
}

// The pairs of x and y turned; turn(i): cos and sin of pair i of the unit.
template <int V, bool kPairs, class F>
__device__ __forceinline__ void rotate(float (&x)[V], float (&y)[V], F turn) {
    float lo[V], hi[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float2 t = turn(i);
        if constexpr (kPairs && V > 1) {
            float(&f)[V] = 2 * i < V ? x : y;
            float(&o)[V] = 2 * i < V ? lo : hi;
            o[2 * i % V] = f[2 * i % V] * t.x - f[(2 * i + 1) % V] * t.y;
            o[(2 * i + 1) % V] = f[(2 * i + 1) % V] * t.x + f[2 * i % V] * t.y;
        } else {
            lo[i] = x[i] * t.x - y[i] * t.y;
            hi[i] = y[i] * t.x + x[i] * t.y;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        x[i] = lo[i];
        y[i] = hi[i];
    }
}

// x and y over the root of their row's mean square, times the weights. By all lanes of a row.
template <int V, int kUnits>
__device__ __forceinline__ void normalise(float (&x)[kUnits][V], float (&y)[kUnits][V], const float (&w0)[kUnits][V],
                                          const float (&w1)[kUnits][V], int L, float inv_dim, float eps) {
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < kUnits; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fmaf(x[j][i], x[j][i], fmaf(y[j][i], y[j][i], ss));
    for (int off = 1; off < L; off <<= 1) ss += __shfl_xor_sync(kFull, ss, off);
    const float by = rsqrtf(fmaf(ss, inv_dim, eps));
#pragma unroll
    for (int j = 0; j < kUnits; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[j][i] *= by * w0[j][i];
            y[j][i] *= by * w1[j][i];
        }
}

// Heads that pass through: one warp per (token, slice of its heads).
template <typename T, int V, bool kPairs, int kPool>
__device__ __forceinline__ void token_heads(const NormArgs& a, long long w) {
    constexpr int kUnits = V == 1 ? 4 : 1, kRound = V == 1 || kPool == kPlain || kPool == kHeadScales ? 2 : 4;
    const int lane = threadIdx.x & 31;
    const int t = int(w / a.slices), slice = int(w % a.slices);
    const int D = a.head_dim, rot = a.rot_dim, rotated = rot / (2 * V);
    const int items = a.hq + (kPool == kNone ? a.hk : kPool == kBlockScales ? 0 : 2 * a.hk);
    const int i0 = int((long long)items * slice / a.slices), i1 = int((long long)items * (slice + 1) / a.slices);
    const bool wants_kv = (kPool == kPlain || kPool == kHeadScales) && i1 > a.hq;

    const Places<V, kPairs, kUnits> at(D, rot, lane);
    Raw<T, V> xs[kRound][kUnits], ys[kRound][kUnits];
    // A round of heads [h, h1): kRound of each group of lanes.
    auto fetch = [&](const T* src, int h, int h1) {
#pragma unroll
        for (int r = 0; r < kRound; ++r)
#pragma unroll
            for (int j = 0; j < kUnits; ++j)
                if (h + r * at.rows < h1 && at.on[j]) {
                    const T* row = src + (long long)(h + r * at.rows) * D;
                    xs[r][j] = *reinterpret_cast<const Raw<T, V>*>(row + at.e0[j]);
                    ys[r][j] = *reinterpret_cast<const Raw<T, V>*>(row + at.e1[j]);
                }
    };
    // The first q heads are on their way while the table is read and the sines are computed.
    const int q1 = min(i1, a.hq);
    const T* q_row = static_cast<const T*>(a.q) + t * a.q_stride;
    if (i0 < q1) fetch(q_row, i0 + at.lr, q1);

    // ---- where this token's k and v rows go (offset in elements of kv head 0), and its position
    int pos = 0;
    bool write_kv = false;
    size_t dst = 0;
    const size_t head_step = size_t(a.page_size) * D;
    if (kPool != kNone && (wants_kv || a.positions == nullptr)) {
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

    float2 turns[kUnits][V];
    auto turn = [&](int u, int i) {
        return u < rotated ? turn_of(pos, __ldg(a.freqs + pair_of<V, kPairs>(u, i, rot)), a.scale) : make_float2(1.f, 0.f);
    };
    // The groups of lanes hold the same pairs of different heads: each of kGroups computes its share of the sines.
    auto share = [&](auto groups) {
        constexpr int kGroups = decltype(groups)::value;
        float2 mine[V / kGroups > 0 ? V / kGroups : 1];
#pragma unroll
        for (int i = 0; i < V / kGroups; ++i) mine[i] = turn(at.lu, i * kGroups + (at.lr & (kGroups - 1)));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int from = i % kGroups * at.L + at.lu;
            turns[0][i] = make_float2(__shfl_sync(kFull, mine[i / kGroups].x, from), __shfl_sync(kFull, mine[i / kGroups].y, from));
        }
    };
    if (V > 1 && at.rows >= 4)
        share(std::integral_constant<int, (V > 1 ? 4 : 1)>{});
    else if (V > 1 && at.rows == 2)
        share(std::integral_constant<int, (V > 1 ? 2 : 1)>{});
    else
#pragma unroll
        for (int j = 0; j < kUnits; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) turns[j][i] = turn(at.lu + 32 * j, i);
    const float inv_dim = 1.f / float(D);
    // Heads [h0, h1) of one kind: q, k or v.
    auto run = [&](int h0, int h1, const T* src, const void* weight, auto kind) {
        constexpr int kKind = decltype(kind)::value;  // 0: q, 1: k, 2: v
        float w0[kUnits][V], w1[kUnits][V];
        if constexpr (kKind < 2) {
            const T* from = static_cast<const T*>(weight);
#pragma unroll
            for (int j = 0; j < kUnits; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    w0[j][i] = from != nullptr && at.on[j] ? float(from[at.e0[j] + i]) : 1.f;
                    w1[j][i] = from != nullptr && at.on[j] ? float(from[at.e1[j] + i]) : 1.f;
                }
        }
        for (int h = h0 + at.lr; h - at.lr < h1; h += at.rows * kRound) {
            if (kKind != 0 || h - at.lr != h0) fetch(src, h, h1);
#pragma unroll
            for (int r = 0; r < kRound; ++r) {
                const int head = h + r * at.rows;
                if (head - at.lr >= h1) break;  // (the whole warp)
                const bool there = head < h1;
                if constexpr (kPool == kPlain && kKind == 2) {  // every bit as it came
                    T* p = static_cast<T*>(a.v_data) + dst + head * head_step;
#pragma unroll
                    for (int j = 0; j < kUnits; ++j)
                        if (there && at.on[j]) {
                            *reinterpret_cast<Raw<T, V>*>(p + at.e0[j]) = xs[r][j];
                            *reinterpret_cast<Raw<T, V>*>(p + at.e1[j]) = ys[r][j];
                        }
                } else {
                    float x[kUnits][V], y[kUnits][V];
#pragma unroll
                    for (int j = 0; j < kUnits; ++j) {
                        if (there && at.on[j]) {
                            widen<T, V>(xs[r][j], x[j]);
                            widen<T, V>(ys[r][j], y[j]);
                        } else {
#pragma unroll
                            for (int i = 0; i < V; ++i) x[j][i] = y[j][i] = 0.f;
                        }
                    }
                    if constexpr (kKind < 2) {
                        if (kPool != kBlockScales || a.eps > 0.f) normalise<V, kUnits>(x, y, w0, w1, at.L, inv_dim, a.eps);
#pragma unroll
                        for (int j = 0; j < kUnits; ++j)
                            if (at.lu + 32 * j < rotated) rotate<V, kPairs>(x[j], y[j], [&](int i) { return turns[j][i]; });
                    }
                    if (!there) continue;
                    if constexpr (kPool == kHeadScales && kKind > 0) {
                        uint8_t* p = static_cast<uint8_t*>(kKind == 2 ? a.v_data : a.k_data) + dst + head * head_step;
                        const float scale = __ldg((kKind == 2 ? a.v_scale : a.k_scale) + head);
#pragma unroll
                        for (int j = 0; j < kUnits; ++j)
                            if (at.on[j]) {
                                store_codes<V>(p + at.e0[j], x[j], scale);
                                store_codes<V>(p + at.e1[j], y[j], scale);
                            }
                    } else {
                        T* p = kKind == 0       ? static_cast<T*>(a.q_out) + t * a.q_out_stride + (long long)head * D
                               : kPool == kNone ? static_cast<T*>(a.k_out) + t * a.k_out_stride + (long long)head * D
                                                : static_cast<T*>(a.k_data) + dst + head * head_step;
#pragma unroll
                        for (int j = 0; j < kUnits; ++j)
                            if (kPool == kBlockScales && at.on[j] && !(a.eps > 0.f) && at.lu + 32 * j >= rotated) {
                                *reinterpret_cast<Raw<T, V>*>(p + at.e0[j]) = xs[r][j];  // every bit as it came
                                *reinterpret_cast<Raw<T, V>*>(p + at.e1[j]) = ys[r][j];
                            } else if (at.on[j]) {
                                store_elems<T, V>(p + at.e0[j], x[j]);
                                store_elems<T, V>(p + at.e1[j], y[j]);
                            }
                    }
                }
            }
        }
    };
    if (i0 < q1) run(i0, q1, q_row, a.q_weight, std::integral_constant<int, 0>{});
    if constexpr (kPool != kBlockScales) {
        if (kPool != kNone && !write_kv) return;
        const int k0 = max(i0 - a.hq, 0), k1 = min(i1 - a.hq, a.hk);
        if (k0 < k1) run(k0, k1, static_cast<const T*>(a.k) + t * a.k_stride, a.k_weight, std::integral_constant<int, 1>{});
    }
    if constexpr (kPool == kPlain || kPool == kHeadScales) {
        const int v0 = max(i0 - a.hq - a.hk, 0), v1 = i1 - a.hq - a.hk;
        if (v0 < v1) run(v0, v1, static_cast<const T*>(a.v) + t * a.v_stride, nullptr, std::integral_constant<int, 2>{});
    }
}

// k and v heads of a tile into blocks.
template <typename T, int V, bool kPairs>
__device__ __forceinline__ void tile_blocks(const NormArgs& a, float* turns, TileShared& sh) {
    constexpr int kUnits = V == 1 ? 4 : 1, kRound = V == 1 ? 2 : 4;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int c = int(blockIdx.x) / a.kv_slices, slice = int(blockIdx.x) - c * a.kv_slices;
    const int D = a.head_dim, rot = a.rot_dim, T_ = a.tile;
    const int rotated = rot / (2 * V);  // units that are rotated; the rest follow

    // Each request's range is checked by a tile of its number (there are two and more for each): a row that is no request's,
    // or two's, is in nobody's tile or in two.
    if (tid == 32 && slice == 0 && c < a.batch) {
        const int s = __ldg(a.new_indptr + c), e = __ldg(a.new_indptr + c + 1);
        if (s < 0 || e < s || e > a.tokens || (c == 0 && s != 0) || (c == a.batch - 1 && e != a.tokens)) atomicOr(a.flags, kFlagBadNewRows);
    }
    // ---- the tile's rows
    if (wid == 0) {
        int count = 0, first = 0, write = 0, old = 0, bad = 0, cache0 = 0, lo = 0;
        {
            const int b = request_of_tile(a.new_indptr, a.batch, T_, c, lane);
            const int s = __ldg(a.new_indptr + b), e = __ldg(a.new_indptr + b + 1);
            const int hi = __ldg(a.indptr + b + 1), last = __ldg(a.last_page_len + b);
            lo = __ldg(a.indptr + b);
            if (s < 0 || e < s || e > a.tokens) {
                bad = kFlagBadNewRows;
            } else {
                const int n = e - s;
                long long ctx = 0;  // tokens before the new ones
                if (n > 0) {
                    if (lo < 0 || hi <= lo || hi > a.num_indices)
                        bad = kFlagBadIndptr;
                    else if (last < 0 || last > a.page_size)
                        bad = kFlagBadLastPageLen;
                    else {
                        ctx = ((long long)hi - lo - 1) * a.page_size + last - n;
                        if (ctx < 0 || ctx + n > 0x7fffffff) bad = kFlagBadNewRows;
                    }
                    if (bad != 0) ctx = 0;
                }
                const int nth = c - (s / T_ + 2 * b);  // tile of the request
                const long long t0 = max(ctx, (ctx / T_ + nth) * T_), t1 = min(ctx + n, (ctx / T_ + nth + 1) * T_);
                if (t1 > t0) {
                    count = int(t1 - t0);
                    first = s + int(t0 - ctx);
                    write = bad == 0;
                    cache0 = int(t0);
                    if (nth == 0) old = int(ctx % a.block);
                }
            }
        }
        if (bad != 0 && lane == 0 && slice == 0) atomicOr(a.flags, bad);
        if (lane == 0) {
            sh.count = count;
            sh.first = first;
            sh.write = write;
            sh.old_rows = old;
        }
        for (int r = lane; r < count; r += 32) {
            const int t = cache0 + r;
            long long dst = -1;
            if (write) {
                const int nth = t / a.page_size, row = t - nth * a.page_size;
                const int page = __ldg(a.indices + lo + nth);
                if (page >= 0 && page < a.num_total_pages)
                    dst = (long long)page * a.hk * a.page_size + row;
                else if (slice == 0)
                    atomicOr(a.flags, kFlagBadPage);
            }
            sh.dst[r] = dst;
            sh.pos[r] = a.positions != nullptr ? __ldg(a.positions + first + r) : t;
        }
    }
    __syncthreads();
    const int count = sh.count, first = sh.first;
    if (count == 0 || !sh.write) return;
    const Places<V, kPairs, kUnits> at(D, rot, lane);
    const int steps = (count + at.rows - 1) / at.rows;
    const bool norm = a.eps > 0.f;
    const float inv_dim = 1.f / float(D);
    const size_t head_rows = size_t(a.page_size);  // pool rows between kv heads
    const int k0 = int((long long)2 * a.hk * slice / a.kv_slices), k1 = int((long long)2 * a.hk * (slice + 1) / a.kv_slices);
    bool is_v = false;
    int h = 0;
    const T* src = nullptr;
    long long stride = 0;
    float w0[kUnits][V], w1[kUnits][V];  // the weights at this lane's places
    Raw<T, V> xs[kRound][kUnits], ys[kRound][kUnits];
    auto begin = [&](int item) {
        is_v = item >= a.hk;
        h = is_v ? item - a.hk : item;
        src = static_cast<const T*>(is_v ? a.v : a.k);
        stride = is_v ? a.v_stride : a.k_stride;
        src += first * stride + (long long)h * D;
    };
    auto load = [&](int step0) {
#pragma unroll
        for (int r = 0; r < kRound; ++r) {
            const int row = (step0 + r) * at.rows + at.lr;
#pragma unroll
            for (int j = 0; j < kUnits; ++j)
                if (row < count && at.on[j]) {
                    xs[r][j] = *reinterpret_cast<const Raw<T, V>*>(src + row * stride + at.e0[j]);
                    ys[r][j] = *reinterpret_cast<const Raw<T, V>*>(src + row * stride + at.e1[j]);
                }
        }
    };
    // The first head's rows are on their way while the sines are computed.
    if (k0 + wid < k1) {
        begin(k0 + wid);
        load(0);
    }
#pragma unroll
    for (int j = 0; j < kUnits; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const T* weight = static_cast<const T*>(a.k_weight);
            w0[j][i] = weight != nullptr && at.on[j] ? float(weight[at.e0[j] + i]) : 1.f;
            w1[j][i] = weight != nullptr && at.on[j] ? float(weight[at.e1[j] + i]) : 1.f;
        }
    // ---- cos and sin of every row and pair, in the order in which lanes read them: V / 2 pieces of two pairs per unit
    for (int x = tid; x < count * rotated * V; x += kThreads) {
        const int i = x % V, ru = x / V, r = ru / rotated, u = ru - r * rotated;
        const int place = V == 1 ? ru : ((r * (V / 2 > 0 ? V / 2 : 1) + i / 2) * rotated + u) * 2 + (i & 1);
        reinterpret_cast<float2*>(turns)[place] = turn_of(sh.pos[r], __ldg(a.freqs + pair_of<V, kPairs>(u, i, rot)), a.scale);
    }
    __syncthreads();
    // The f32 values of a row that was loaded as round r (all lanes call it).
    auto values = [&](int r, int row, float(&x)[kUnits][V], float(&y)[kUnits][V]) {
        const bool there = row < count;
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            if (there && at.on[j]) {
                widen<T, V>(xs[r][j], x[j]);
                widen<T, V>(ys[r][j], y[j]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) x[j][i] = y[j][i] = 0.f;
            }
        }
        if (is_v) return;
        if (norm) normalise<V, kUnits>(x, y, w0, w1, at.L, inv_dim, a.eps);
        if (!there) return;
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            const int u = at.lu + 32 * j;
            if (u >= rotated) continue;
            rotate<V, kPairs>(x[j], y[j], [&](int i) {
                if constexpr (V == 1) return reinterpret_cast<const float2*>(turns)[row * rotated + u];
                const float4 t = reinterpret_cast<const float4*>(turns)[(row * (V > 1 ? V / 2 : 1) + i / 2) * rotated + u];
                return i % 2 == 0 ? make_float2(t.x, t.y) : make_float2(t.z, t.w);
            });
        }
    };
    const int old = sh.old_rows;  // new row r is row old + r of the tile's blocks
    const int nblk = (old + count + a.block - 1) / a.block;
    // The scales of a head's blocks from their largest magnitudes, a lane for each block; then its older rows, if the first
    // one's scale grew.
    auto settle = [&](unsigned* most_of, float* inv_of) {
        uint8_t* pool = static_cast<uint8_t*>(is_v ? a.v_data : a.k_data);
        int grow = 0;  // of the first block, whose older rows it touches
        if (lane < nblk) {
            const int r0 = max(0, lane * a.block - old);  // the block's first new row
            const long long dst = sh.dst[r0];
            float inv = 0.f;
            if (dst >= 0) {
                const long long page = dst / (a.hk * (long long)a.page_size);
                const int row = int(dst - page * a.hk * a.page_size), per = a.page_size / a.block;
                float* at = (is_v ? a.v_scale : a.k_scale) + (page * a.hk + h) * per + row / a.block;
                const float most = __uint_as_float(most_of[lane]);
                float s;
                if (lane == 0 && old > 0) {
                    const float was = fmaxf(*at, kLeastScale);
                    s = was;
                    const float limit = kEdge * was;
                    if (most > limit) {  // (by exponents: the quotient may be past the largest f32)
                        int em, el;
                        const float fm = frexpf(most, &em), fl = frexpf(limit, &el);
                        grow = em - el + (fm > fl ? 1 : 0);
                        s = scalbnf(was, grow);
                    }
                    if (s != *at) *at = s;
                } else {
                    s = fmaxf(most / kTop, kLeastScale);
                    *at = s;
                }
                inv = 1.f / s;
            }
            inv_of[lane] = inv;
        }
        grow = __shfl_sync(kFull, grow, 0);
        if (grow > 0) {  // the older rows, 8 codes a lane
            const float by = scalbnf(1.f, -grow);
            uint8_t* rows = pool + (size_t(sh.dst[0]) - old + h * head_rows) * D;
            for (int x = lane * 8; x < old * D; x += 256) {
                float f[8];
                e4m3x8_to_f32(*reinterpret_cast<const uint2*>(rows + x), f);
                store_codes_by<8>(rows + x, f, by);
            }
        }
    };
    auto magnitude = [&](const float(&x)[kUnits][V], const float(&y)[kUnits][V]) {
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < kUnits; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float p = fabsf(x[j][i]), q = fabsf(y[j][i]);
                top = fmaxf(top, p <= 3.402823466e38f ? p : 0.f);  // infinities and NaN have no say
                top = fmaxf(top, q <= 3.402823466e38f ? q : 0.f);
            }
        for (int off = 1; off < at.L; off <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
        return top;
    };
    auto write = [&](int row, const float(&x)[kUnits][V], const float(&y)[kUnits][V], const float* inv_of) {
        if (row >= count || sh.dst[row] < 0) return;
        const float inv = inv_of[(old + row) / a.block];
        uint8_t* p = static_cast<uint8_t*>(is_v ? a.v_data : a.k_data) + (size_t(sh.dst[row]) + h * head_rows) * D;
#pragma unroll
        for (int j = 0; j < kUnits; ++j)
            if (at.on[j]) {
                store_codes_by<V>(p + at.e0[j], x[j], inv);
                store_codes_by<V>(p + at.e1[j], y[j], inv);
            }
    };
    for (int item = k0 + wid; item < k1; item += kWarps) {
        const bool loaded = item == k0 + wid && steps <= kRound;
        begin(item);
        if (lane < kMaxBlocks) sh.most[wid][lane] = 0u;
        __syncwarp();
        for (int s0 = 0; s0 < steps; s0 += kRound) {
            if (!loaded) load(s0);
#pragma unroll
            for (int r = 0; r < kRound; ++r) {
                const int row = (s0 + r) * at.rows + at.lr;
                if (s0 + r >= steps) break;
                float x[kUnits][V], y[kUnits][V];
                values(r, row, x, y);
                const float top = magnitude(x, y);
                if (at.lu == 0 && row < count) atomicMax(&sh.most[wid][(old + row) / a.block], __float_as_uint(top));
            }
        }
        __syncwarp();
        settle(sh.most[wid], sh.inv[wid]);
        __syncwarp();
        for (int s0 = 0; s0 < steps; s0 += kRound) {
            if (steps > kRound) load(s0);
#pragma unroll
            for (int r = 0; r < kRound; ++r) {
                const int row = (s0 + r) * at.rows + at.lr;
                if (s0 + r >= steps) break;
                float x[kUnits][V], y[kUnits][V];
                values(r, row, x, y);
                write(row, x, y, sh.inv[wid]);
            }
        }
        __syncwarp();  // the next head uses the same places
    }
}

template <typename T, int V, bool kPairs, int kPool>
__global__ void __launch_bounds__(kThreads, kPool == kBlockScales ? 4 : kPool == kNone ? 5 : 6)
    norm_rope_kernel(const NormArgs a) {
    if constexpr (kPool == kBlockScales) {
        extern __shared__ __align__(16) float turns[];  // cos, sin of the tile's rows and pairs
        __shared__ TileShared sh;
        if (int(blockIdx.x) < a.kv_ctas) {
            tile_blocks<T, V, kPairs>(a, turns, sh);
            return;
        }
    }
    const long long w = (long long)(int(blockIdx.x) - a.kv_ctas) * kWarps + (threadIdx.x >> 5);
    if (w < (long long)a.tokens * a.slices) token_heads<T, V, kPairs, kPool>(a, w);
}

template <typename T, int V, bool kPairs>
const void* pick_pool(int pool) {
    switch (pool) {
        case kNone: return reinterpret_cast<const void*>(norm_rope_kernel<T, V, kPairs, kNone>);
        case kPlain: return reinterpret_cast<const void*>(norm_rope_kernel<T, V, kPairs, kPlain>);
    }
    if constexpr (sizeof(T) == 2)
        return pool == kHeadScales ? reinterpret_cast<const void*>(norm_rope_kernel<T, V, kPairs, kHeadScales>)
                                   : reinterpret_cast<const void*>(norm_rope_kernel<T, V, kPairs, kBlockScales>);
    return nullptr;
}

template <typename T>
const void* pick(int pool, int layout, bool wide) {
    constexpr int kVec = Elt<T>::kVec;
    if (layout == PD_ROPE_PAIRS) return wide ? pick_pool<T, kVec, true>(pool) : pick_pool<T, 1, true>(pool);
    return wide ? pick_pool<T, kVec, false>(pool) : pick_pool<T, 1, false>(pool);
}

pd_status launch(NormArgs& a, pd_dtype dt, Pool pool, int layout, cudaStream_t stream) {
    const int vec = dt == PD_F32 ? 4 : 8;
    const auto fits = [&](const void* p, long long stride) {
        return p == nullptr || (host::aligned(p, 16) && stride % vec == 0);
    };
    const bool wide = a.rot_dim % (2 * vec) == 0 && a.head_dim % (2 * vec) == 0 && fits(a.q, a.q_stride) && fits(a.q_out, a.q_out_stride) &&
                      fits(a.k, a.k_stride) && fits(a.k_out, a.k_out_stride) && fits(a.v, a.v_stride);
    int sms = 0;
    pd_status st = host::sm_count(&sms);
    if (st != PD_OK) return st;
    // Few tokens: a token's heads in slices, so that the card has about 8 warps per SM (see pd_rope.cu).
    const int items = a.hq + (pool == kNone ? a.hk : pool == kBlockScales ? 0 : 2 * a.hk);
    const long long want = ((long long)sms * 8 + a.tokens - 1) / a.tokens, most = (items + 3) / 4;
    a.slices = int(want < 1 || most < 1 ? 1 : want > most ? most : want);
    const long long warps = items > 0 ? (long long)a.tokens * a.slices : 0;
    // Tiles: their k and v heads in slices of whole rounds of a CTA's warps, for about 4 CTAs per SM.
    long long kv = 0;
    int smem = 0;
    if (pool == kBlockScales) {
        a.tile = a.block * (a.block < 16 ? 16 / a.block : 1);
        const long long tiles = (long long)a.tokens / a.tile + 2ll * a.batch, rounds = (2ll * a.hk + kWarps - 1) / kWarps;
        const long long cut = ((long long)sms * 4 + tiles - 1) / tiles;
        long long each = cut >= rounds ? 1 : (rounds + cut - 1) / cut;  // rounds of a slice
        while (rounds % each != 0) ++each;
        a.kv_slices = int(rounds / each);
        kv = tiles * a.kv_slices;
        smem = a.tile * a.rot_dim / 2 * 8;
    }
    const long long ctas = kv + (warps + kWarps - 1) / kWarps;
    if (ctas > 0x7fffffff) return host::fail(PD_ERR_INVALID, "batch and the number of tokens are too large");
    a.kv_ctas = int(kv);
    const void* fn = dt == PD_F32   ? pick<float>(pool, layout, wide)
                     : dt == PD_F16 ? pick<__half>(pool, layout, wide)
                                    : pick<__nv_bfloat16>(pool, layout, wide);
    if (smem > 40 * 1024 && (st = host::allow_smem(fn, smem)) != PD_OK) return st;
    void* args[] = {&a};
    const cudaError_t e = cudaLaunchKernel(fn, dim3(unsigned(ctas)), dim3(kThreads), args, size_t(smem), stream);
    return e == cudaSuccess ? host::ok() : host::cuda_fail(e, "norm and rotation launch");
}

pd_status check_norm(float eps, const void* q_weight, const void* k_weight, size_t elem) {
    if (!(eps > 0.f) || !std::isfinite(eps)) return host::fail(PD_ERR_INVALID, "eps must be finite and positive");
    if (!host::aligned(q_weight, elem) || !host::aligned(k_weight, elem))
        return host::fail(PD_ERR_UNSUPPORTED, "q_weight and k_weight must be aligned to their element");
    return PD_OK;
}

pd_status append_impl(const void* q, const void* k_new, const void* v_new, const void* q_weight, const void* k_weight,
                      const int32_t* positions, const uint64_t* freqs, void* q_out, float* k_scale, float* v_scale,
                      void* k_data, void* v_data, const int32_t* indices, const int32_t* indptr,
                      const int32_t* last_page_len, const int32_t* new_indptr, int batch, int total_new, int Hq, int Hk,
                      int D, int rot_dim, int page_size, int num_total_pages, int num_indices, int block,
                      long long q_stride, long long k_stride, long long v_stride, float eps, int layout,
                      float rope_scale, pd_dtype dt, void* workspace, size_t workspace_bytes, void* stream, Pool pool) {
    if (D != 64 && D != 128 && D != 256) return host::fail(PD_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256 (got %d)", D);
    pd_status st = host::check_rotation(total_new, D, rot_dim, layout, rope_scale, freqs, dt);
    if (st != PD_OK) return st;
    if (pool != kPlain && dt == PD_F32) return host::fail(PD_ERR_UNSUPPORTED, "E4M3 pools take PD_F16 or PD_BF16 rows");
    const size_t e = host::elem_size(dt);
    if (pool == kBlockScales && eps == 0.f) {
        if (q_weight || k_weight) return host::fail(PD_ERR_INVALID, "eps = 0 leaves the norms out: q_weight and k_weight must be null");
    } else if ((st = check_norm(eps, q_weight, k_weight, e)) != PD_OK) {
        return st;
    }
    if (batch <= 0 || Hk <= 0 || page_size <= 0 || num_total_pages <= 0)
        return host::fail(PD_ERR_INVALID, "batch, num_kv_heads, page_size and num_total_pages must be positive");
    if (pool == kBlockScales && (st = host::check_block(block, page_size)) != PD_OK) return st;
    if (num_indices < 0 || Hq < 0 || Hq > (1 << 20) || Hk > (1 << 20) || batch > (1 << 28))
        return host::fail(PD_ERR_INVALID, "num_indices and num_qo_heads must not be negative, heads at most 2^20, batch at most 2^28");
    if (!k_data || !v_data || !indptr || !last_page_len || !new_indptr || (num_indices > 0 && !indices) ||
        (total_new > 0 && (!k_new || !v_new || (Hq > 0 && (!q || !q_out)))) || (pool != kPlain && (!k_scale || !v_scale)))
        return host::fail(PD_ERR_INVALID, "null pointer argument");
    if (k_stride < (long long)Hk * D || v_stride < (long long)Hk * D || (Hq > 0 && q_stride < (long long)Hq * D))
        return host::fail(PD_ERR_INVALID, "a token's stride must hold its heads");
    // (one token lies where it lies whatever its stride)
    if (Hq > 0 && total_new > 1 && q == q_out && q_stride != (long long)Hq * D)
        return host::fail(PD_ERR_INVALID, "q_out may be q only where q_stride is num_qo_heads * head_dim");
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
    NormArgs a{};
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
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.eps = eps;
    a.positions = positions;
    a.freqs = freqs;
    a.scale = rope_scale;
    a.head_dim = D;
    a.rot_dim = rot_dim;
    a.tokens = total_new;
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
    a.block = block;
    a.flags = static_cast<int*>(workspace);
    return launch(a, dt, pool, layout, static_cast<cudaStream_t>(stream));
}

}  // namespace

namespace host {

pd_status check_block(int block_tokens, int page_size) {
    if (block_tokens <= 0 || block_tokens > PD_MAX_BLOCK_TOKENS || page_size % block_tokens != 0)
        return fail(PD_ERR_INVALID, "block_tokens must be in [1, %d] and divide page_size (got %d of %d)", PD_MAX_BLOCK_TOKENS,
                    block_tokens, page_size);
    return PD_OK;
}

}  // namespace host
}  // namespace pd

using namespace pd;

extern "C" {

pd_status pd_norm_rope(const void* q, const void* k, const void* q_weight, const void* k_weight, const int32_t* positions,
                       const uint64_t* freqs, void* q_out, void* k_out, int num_tokens, int num_qo_heads,
                       int num_kv_heads, int head_dim, int rot_dim, int64_t q_stride, int64_t k_stride,
                       int64_t q_out_stride, int64_t k_out_stride, float eps, int layout, float rope_scale,
                       pd_dtype dtype, void* stream) {
    if (num_qo_heads <= 0 || num_kv_heads < 0 || num_qo_heads > (1 << 20) || num_kv_heads > (1 << 20))
        return host::fail(PD_ERR_INVALID, "num_qo_heads must be in [1, 2^20] and num_kv_heads in [0, 2^20]");
    if (head_dim <= 0 || head_dim % 2 != 0 || head_dim > 256)
        return host::fail(PD_ERR_UNSUPPORTED, "head_dim must be even and in [2, 256] (got %d)", head_dim);
    pd_status st = host::check_rotation(num_tokens, head_dim, rot_dim, layout, rope_scale, freqs, dtype);
    if (st != PD_OK) return st;
    const size_t e = host::elem_size(dtype);
    if ((st = check_norm(eps, q_weight, k_weight, e)) != PD_OK) return st;
    const bool with_k = num_kv_heads > 0;
    if (num_tokens > 0 && (!q || !q_out || (with_k && (!k || !k_out)) || (rot_dim > 0 && !positions)))
        return host::fail(PD_ERR_INVALID, "null pointer argument");
    const long long q_row = (long long)num_qo_heads * head_dim, k_row = (long long)num_kv_heads * head_dim;
    if (q_stride < q_row || q_out_stride < q_row || (with_k && (k_stride < k_row || k_out_stride < k_row)))
        return host::fail(PD_ERR_INVALID, "a token's stride must hold its heads");
    if (num_tokens > 1 && ((q == q_out && q_stride != q_out_stride) || (with_k && k == k_out && k_stride != k_out_stride)))
        return host::fail(PD_ERR_INVALID, "in place, both strides must be the same");
    if (!host::aligned(q, e) || !host::aligned(q_out, e) || !host::aligned(k, e) || !host::aligned(k_out, e) || !host::aligned(positions, 4))
        return host::fail(PD_ERR_UNSUPPORTED, "q, k and their outputs must be aligned to their element, positions to 4 bytes");
    if (num_tokens == 0) return host::ok();
    NormArgs a{};
    a.q = q;
    a.q_out = q_out;
    a.q_stride = q_stride;
    a.q_out_stride = q_out_stride;
    a.hq = num_qo_heads;
    a.k = with_k ? k : nullptr;
    a.k_out = with_k ? k_out : nullptr;
    a.k_stride = with_k ? k_stride : 0;
    a.k_out_stride = with_k ? k_out_stride : 0;
    a.hk = num_kv_heads;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.eps = eps;
    a.positions = positions;
    a.freqs = freqs;
    a.scale = rope_scale;
    a.head_dim = head_dim;
    a.rot_dim = rot_dim;
    a.tokens = num_tokens;
    return launch(a, dtype, kNone, layout, static_cast<cudaStream_t>(stream));
}

pd_status pd_paged_norm_rope_append(const void* q, const void* k_new, const void* v_new, const void* q_weight,
                                    const void* k_weight, const int32_t* positions, const uint64_t* freqs, void* q_out,
                                    void* k_data, void* v_data, const int32_t* indices, const int32_t* indptr,
                                    const int32_t* last_page_len, const int32_t* new_indptr, int batch, int total_new,
                                    int num_qo_heads, int num_kv_heads, int head_dim, int rot_dim, int page_size,
                                    int num_total_pages, int num_indices, int64_t q_stride, int64_t k_stride,
                                    int64_t v_stride, float eps, int layout, float rope_scale, pd_dtype dtype,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    return append_impl(q, k_new, v_new, q_weight, k_weight, positions, freqs, q_out, nullptr, nullptr, k_data, v_data,
                       indices, indptr, last_page_len, new_indptr, batch, total_new, num_qo_heads, num_kv_heads, head_dim,
                       rot_dim, page_size, num_total_pages, num_indices, 0, q_stride, k_stride, v_stride, eps, layout,
                       rope_scale, dtype, workspace, workspace_bytes, stream, kPlain);
}

pd_status pd_paged_norm_rope_append_fp8(const void* q, const void* k_new, const void* v_new, const void* q_weight,
                                        const void* k_weight, const int32_t* positions, const uint64_t* freqs,
                                        void* q_out, const float* k_scale, const float* v_scale, void* k_data,
                                        void* v_data, const int32_t* indices, const int32_t* indptr,
                                        const int32_t* last_page_len, const int32_t* new_indptr, int batch,
                                        int total_new, int num_qo_heads, int num_kv_heads, int head_dim, int rot_dim,
                                        int page_size, int num_total_pages, int num_indices, int64_t q_stride,
                                        int64_t k_stride, int64_t v_stride, float eps, int layout, float rope_scale,
                                        pd_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
    return append_impl(q, k_new, v_new, q_weight, k_weight, positions, freqs, q_out, const_cast<float*>(k_scale),
                       const_cast<float*>(v_scale), k_data, v_data, indices, indptr, last_page_len, new_indptr, batch,
                       total_new, num_qo_heads, num_kv_heads, head_dim, rot_dim, page_size, num_total_pages, num_indices,
                       0, q_stride, k_stride, v_stride, eps, layout, rope_scale, dtype, workspace, workspace_bytes, stream,
                       kHeadScales);
}

pd_status pd_paged_rope_append_fp8_blocks(const void* q, const void* k_new, const void* v_new, const void* q_weight,
                                          const void* k_weight, const int32_t* positions, const uint64_t* freqs,
                                          void* q_out, float* k_scale, float* v_scale, void* k_data, void* v_data,
                                          const int32_t* indices, const int32_t* indptr, const int32_t* last_page_len,
                                          const int32_t* new_indptr, int batch, int total_new, int num_qo_heads,
                                          int num_kv_heads, int head_dim, int rot_dim, int page_size,
                                          int num_total_pages, int num_indices, int block_tokens, int64_t q_stride,
                                          int64_t k_stride, int64_t v_stride, float eps, int layout, float rope_scale,
                                          pd_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
    return append_impl(q, k_new, v_new, q_weight, k_weight, positions, freqs, q_out, k_scale, v_scale, k_data, v_data,
                       indices, indptr, last_page_len, new_indptr, batch, total_new, num_qo_heads, num_kv_heads, head_dim,
                       rot_dim, page_size, num_total_pages, num_indices, block_tokens, q_stride, k_stride, v_stride, eps,
                       layout, rope_scale, dtype, workspace, workspace_bytes, stream, kBlockScales);
}

}  // extern "C"
