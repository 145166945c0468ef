// Attention of several query tokens per request (a chain or a tree of drafted
// tokens, or a piece of a prompt) over a paged KV cache: the work partition
// and its walk, the merge of split segments, and the CUDA-core kernel.
//
// Segments. The rows of one request and one tile of q heads of a kv head (at
// most `hpt` heads) are cut into segments of up to `nps` nodes; a segment's
// rows share every K/V row that they read. Its keys are cut into blocks of
// `spb` slots of `slot_rows` tokens (a page is `cpp` slots; a page that is not
// a whole number of slots leaves rows of its last one unused). In a chain a
// segment's blocks end with its last node's own token.
//
// Partition. A segment costs its blocks and `seg_cost` units more (its q, its
// output), which lie before its first block. All segments, in the order
// (request, head tile, segment), are one line of U units, cut into shares of S
// = ceil(U / workers); a worker is a CTA, or one of the two halves of one. SMs
// stream at rates that differ by up to a quarter, so the last eighth of every
// share of 48 units or more is a range of its own that goes to whichever worker
// asks first when it comes to the end of what it has (64 ragged trees over an
// E4M3 pool 162 -> 145 us; shorter shares lose more to the longer merge: 32
// chains of 4, 62 -> 68 us). The cuts are fixed: results do not depend on who runs a
// range. A segment inside one range is written out there; one that is cut
// leaves a partial (o, lse) in each of its ranges, and the merge kernel combines
// them in order. Only the device knows the lengths: every CTA sums the requests'
// units itself (each thread a run of requests, one block-wide scan) and finds
// its shares; the range whose start is the first cut through a segment's blocks
// writes the merge's descriptor. After a wait that ran out a tail may have gone
// to nobody and its descriptor may be of another call: the merge reads none
// whose places it does not find in this call's partials and rows.
#pragma once

#include "pd_merge.cuh"

namespace pd {

constexpr int kFlagBadNewRows = 0x10;

struct TreeSplit {
    int parts;       // 0: nothing to merge
    int row0;        // the request's first q row + the segment's first node
    int nodes;       // nodes of the segment
    int hh;          // head tile
    int r0;          // range of the first part
    int slot0;       // its partial slot; part p > 0 is in slot 2 (r0 + p)
    int pad[2];      // 32 bytes: one sector each
};

struct TreeArgs {
    const void* q;
    const void* k;
    const void* v;
    const int32_t* indices;
    const int32_t* indptr;
    const int32_t* last_page_len;
    const int32_t* new_indptr;  // null: one node per request, and a request without tokens is no error
    const uint32_t* mask;  // null: a chain
    void* o;
    float* lse;
    const float* k_scale;  // E4M3 pools: of each kv head; block-scaled pools: [page][kv head][scales_per_page]
    const float* v_scale;
    int scales_per_page;
    FastDiv by_block;  // by the rows of a block
    int run;           // 16, 4 or 1: so many rows from a multiple of that on are of one block
    float* part_o;    // [2 * ranges][seg_rows][D], normalised
    float* part_lse;  // [2 * ranges][seg_rows], log2 units
    TreeSplit* splits;  // [ranges]; the first holds a TreeLine
    unsigned* claims;   // ranges asked for so far in this call; the merge sets it back to 0
    int* flags;
    int batch, total_new, mask_words, num_qo_heads, num_kv_heads, group;
    int page_size, num_total_pages, num_indices;
    int hs, hpt;         // head tiles per group, q heads per tile (the last may hold fewer)
    int npt, nps;        // nodes per row tile, nodes per segment (one or two row tiles)
    int tile_shift, seg_rows;  // rows of a row tile (log2) and of a segment, as the partials are laid out
    int slot_shift, cpp, spb_shift;  // rows of a slot (log2), slots of a page, slots of a block (log2)
    FastDiv by_page, by_cpp, by_nps, by_hpt, by_hs, by_heads;  // by page_size, cpp, nps, hpt, hs, hs * num_kv_heads
    int seg_cost;        // units that a segment costs beside its blocks
    int tails;           // shares may have tails (a merge follows)
    int whole;           // segments are not cut: each is one unit (no merge follows)
    int packed;          // pages are whole slots: the tokens of a block are consecutive
    float scale_log2;    // sm_scale * log2(e)
    int test_extra_tx;   // test-only wait-timeout injection (pd_test_inject_wait_timeout); normally 0
};

// One request as the table gives it. A bad one keeps its nodes and loses its
// tokens (len 0), so that every one of its rows is written as empty.
struct TreeReq {
    int n, start;  // nodes, first q row
    int len, lo;   // tokens, first entry of indices
    int bad;       // status bits
    __device__ __forceinline__ int ctx() const { return len - n; }
};

__device__ __forceinline__ TreeReq tree_request(const TreeArgs& a, int b) {
    TreeReq r = {0, 0, 0, 0, 0};
    const bool single = a.new_indptr == nullptr;
    const int s = single ? b : __ldg(a.new_indptr + b), e = single ? b + 1 : __ldg(a.new_indptr + b + 1);
    const int lo = __ldg(a.indptr + b), hi = __ldg(a.indptr + b + 1);
    int last = __ldg(a.last_page_len + b);
    if (s < 0 || e < s || e > a.total_new) {
        r.bad = kFlagBadNewRows;
        return r;
    }
    r.start = s;
    r.n = e - s;
    if (lo < 0 || hi < lo || hi > a.num_indices) {
        r.bad = kFlagBadIndptr;
        return r;
    }
    long long len = 0;
    if (hi > lo) {
        if (last < 0 || last > a.page_size) {
            r.bad = kFlagBadLastPageLen;
            last = last < 0 ? 0 : a.page_size;
        }
        len = (long long)(hi - lo - 1) * a.page_size + last;
    }
    if (len < r.n || len > 0x3fffffff) {
        if (!single || len > 0) r.bad |= kFlagBadNewRows;
        return r;
    }
    r.len = int(len);
    r.lo = lo;
    return r;
}

__device__ __forceinline__ int tree_slots(const TreeArgs& a, int tokens) {
    const int page = a.by_page.div(tokens), row = tokens - page * a.page_size;
    return page * a.cpp + ((row + (1 << a.slot_shift) - 1) >> a.slot_shift);
}

// The slot that holds a token.
__device__ __forceinline__ int tree_slot_of(const TreeArgs& a, int token) {
    const int page = a.by_page.div(token), row = token - page * a.page_size;
    return page * a.cpp + (row >> a.slot_shift);
}

// Key blocks of segment tau; at least one, so that a segment with no keys is still written.
__device__ __forceinline__ int tree_blocks(const TreeArgs& a, const TreeReq& r, int tau) {
    int limit = r.len;
    if (a.mask == nullptr) limit = min(limit, max(0, r.ctx()) + min(r.n, (tau + 1) * a.nps));
    return max(1, (tree_slots(a, limit) + (1 << a.spb_shift) - 1) >> a.spb_shift);
}

// Units of segment tau.
__device__ __forceinline__ int tree_units(const TreeArgs& a, const TreeReq& r, int tau) {
    return a.whole ? 1 : tree_blocks(a, r, tau) + a.seg_cost;
}

__device__ __forceinline__ long long tree_cost(const TreeArgs& a, const TreeReq& r) {
    const int segs = a.by_nps.div(r.n + a.nps - 1);
    long long sum = 0;
    if (a.whole)
        return (long long)segs * a.hs * a.num_kv_heads;
    if (a.mask != nullptr || segs <= 1) {
        sum = segs > 0 ? (long long)segs * tree_blocks(a, r, segs - 1) : 0;
    } else {
        for (int t = 0; t < segs; ++t) sum += tree_blocks(a, r, t);
    }
    sum += (long long)segs * a.seg_cost;
    return sum * a.hs * a.num_kv_heads;
}

// ceil(x / y); most lines are short enough for a 32-bit division.
__device__ __forceinline__ long long tree_ceil_div(long long x, int y) {
    return x < 0x7fffffffll - y ? (unsigned(x) + unsigned(y) - 1u) / unsigned(y) : (x + y - 1) / y;
}

// The line of units and its cuts: range r is share r, or (with tails) r / 2 is
// the share and r % 2 its tail.
struct TreeLine {
    long long total, share, tail;
    __device__ __forceinline__ static TreeLine of(const TreeArgs& a, long long total, int workers) {
        TreeLine l;
        l.total = total;
        l.share = tree_ceil_div(total, workers);
        l.tail = !a.tails || l.share < 48 ? 0 : l.share / 8;
        return l;
    }
    __device__ __forceinline__ long long start(int r) const {
        return tail == 0 ? r * share : (r / 2 + 1) * share - (r % 2 != 0 ? tail : share);
    }
    __device__ __forceinline__ long long end(int r) const { return min(start(r + 1), total); }
    __device__ __forceinline__ int range_of(long long u) const {
        const int s = u < 0x7fffffffll ? int(unsigned(u) / unsigned(share)) : int(u / share);
        return tail == 0 ? s : 2 * s + (u - s * share >= share - tail ? 1 : 0);
    }
};

static_assert(sizeof(TreeLine) <= sizeof(TreeSplit), "the line lies where range 0, which is no cut, would have its split");

// A range and the walk over its segments.
struct TreeWalk {
    int range;
    int b, hh, tau;
    int pos;                     // unit within the segment: its blocks start at seg_cost
    long long unit, begin, end;  // current unit; the range
    TreeReq r;

    // One portion of a segment: blocks [blk0, blk1) of nblk.
    struct Seg {
        int hh, kvh, head0, heads;   // head tile, its kv head, its first q head and how many
        int row0, node0, nodes;      // first q row, first node within the request, nodes
        int blk0, blk1;
        int tail0;                   // first block that holds a token from the context's end on
        int slots;                   // slots of the request
        int slot;                    // partial slot; -1: the whole segment, written out
        TreeReq r;
    };

    __device__ __forceinline__ bool next(const TreeArgs& a, Seg* s) {
        while (unit < end) {
            while (tau * a.nps >= r.n) {  // past the request's last segment
                tau = 0;
                if (++hh >= a.hs * a.num_kv_heads || r.n == 0) {
                    hh = 0;
                    if (++b >= a.batch) return false;
                    r = tree_request(a, b);
                }
            }
            const int nblk = tree_blocks(a, r, tau), cost = a.whole ? 1 : nblk + a.seg_cost;
            const long long first = unit - pos + a.seg_cost;  // unit of the segment's first block
            const int take = int(min((long long)(cost - pos), end - unit));
            s->blk0 = a.whole ? 0 : max(0, pos - a.seg_cost);
            s->blk1 = a.whole ? nblk : max(0, pos + take - a.seg_cost);
            s->node0 = tau * a.nps;
            unit += take;
            pos = 0;
            ++tau;
            if (s->blk1 <= s->blk0) continue;  // the range ends before the segment's first block
            s->r = r;
            s->hh = hh;
            s->kvh = a.by_hs.div(hh);
            const int h0 = (hh - s->kvh * a.hs) * a.hpt;
            s->head0 = s->kvh * a.group + h0;
            s->heads = min(a.hpt, a.group - h0);
            s->nodes = min(a.nps, r.n - s->node0);
            s->row0 = r.start + s->node0;
            s->tail0 = tree_slot_of(a, max(0, r.ctx())) >> a.spb_shift;
            s->slots = tree_slots(a, r.len);
            s->slot = s->blk0 == 0 && s->blk1 == nblk ? -1 : 2 * range + (first > begin ? 1 : 0);
            return true;
        }
        return false;
    }

    // The place of unit `left` of request b's units.
    __device__ __forceinline__ void place(const TreeArgs& a, int request, const TreeReq& req, long long cost, long long left) {
        b = request;
        r = req;
        if (cost < 0x7fffffffll) {
            const int each = a.by_heads.div(int(cost));
            hh = int(unsigned(left) / unsigned(each));
            left -= (long long)hh * each;
        } else {
            const long long each = cost / (a.hs * a.num_kv_heads);
            hh = int(left / each);
            left -= hh * each;
        }
        for (tau = 0;; ++tau) {
            const int c = tree_units(a, r, tau);
            if (left < c) break;
            left -= c;
        }
        pos = int(left);
    }

    // The merge's descriptor of a segment whose first cut is this range's start. One thread, before next().
    __device__ __forceinline__ void write_split(const TreeArgs& a, const TreeLine& line) const {
        TreeSplit s{};
        if (unit < end && range > 0 && !a.whole) {
            const long long first = unit - pos + a.seg_cost, prev = line.start(range - 1);
            if (first < unit && first >= prev) {
                s.r0 = range - 1;
                s.parts = line.range_of(first + tree_blocks(a, r, tau) - 1) - s.r0 + 1;
                s.slot0 = 2 * s.r0 + (first > prev ? 1 : 0);
                s.hh = hh;
                s.row0 = r.start + tau * a.nps;
                s.nodes = min(a.nps, r.n - tau * a.nps);
            }
        }
        if (range > 0) a.splits[range] = s;
    }

    // Find range `rg` by a whole warp: each lane sums a run of requests.
    __device__ __forceinline__ void locate(const TreeArgs& a, const TreeLine& line, int rg) {
        const int lane = threadIdx.x & 31;
        const int per = (a.batch + 31) / 32, b0 = min(lane * per, a.batch), b1 = min(b0 + per, a.batch);
        range = rg;
        unit = begin = line.start(rg);
        end = line.end(rg);
        long long mine = 0;
        for (int x = b0; x < b1; ++x) mine += tree_cost(a, tree_request(a, x));
        long long inc = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(kFull, inc, off);
            if (lane >= off) inc += y;
        }
        long long left = unit - (inc - mine);
        const unsigned here = __ballot_sync(kFull, left >= 0 && left < mine);
        const int src = __ffs(here) - 1;  // some lane: the range is not empty
        left = __shfl_sync(kFull, left, src);
        for (int x = src * per;; ++x) {
            const TreeReq req = tree_request(a, x);
            const long long c = tree_cost(a, req);
            if (left < c) {
                place(a, x, req, c, left);
                return;
            }
            left -= c;
        }
    }
};

struct TreePlanScratch {
    long long sums[32];
    long long total;
    struct {
        int b, hh, tau, pos;
        TreeReq r;
    } at[2];  // where each worker of the CTA starts
};

// Find the shares of this CTA's kWorkers workers. All threads of the block
// call it; ends with a block barrier, after which tree_start gives the walks.
template <int kWorkers>
__device__ __forceinline__ void tree_plan(const TreeArgs& a, TreePlanScratch* sc) {
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, nt = blockDim.x, nw = nt >> 5;
    const int per = (a.batch + nt - 1) / nt;
    const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    long long mine = 0, last = 0;
    TreeReq r{};
    for (int b = b0; b < b1; ++b) {
        r = tree_request(a, b);
        if (r.bad != 0 && blockIdx.x == 0) atomicOr(a.flags, r.bad);
        last = tree_cost(a, r);
        mine += last;
    }
    long long inc = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long x = __shfl_up_sync(kFull, inc, off);
        if (lane >= off) inc += x;
    }
    if (lane == 31) sc->sums[wid] = inc;
    if (tid < kWorkers) sc->at[tid].b = -1;
    __syncthreads();
    long long before = inc - mine, total = 0;
    for (int w = 0; w < min(nw, (a.batch + 31) / 32); ++w) {  // the others hold no request
        const long long x = sc->sums[w];
        if (w < wid) before += x;
        total += x;
    }
    const TreeLine line = TreeLine::of(a, total, int(gridDim.x) * kWorkers);
    if (tid == 0) {
        sc->total = total;
        if (blockIdx.x == 0) *reinterpret_cast<TreeLine*>(a.splits) = line;
    }
#pragma unroll
    for (int k = 0; k < kWorkers; ++k) {
        const long long unit = ((long long)blockIdx.x * kWorkers + k) * line.share;
        if (unit >= total || unit < before || unit >= before + mine) continue;
        long long left = unit - before;
        for (int b = b0; b < b1; ++b) {
            if (b1 - b0 > 1) r = tree_request(a, b);  // (one request per thread: r is it)
            const long long c = b1 - b0 > 1 ? tree_cost(a, r) : last;
            if (left >= c) {
                left -= c;
                continue;
            }
            TreeWalk w;
            w.place(a, b, r, c, left);
            sc->at[k] = {b, w.hh, w.tau, w.pos, r};
            break;
        }
    }
    __syncthreads();
}

// The line, and the walk over the share (without its tail) of worker k of this CTA.
template <int kWorkers>
__device__ __forceinline__ TreeLine tree_line(const TreeArgs& a, const TreePlanScratch* sc) {
    return TreeLine::of(a, sc->total, int(gridDim.x) * kWorkers);
}
template <int kWorkers>
__device__ __forceinline__ TreeWalk tree_start(const TreeLine& line, const TreePlanScratch* sc, int k) {
    TreeWalk w;
    const int worker = int(blockIdx.x) * kWorkers + k;
    w.range = line.tail == 0 ? worker : 2 * worker;
    w.unit = w.begin = line.start(w.range);
    w.b = sc->at[k].b;
    w.hh = sc->at[k].hh;
    w.tau = sc->at[k].tau;
    w.pos = sc->at[k].pos;
    w.r = sc->at[k].r;
    w.end = w.b < 0 ? w.unit : line.end(w.range);
    return w;
}

// The next tail that nobody has asked for, by a whole warp. false: none.
__device__ __forceinline__ bool tree_claim(const TreeArgs& a, const TreeLine& line, int* range) {
    if (line.tail == 0) return false;
    int t = 0;
    if ((threadIdx.x & 31) == 0) t = int(atomicAdd(a.claims, 1u));
    t = __shfl_sync(kFull, t, 0);
    *range = 2 * t + 1;
    return line.start(*range) < line.total;
}

// Which of 32 consecutive tokens t0 .. t0 + 31 (only the first `count` stand
// for tokens) node `node` of the request attends, as bits.
__device__ __forceinline__ uint32_t tree_allow(const TreeArgs& a, const TreeReq& r, int node, int t0, int count) {
    uint32_t bits = count >= 32 ? ~0u : count <= 0 ? 0u : (1u << count) - 1u;
    if (t0 + 32 > r.len) bits &= r.len <= t0 ? 0u : r.len - t0 >= 32 ? ~0u : (1u << (r.len - t0)) - 1u;
    const int i0 = t0 - r.ctx();  // node index of t0
    if (i0 + 32 <= 0 || bits == 0u) return bits;
    if (a.mask == nullptr) {
        const int seen = node + 1 - i0;  // tokens t0 .. of the chain up to the node itself
        return bits & (seen >= 32 ? ~0u : seen <= 0 ? 0u : (1u << seen) - 1u);
    }
    const uint32_t* row = a.mask + size_t(r.start + node) * a.mask_words;
    auto word = [&](int w) { return w < 0 ? ~0u : w < a.mask_words ? __ldg(row + w) : 0u; };
    const int w = i0 >= 0 ? i0 / 32 : -1, sh = i0 - 32 * w;  // sh in 0 .. 31
    return bits & __funnelshift_r(word(w), word(w + 1), sh);
}

// q row (and o row) index of row `row` of a segment, or -1.
__device__ __forceinline__ long long tree_row(const TreeArgs& a, int row0, int nodes, int hh, int row) {
    const int tile = row >> a.tile_shift, x = row - (tile << a.tile_shift);
    const int y = a.by_hpt.div(x), kvh = a.by_hs.div(hh);
    const int node = tile * a.npt + y, h = (hh - kvh * a.hs) * a.hpt + x - y * a.hpt;
    if (x >= a.npt * a.hpt || node >= nodes || h >= a.group) return -1;
    return (long long)(row0 + node) * a.num_qo_heads + kvh * a.group + h;
}

// Whether a descriptor of range `range` points into the partials of `ranges`
// ranges and the rows of this call.
__device__ __forceinline__ bool tree_split_fits(const TreeArgs& a, const TreeSplit& s, int range, int ranges) {
    return s.r0 == range - 1 && unsigned(s.parts) <= unsigned(ranges - range + 1) && (s.slot0 | 1) == 2 * range - 1 &&
           unsigned(s.hh) < unsigned(a.hs * a.num_kv_heads) && unsigned(s.nodes) <= unsigned(a.nps) && s.row0 >= 0 &&
           s.row0 <= a.total_new - s.nodes;
}

constexpr int kMergeBlocks = 4;  // blocks per possible split

// One warp per row of a split segment at a time: parts in the order of the
// line. Bound by its two dependent reads (descriptor, then partials): 5.4 us for
// the 303 cuts of 32 chains of 4, launched early so that its start is hidden.
template <typename T, int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreeArgs a) {
    constexpr int kPer = D / 32;
    const float kNegInf = -__int_as_float(0x7f800000);
    grid_dependency_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.claims = 0;
    const int range = int(blockIdx.x / kMergeBlocks) + 1;
    const TreeLine line = *reinterpret_cast<const TreeLine*>(a.splits);
    if (line.start(range) >= line.total) return;
    TreeSplit s = a.splits[range];
    // (as no split, not as another exit: that took 106 registers instead of 64, and 60 us of chains 2 us more)
    if (!tree_split_fits(a, s, range, int(gridDim.x / kMergeBlocks) + 1)) s.parts = 0;
    if (s.parts == 0) return;
    for (int i = int(blockIdx.x % kMergeBlocks) * 8 + (threadIdx.x >> 5); i < s.nodes * a.hpt; i += 8 * kMergeBlocks) {
        const int per_tile = a.npt * a.hpt, tile = i / per_tile, row = (tile << a.tile_shift) + i - tile * per_tile;
        const long long at = tree_row(a, s.row0, s.nodes, s.hh, row);
        if (at < 0) continue;  // past the group's last head
        auto slot = [&](int p) { return size_t(p == 0 ? s.slot0 : 2 * (s.r0 + p)) * a.seg_rows + row; };
        float acc[kPer] = {};
        const float L = merge_rows<kPer, 8>(
            s.parts, [&](int p) { return a.part_lse[slot(p)]; }, [&](int p) { return a.part_o + slot(p) * D; }, acc);
        store_row<T, kPer>(static_cast<T*>(a.o) + at * D, acc);
        if ((threadIdx.x & 31) == 0) a.lse[at] = L == kNegInf ? kNegInf : L * kLn2;
    }
}

// A partial's lse for the merge, whose maximum over the parts would pass over
// NaN: infinity comes through it, and makes the weights, o and lse NaN again.
__device__ __forceinline__ float tree_part_lse(float lse2) { return isnan(lse2) ? __int_as_float(0x7f800000) : lse2; }

// ---------------------------------------------------------------- CUDA cores

// Four elements of a pool row to f32 (of q too, s = 1); s scales E4M3 codes.
template <typename KV>
__device__ __forceinline__ void pool_load4(const KV* p, float s, float* f) {
    if constexpr (sizeof(KV) == 4) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(p));
        f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w;
    } else if constexpr (sizeof(KV) == 2) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
        float t[8];
        Elt<KV>::to_f32(make_uint4(w.x, w.y, 0u, 0u), t);
        f[0] = t[0], f[1] = t[1], f[2] = t[2], f[3] = t[3];
    } else {
        float t[8];
        e4m3x8_to_f32(make_uint2(__ldg(reinterpret_cast<const uint32_t*>(p)), 0u), t);
        f[0] = t[0] * s, f[1] = t[1] * s, f[2] = t[2] * s, f[3] = t[3] * s;
    }
}

// 16 bytes from global to shared memory, or 16 zero bytes.
__device__ __forceinline__ void copy16_async(void* dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <int D, int kCols>  // kCols: threads that share a row (at most D / 4)
struct CfgTreeCc {
    static constexpr int kKeys = 32, kThreads = 128;
    static constexpr int kRows = 2 * kThreads / kCols;
    static constexpr int kPer = kKeys / kCols;  // keys of a thread's scores
    static constexpr int kBlockTokens = 32;  // short, so that a small call spreads over SMs
    static constexpr int kWindow = 128;      // tokens whose rows are looked up at a time
    static constexpr int kLd = D + 4;  // row step of q and K in shared memory: 16-byte reads of 8 rows hit all banks
    static constexpr int kBufs = D == 256 ? 1 : 2;   // of K and V: the next keys on their way
    static constexpr int kLdP = kKeys + 4;           // row step of the weights: 16-byte reads
    static constexpr int kKv = kKeys * kLd + kKeys * D;
    static constexpr int kFloats = kRows * kLd + kBufs * kKv + kRows * kLdP;
    static constexpr int kBytes = kFloats * 4;
    static constexpr int kBlocksPerSm = D == 64 ? (kCols > 8 ? 5 : 4) : D == 128 && kCols == 32 ? 3 : 2;
};

// f32 arithmetic on CUDA cores: f32 q (no tensor-core type holds it) and
// groups of more than 128 heads. 32 rows x 32 keys per step: thread (tr, tc)
// of 16 x 8 holds rows 2 tr, 2 tr + 1: scores of keys tc + 8 i, outputs of
// columns 4 tc + 32 i. The 8 lanes of a row sit in one warp, so the softmax
// needs no block barrier. Bound by FFMA issue: 4 D flops per row and key
// against shared-memory reads of 6 (scores) and 1 (outputs) vectors per 32 and
// 8 multiply-adds. Where requests have up to 8 or 16 rows, 32 or 16 threads
// share a row, so that every thread has rows to work for (8 requests of up to
// 2484 tokens: 2 rows of head_dim 256 over 16 kv heads 226 -> 115 us, 16 rows of
// head_dim 128 over 8 kv heads 82 -> 59 us; 32 requests, 4 rows of head_dim 128:
// 360 -> 154 us, 57% of the copy rate).
// A small call is latency: one request of 100 tokens, 6 nodes takes 9.7 us on
// the device, most of it the walk's and the first copies' round trips (the call
// 11.5 us; with blocks of 128 tokens, cut and merged, 19.9).
template <typename T, typename KV, int D, int kCols>
__global__ void __launch_bounds__(128, CfgTreeCc<D, kCols>::kBlocksPerSm) tree_cc_kernel(const TreeArgs a) {
    using C = CfgTreeCc<D, kCols>;
    constexpr int kPer = C::kPer, kVecs = D / (4 * kCols);
    const float kNegInf = -__int_as_float(0x7f800000);
    extern __shared__ __align__(16) float tree_smem[];
    __shared__ TreePlanScratch plan;
    __shared__ long long row_offs[C::kWindow];  // element offset of each key's row in the pools; -1: none
    float* sq = tree_smem;
    float* kv = sq + C::kRows * C::kLd;
    float* sp = kv + C::kBufs * C::kKv;
    const int tid = threadIdx.x, tr = tid / kCols, tc = tid % kCols;
    tree_plan<1>(a, &plan);
    const TreeLine line = tree_line<1>(a, &plan);
    TreeWalk walk = tree_start<1>(line, &plan, 0);
    if (tid == 0) walk.write_split(a, line);
    launch_dependents();
    TreeWalk::Seg s;
    for (;;) {
        if (!walk.next(a, &s)) {
            __shared__ int claimed;
            __syncthreads();
            if (tid < 32) {
                int range;
                const bool got = tree_claim(a, line, &range);
                if (tid == 0) claimed = got ? range : -1;
            }
            __syncthreads();
            if (claimed < 0) break;
            walk.locate(a, line, claimed);
            if (tid == 0) walk.write_split(a, line);
            continue;
        }
        __syncthreads();
        const float ks = a.k_scale != nullptr ? __ldg(a.k_scale + s.kvh) : 1.f;
        const float vs = a.v_scale != nullptr ? __ldg(a.v_scale + s.kvh) : 1.f;
        for (int i = tid; i < C::kRows * (D / 4); i += C::kThreads) {
            const int row = i / (D / 4), e = i % (D / 4) * 4;
            const long long at = tree_row(a, s.row0, s.nodes, s.hh, row);
            float f[4] = {};
            if (at >= 0) pool_load4(static_cast<const T*>(a.q) + at * D + e, 1.f, f);
            *reinterpret_cast<float4*>(sq + row * C::kLd + e) = make_float4(f[0], f[1], f[2], f[3]);
        }
        float m[2] = {kNegInf, kNegInf}, l[2] = {}, o[2][4 * kVecs] = {};
        const int node[2] = {s.node0 + a.by_hpt.div(2 * tr), s.node0 + a.by_hpt.div(2 * tr + 1)};
        int window;  // first token of row_offs
        // Keys t0 .. of the pools into buffer `buf` (zeros where there is no row): asynchronous copies of f32
        // pools, loads and conversions of others.
        auto load = [&](int t0, int buf) {
            float* sk = kv + buf * C::kKv;
            float* sv = sk + C::kKeys * C::kLd;
            for (int i = tid; i < C::kKeys * (D / 4); i += C::kThreads) {
                const int key = i / (D / 4), e = i % (D / 4) * 4;
                const long long off = row_offs[t0 - window + key];
                if constexpr (sizeof(KV) == 4) {
                    const long long at = off < 0 ? 0 : off + e;
                    copy16_async(sk + key * C::kLd + e, static_cast<const float*>(a.k) + at, off >= 0);
                    copy16_async(sv + key * D + e, static_cast<const float*>(a.v) + at, off >= 0);
                } else {
                    float fk[4] = {}, fv[4] = {};
                    if (off >= 0) {
                        pool_load4(static_cast<const KV*>(a.k) + off + e, ks, fk);
                        pool_load4(static_cast<const KV*>(a.v) + off + e, vs, fv);
                    }
                    *reinterpret_cast<float4*>(sk + key * C::kLd + e) = make_float4(fk[0], fk[1], fk[2], fk[3]);
                    *reinterpret_cast<float4*>(sv + key * D + e) = make_float4(fv[0], fv[1], fv[2], fv[3]);
                }
            }
            copy_commit();
        };
        const int t_end = min(s.blk1 * C::kBlockTokens, s.r.len);
        window = s.blk0 * C::kBlockTokens - C::kWindow;
        for (int t0 = s.blk0 * C::kBlockTokens; t0 < t_end; t0 += C::kKeys) {
            const int buf = t0 / C::kKeys % C::kBufs;
            if (t0 >= window + C::kWindow) {
                __syncthreads();
                window = t0;
                const int t = t0 + tid;
                long long off = -1;
                if (t < s.r.len) {
                    const int nth = a.by_page.div(t), page = __ldg(a.indices + s.r.lo + nth);
                    if (page >= 0 && page < a.num_total_pages)
                        off = (((long long)page * a.num_kv_heads + s.kvh) * a.page_size + t - nth * a.page_size) * D;
                    else
                        atomicOr(a.flags, kFlagBadPage);
                }
                row_offs[tid] = off;
                __syncthreads();
                load(t0, buf);
            } else if (C::kBufs == 1) {
                __syncthreads();
                load(t0, buf);
            }
            copy_wait();
            __syncthreads();
            const bool ahead = C::kBufs == 2 && t0 + C::kKeys < t_end && t0 + C::kKeys < window + C::kWindow;
            if (ahead) load(t0 + C::kKeys, buf ^ 1);
            const float* sk = kv + buf * C::kKv;
            const float* sv = sk + C::kKeys * C::kLd;
            const long long* row_off = row_offs + (t0 - window);
            float x[2][kPer] = {};
#pragma unroll 4
            for (int e = 0; e < D; e += 4) {
                const float4 q0 = *reinterpret_cast<const float4*>(sq + (2 * tr) * C::kLd + e);
                const float4 q1 = *reinterpret_cast<const float4*>(sq + (2 * tr + 1) * C::kLd + e);
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const float4 k = *reinterpret_cast<const float4*>(sk + (tc + kCols * i) * C::kLd + e);
                    x[0][i] = fmaf(q0.w, k.w, fmaf(q0.z, k.z, fmaf(q0.y, k.y, fmaf(q0.x, k.x, x[0][i]))));
                    x[1][i] = fmaf(q1.w, k.w, fmaf(q1.z, k.z, fmaf(q1.y, k.y, fmaf(q1.x, k.x, x[1][i]))));
                }
            }
            const bool tail = t0 + C::kKeys > s.r.ctx();  // holds tokens that some row does not attend
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t allow = tree_allow(a, s.r, min(node[j], s.r.n - 1), t0, C::kKeys);
                float top = kNegInf;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const bool in = ((allow >> (tc + kCols * i)) & 1u) != 0 && row_off[tc + kCols * i] >= 0;
                    x[j][i] = in ? x[j][i] * a.scale_log2 : kNegInf;
                    top = fmaxf(top, x[j][i]);
                }
#pragma unroll
                for (int off = 1; off < kCols; off <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
                const float mn = fmaxf(m[j], top), mu = mn == kNegInf ? 0.f : mn;
                const float al = ex2(m[j] - mu);
                m[j] = mn;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const float p = ex2(x[j][i] - mu);
                    sum += p;
                    sp[(2 * tr + j) * C::kLdP + tc + kCols * i] = p;
                }
                l[j] = l[j] * al + sum;
#pragma unroll
                for (int i = 0; i < 4 * kVecs; ++i) o[j][i] *= al;
            }
            __syncwarp();
            auto accumulate = [&](auto guard) {
#pragma unroll 2
                for (int key4 = 0; key4 < C::kKeys; key4 += 4) {
                    const float4 w0 = *reinterpret_cast<const float4*>(sp + (2 * tr) * C::kLdP + key4);
                    const float4 w1 = *reinterpret_cast<const float4*>(sp + (2 * tr + 1) * C::kLdP + key4);
                    const float p0s[4] = {w0.x, w0.y, w0.z, w0.w}, p1s[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float p0 = p0s[x], p1 = p1s[x];
#pragma unroll
                        for (int i = 0; i < kVecs; ++i) {
                            const float4 v = *reinterpret_cast<const float4*>(sv + (key4 + x) * D + 4 * (tc + kCols * i));
                            const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                // a row that does not attend the key takes no part of it, not 0 * NaN either
                                if (!decltype(guard)::value || p0 != 0.f) o[0][4 * i + c] = fmaf(p0, f[c], o[0][4 * i + c]);
                                if (!decltype(guard)::value || p1 != 0.f) o[1][4 * i + c] = fmaf(p1, f[c], o[1][4 * i + c]);
                            }
                        }
                    }
                }
            };
            if (tail)
                accumulate(std::true_type{});
            else
                accumulate(std::false_type{});
            __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = 2 * tr + j;
            float L = l[j];
#pragma unroll
            for (int off = 1; off < kCols; off <<= 1) L += __shfl_xor_sync(kFull, L, off);
            const long long at = tree_row(a, s.row0, s.nodes, s.hh, row);
            if (at < 0) continue;
            // empty by the sum: the maximum passes over scores of NaN, the sum does not
            const float inv = L == 0.f ? 0.f : 1.f / L;
            const float lse2 = L == 0.f ? kNegInf : m[j] + log2f(L);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                float f[8] = {};
#pragma unroll
                for (int c = 0; c < 4; ++c) f[c] = o[j][4 * i + c] * inv;
                const int e = 4 * (tc + kCols * i);
                if (s.slot >= 0) {
                    *reinterpret_cast<float4*>(a.part_o + (size_t(s.slot) * a.seg_rows + row) * D + e) =
                        make_float4(f[0], f[1], f[2], f[3]);
                } else if constexpr (sizeof(T) == 4) {
                    *reinterpret_cast<float4*>(static_cast<T*>(a.o) + at * D + e) = make_float4(f[0], f[1], f[2], f[3]);
                } else {
                    *reinterpret_cast<uint2*>(static_cast<T*>(a.o) + at * D + e) =
                        make_uint2(Elt<T>::pack(f[0], f[1]), Elt<T>::pack(f[2], f[3]));
                }
            }
            if (tc == 0) {
                if (s.slot >= 0)
                    a.part_lse[size_t(s.slot) * a.seg_rows + row] = tree_part_lse(lse2);
                else
                    a.lse[at] = lse2 == kNegInf ? kNegInf : lse2 * kLn2;
            }
        }
    }
}

}  // namespace pd
