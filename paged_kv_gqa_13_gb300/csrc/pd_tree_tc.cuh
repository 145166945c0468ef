// Tree decode on the 5th-generation tensor cores (tcgen05.mma kind::f16, f32
// accumulators in tensor memory) for 16-bit q over 16-bit paged pools.
//
// A row tile is up to 128 rows (nodes x q heads of one kv head): the M of both
// products. Per block of KB keys and row tile: S = Q K^T (A = Q and B = K from
// shared memory, K-major as they lie), then the softmax warps turn S into
// weights P in place (tensor memory), then O += P V (A = P from tensor memory,
// B = V from shared memory, MN-major as it lies).
//
// Two row-tile pipelines t = 0, 1, each with its own S/P and O columns and its
// own 4 softmax warps, run out of phase: while one's softmax runs, the tensor
// cores work for the other. A segment of more than one row tile (up to two)
// gives each pipeline its own rows, both over every block ("wide"); one of a
// single row tile gives both the same rows over alternate blocks, and joins
// the two (m, l, O) at the end. At head_dim 256 tensor memory holds one O:
// blocks of 64 keys, S double-buffered, one set of softmax warps.
//
// Roles (16 warps): 0-3 and 4-7 softmax of pipeline 0 and 1; 8, 12 and 13
// producers (TMA of q, K and V into a ring of slots of one K or V block), 9 and
// 11 issue the mma of pipeline 0 and 1, 10 walks the segments;
// 14 and 15 make V safe where weights can be zero: a zero weight does not undo a
// NaN or an infinity, so in blocks that hold tokens some row does not attend,
// rows past the end are zeroed and non-finite elements of node rows are
// replaced by zero, to be added to the rows that attend them at the end.
// Registers move from the last two warpgroups to the softmax warps, whose
// threads hold a row of S.
//
// Producer, mma and inspectors follow the same sequence of steps, which each
// of them generates for itself (TcSteps): a pipeline's next S is issued as
// soon as its last P V has been, so the ring is filled in the order in which
// the mma warp waits.
//
// The running maximum of a row moves only when it rises by more than 2^8 (the
// weights then stay below 2^8, and O, in tensor memory, is rescaled rarely).
#pragma once

#include "pd_decode_tc.cuh"
#include "pd_tree.cuh"

namespace pd {

// ---------------------------------------------------------------- PTX wrappers

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// Instruction descriptor of kind::f16: 16-bit A and B of one type, f32 accumulator.
// neg_a: A is negated; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t tc_idesc_f16(bool bf16, int M, int N, bool b_mn) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | (uint32_t(N >> 3) << 17) |
           (uint32_t(M >> 4) << 24);
}
constexpr uint32_t kIdescNegA = 1u << 13;

// D = A * B (+ D when acc), A and B from shared memory.
__device__ __forceinline__ void tc_mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(acc))
        : "memory");
}

// The same with A in tensor memory (two 16-bit elements per column).
__device__ __forceinline__ void tc_mma_f16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(acc))
        : "memory");
}

// 32 consecutive columns of this thread's tensor-memory lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int R>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// Wait for phase `parity` of `bar`; false when the CTA is aborting or the wait
// runs out, which sets the abort flag and the status bit. The limit is counted
// on the SM clock (4e9 cycles, about 2 s): a read of the global timer takes
// longer than most of these waits.
constexpr long long kWaitCycles = 4000000000ll;
__device__ __forceinline__ bool tree_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* flags) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    for (;;) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (clock64() - t0 > kWaitCycles) {
            *abort_flag = 1;
            atomicOr(flags, kFlagTimeout);
            return false;
        }
    }
}
// The same for a whole warp: true only if every lane's wait succeeded.
__device__ __forceinline__ bool tree_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* flags) {
    return __all_sync(kFull, tree_wait(bar, parity, abort_flag, flags));
}

// ---------------------------------------------------------------- configuration

template <int D>
struct CfgTree {
    static constexpr int kRows = 128;
    static constexpr int kTiles = D == 256 ? 1 : 2;    // O accumulators
    static constexpr int kKeys = D == 256 ? 64 : 128;  // keys per block
    static constexpr int kHalves = D / 64;             // 128-byte column blocks of a row
    static constexpr int kSlotBytes = kKeys * D * 2;   // one K or V block
    static constexpr int kQBytes = kRows * D * 2;      // one row tile of q
    static constexpr int kQSlots = kTiles;
    static constexpr int kSlots = D == 64 ? 10 : 5;
    static constexpr int kRingOff = kQSlots * kQBytes;
    static constexpr int kBarOff = kRingOff + kSlots * kSlotBytes;
    // barriers: full[], empty[], vok[] per slot, then these
    static constexpr int kBars = 3 * kSlots + 2 * 2 + 2 + 2 + 2 + 4 + 2 * 8;
    static constexpr int kStatOff = kBarOff + (kBars * 8 + 15) / 16 * 16;  // pipeline 1's (m, l) per row
    static constexpr int kMiscOff = kStatOff + kRows * 8;  // tensor-memory address, abort flag, bad-V tags[4]
    static constexpr int kBadRing = 16;  // more than the K blocks that the producer is ahead of the softmax warps
    static constexpr int kSegOff = kMiscOff + 32 + 4 * kBadRing;
    static constexpr int kBytes = kSegOff + 8 * 64 + 1024;  // 1024: alignment of the base
    static constexpr int kProducers = 3, kInspectors = 2;
    static constexpr int kWalkers = kProducers + kTiles + kInspectors + 4 * kTiles;  // warps that read the segments
    static constexpr int kOCols = D;
    static constexpr int kSCol = kTiles * D;
    static constexpr int kThreads = 512;
    static_assert(kSCol + 2 * kKeys <= 512, "tensor memory");
    static_assert(kBytes <= 232448, "shared memory");
};

// Segments come to the roles through a ring in shared memory, filled by one
// warp that walks them. blk1 = blk0 ends the line.
struct alignas(16) TcSeg {
    int blk0, blk1, tail0, slots;     // blocks; first block with node tokens; slots of the request
    int slot, row0, node0, nodes;     // partial slot or -1; q rows and nodes of the segment
    int hh, head0, kvh, lo;           // head tile, its first q head and kv head; first entry of indices
    int len, n, start, wide;          // the request: tokens, nodes, first q row; two row tiles
    __device__ __forceinline__ TreeReq req() const {
        TreeReq r;
        r.n = n;
        r.start = start;
        r.len = len;
        r.lo = lo;
        return r;
    }
};
constexpr int kSegRing = 8;

// One step of the sequence. Job j of a segment is block j / 2 for pipeline
// j % 2 (wide), or block j for pipeline (S buffer, at head_dim 256) j % 2.
struct TcStep {
    int j = 0, jobs = 0, seg = -1;  // job, jobs of the segment, segments before it
    int blk0 = 0, tail0 = 0;
    bool wide = false;
    __device__ __forceinline__ bool enter(const TcSeg& s) {
        wide = s.wide != 0;
        blk0 = s.blk0;
        tail0 = s.tail0;
        jobs = (s.blk1 - blk0) * (wide ? 2 : 1);
        j = 0;
        ++seg;
        return jobs > 0;
    }
    __device__ __forceinline__ int block() const { return blk0 + (wide ? j >> 1 : j); }
    __device__ __forceinline__ bool tail() const { return block() >= tail0; }
    __device__ __forceinline__ int row_tile() const { return wide ? j & 1 : 0; }
    __device__ __forceinline__ bool opens_tile() const { return j == 0 || (wide && j == 1); }
    __device__ __forceinline__ bool closes_tile() const { return j + 1 == jobs || (wide && j + 2 == jobs); }
    __device__ __forceinline__ bool first_use() const { return !wide || (j & 1) == 0; }  // of its K (or V) block
};

// The order of the mma warp's steps. seg_wait(i) waits for segment i and
// returns it (null to stop), seg_free(i) gives it back; on_qk(step, seg) and
// on_pv(step, seg) return false to stop.
template <class SegWait, class SegFree, class OnQk, class OnPv>
__device__ __forceinline__ void tc_steps(SegWait seg_wait, SegFree seg_free, OnQk on_qk, OnPv on_pv) {
    TcStep q, p;
    const TcSeg *sq = seg_wait(0), *sp = sq;
    if (sq == nullptr || !q.enter(*sq)) return;
    p = q;
    bool more = true;
    int ahead = 0;  // bit t: pipeline t has an S whose P V is still to come
    for (;;) {
        while (more && ((ahead >> (q.j & 1)) & 1) == 0) {
            if (!on_qk(q, *sq)) return;
            ahead |= 1 << (q.j & 1);
            if (++q.j == q.jobs) {
                if ((sq = seg_wait(q.seg + 1)) == nullptr) return;
                more = q.enter(*sq);
            }
        }
        if (!on_pv(p, *sp)) return;
        ahead &= ~(1 << (p.j & 1));
        if (++p.j == p.jobs) {
            seg_free(p.seg);
            if ((sp = seg_wait(p.seg + 1)) == nullptr || !p.enter(*sp)) return;
        }
    }
}

// A place in a ring of N slots and the phase of its barriers.
template <int N>
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == N) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// Token of column col of block blk (col % slot_rows rows into its slot); -1 for a row past its page.
__device__ __forceinline__ int tree_token(const TreeArgs& a, int blk, int col) {
    const int s = blk * a.spb + col / a.slot_rows;
    const int row = s % a.cpp * a.slot_rows + col % a.slot_rows;
    return row < a.page_size ? s / a.cpp * a.page_size + row : -1;
}

// ---------------------------------------------------------------- the kernel

template <typename T, int D>
__global__ void __launch_bounds__(512, 1)
    tree_tc_kernel(const TreeArgs a, const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                   const __grid_constant__ CUtensorMap tmv) {
    using C = CfgTree<D>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    const float kNegInf = -__int_as_float(0x7f800000);
    extern __shared__ __align__(16) uint8_t tree_tc_smem[];
    uint8_t* smem = tree_tc_smem + ((1024u - (smem_u32(tree_tc_smem) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    auto bar = [&](int i) { return sbase + C::kBarOff + 8u * uint32_t(i); };
    constexpr int kFullB = 0, kEmptyB = C::kSlots, kVokB = 2 * C::kSlots, kQFull = 3 * C::kSlots, kQEmpty = kQFull + 2,
                  kSFull = kQEmpty + 2, kPFull = kSFull + 2, kPvDone = kPFull + 2, kOneDone = kPvDone + 2,
                  kOneFree = kOneDone + 1, kAllDone = kOneFree + 1, kSegFull = kAllDone + 2, kSegFree = kSegFull + kSegRing;
    static_assert(kSegFree + kSegRing == C::kBars, "barrier count");
    float2* stat = reinterpret_cast<float2*>(smem + C::kStatOff);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
    volatile int* bad_v = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 16);
    // slots of each K block whose page id is bad, by the K block's number in this CTA
    volatile uint32_t* bad_slots = reinterpret_cast<volatile uint32_t*>(smem + C::kMiscOff + 32);

    if (tid == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(bar(kFullB + i), 1);
            mbar_init(bar(kEmptyB + i), C::kTiles + C::kInspectors);  // the mma warps and the inspectors
            mbar_init(bar(kVokB + i), C::kInspectors);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kQFull + i), 1);
            mbar_init(bar(kQEmpty + i), C::kTiles);
            mbar_init(bar(kSFull + i), 1);
            mbar_init(bar(kPFull + i), 4);
            mbar_init(bar(kPvDone + i), 1);
        }
        for (int i = 0; i < kSegRing; ++i) {
            mbar_init(bar(kSegFull + i), 1);
            mbar_init(bar(kSegFree + i), C::kWalkers);
        }
        mbar_init(bar(kOneDone), 4);
        mbar_init(bar(kOneFree), 4);
        mbar_init(bar(kAllDone), 1);
        mbar_init(bar(kAllDone + 1), 1);
        fence_mbar_init();
        *abort_flag = 0;
        for (int i = 0; i < 4; ++i) bad_v[i] = 0;
    }
    if (wid == 9) tmem_alloc(smem_u32(tslot), 512);
    if (wid == 8 && lane == 0) {
        prefetch_tensormap(&tmq);
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
    }
    TreeWalk walk = tree_plan(a, reinterpret_cast<TreePlanScratch*>(smem + C::kRingOff));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    launch_dependents();
    const uint32_t tmem = *tslot;
    TcSeg* segs = reinterpret_cast<TcSeg*>(smem + C::kSegOff);
    // one lane / a whole warp
    auto seg_wait1 = [&](int i) -> const TcSeg* {
        return tree_wait(bar(kSegFull + i % kSegRing), uint32_t(i / kSegRing) & 1u, abort_flag, a.flags) ? segs + i % kSegRing : nullptr;
    };
    auto seg_wait = [&](int i) -> const TcSeg* {
        return tree_wait_warp(bar(kSegFull + i % kSegRing), uint32_t(i / kSegRing) & 1u, abort_flag, a.flags) ? segs + i % kSegRing
                                                                                                            : nullptr;
    };
    auto seg_free1 = [&](int i) { mbar_arrive(bar(kSegFree + i % kSegRing)); };
    auto seg_free = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSegFree + i % kSegRing));
    };

    if (wid >= 8) {
        regs_dec<64>();
        if (wid == 10) {
            // ============================================================ segments
            TreeWalk::Seg s;
            for (int i = 0;; ++i) {
                const bool more = walk.next(a, &s);
                if (i >= kSegRing &&
                    !tree_wait_warp(bar(kSegFree + i % kSegRing), uint32_t(i / kSegRing - 1) & 1u, abort_flag, a.flags))
                    break;
                if (lane == 0) {
                    TcSeg x{};
                    if (more)
                        x = TcSeg{s.blk0, s.blk1,  s.tail0, s.slots, s.slot,  s.row0, s.node0,   s.nodes,
                                  s.hh,   s.head0, s.kvh,   s.r.lo,  s.r.len, s.r.n,  s.r.start, C::kTiles == 2 && s.nodes > a.npt};
                    segs[i % kSegRing] = x;
                    mbar_arrive(bar(kSegFull + i % kSegRing));
                }
                __syncwarp();
                if (!more) break;
            }
        } else if (wid == 8 || wid == 12 || wid == 13) {
            // ============================================================ producers (load i by producer i % kProducers)
            const uint64_t once = l2_evict_first_policy(), again = l2_evict_normal_policy();
            Ring<C::kSlots> ring;
            Ring<C::kQSlots> qring;
            int loads = 0, qloads = 0, kblocks = 0;
            const int me = wid == 8 ? 0 : wid - 11;  // warps 8, 12, 13
            int turn = 0;                            // the producer whose load is next
            // one box per lane: slot_rows rows x 64 columns
            const int sl = lane / C::kHalves, hf = lane % C::kHalves;
            auto load_block = [&](const TcSeg& s, int blk, const CUtensorMap* tm, bool is_k) -> bool {
                const bool mine = turn == me;
                const int p = blk * a.spb + sl;
                int page = a.num_total_pages, row = 0;  // page out of range: the copy fills zeros
                bool bad = false;
                if (mine && sl < a.spb && p < s.slots) {
                    const int at = a.cpp > 1 ? p / a.cpp : p;
                    row = (p - at * a.cpp) * a.slot_rows;
                    page = __ldg(a.indices + s.lo + at);
                    bad = page < 0 || page >= a.num_total_pages;
                    if (bad) page = a.num_total_pages;
                }
                // every producer sees every slot come free, so that no barrier gets two phases ahead of it
                if (loads >= C::kSlots && !tree_wait_warp(bar(kEmptyB + ring.slot), ring.phase ^ 1u, abort_flag, a.flags)) return false;
                if (mine) {
                    if (is_k) {
                        const unsigned found = __ballot_sync(kFull, bad);
                        if (lane == 0) {
                            unsigned bits = 0;
                            for (unsigned f = found; f != 0u; f &= f - 1u) bits |= 1u << ((__ffs(f) - 1) / C::kHalves);
                            bad_slots[kblocks % C::kBadRing] = bits;
                            if (bits != 0u) atomicOr(a.flags, kFlagBadPage);
                        }
                    }
                    if (lane == 0) mbar_arrive_expect_tx(bar(kFullB + ring.slot), C::kSlotBytes);
                    __syncwarp();
                    if (sl < a.spb)
                        tma_load_4d(sbase + C::kRingOff + ring.slot * C::kSlotBytes + hf * (C::kKeys * 128) + sl * a.slot_rows * 128,
                                    tm, hf * 64, row, s.kvh, page, bar(kFullB + ring.slot), s.n > a.nps ? again : once);
                }
                kblocks += is_k;
                ++loads;
                ring.next();
                if (++turn == C::kProducers) turn = 0;
                return true;
            };
            tc_steps(
                seg_wait, seg_free,
                [&](const TcStep& w, const TcSeg& s) {
                    if (me == 0 && w.opens_tile()) {
                        if (qloads >= C::kQSlots && !tree_wait_warp(bar(kQEmpty + qring.slot), qring.phase ^ 1u, abort_flag, a.flags))
                            return false;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(bar(kQFull + qring.slot), uint32_t(a.npt * a.hpt) * D * 2);
                            for (int h = 0; h < C::kHalves; ++h)
                                tma_load_3d(sbase + qring.slot * C::kQBytes + h * (C::kRows * 128), &tmq, h * 64, s.head0,
                                            s.row0 + w.row_tile() * a.npt, bar(kQFull + qring.slot));
                        }
                        __syncwarp();
                        ++qloads;
                        qring.next();
                    }
                    return !w.first_use() || load_block(s, w.block(), &tmk, true);
                },
                [&](const TcStep& w, const TcSeg& s) {
                    return !w.first_use() || load_block(s, w.block(), &tmv, false);
                });
            // copies issued last may still be landing when another role has stopped early
            for (int i = max(0, loads - C::kSlots); i < loads; ++i)
                mbar_wait_bounded(bar(kFullB + i % C::kSlots), uint32_t(i / C::kSlots) & 1u);
            for (int i = max(0, qloads - C::kQSlots); i < qloads; ++i)
                mbar_wait_bounded(bar(kQFull + i % C::kQSlots), uint32_t(i / C::kQSlots) & 1u);
        } else if (wid == 9 || (C::kTiles == 2 && wid == 11)) {
            // ============================================================ mma
            // Warp 9 issues for pipeline 0, warp 11 for pipeline 1 (head_dim 256: warp
            // 9 for both S buffers, whose P V add to one O in order). A warp steps
            // over the other's jobs, so that it sees every load land, but does not
            // wait for the other's weights: while one prepares and waits, the tensor
            // cores run what the other has issued.
            const int own = wid == 9 ? 0 : 1;
            if (lane == 0) {
                const uint32_t idesc_s = tc_idesc_f16(kBf16, C::kRows, C::kKeys, false) | (a.scale_log2 < 0.f ? kIdescNegA : 0u);
                constexpr uint32_t idesc_o = tc_idesc_f16(kBf16, C::kRows, D, true);
                // operand descriptors of slot 0 (K K-major, V MN-major) and of q slot 0; addresses count 16 bytes
                const uint64_t kdesc = smem_desc_sw128(sbase + C::kRingOff, 16, 1024);
                const uint64_t vdesc = smem_desc_sw128(sbase + C::kRingOff, C::kKeys * 128, 1024);
                const uint64_t qdesc = smem_desc_sw128(sbase, 16, 1024);
                Ring<C::kSlots> ring;
                Ring<C::kQSlots> qring;
                int kslot = 0, vslot = 0, qtile[2] = {0, 0};
                uint32_t vok = 0;          // phase of each slot's vok barrier
                uint32_t p_phase = 0;      // bit t: phase of pfull t
                auto take = [&](int* slot) {
                    *slot = ring.slot;
                    const bool ok = tree_wait(bar(kFullB + ring.slot), ring.phase, abort_flag, a.flags);
                    ring.next();
                    return ok;
                };
                tc_steps(
                    seg_wait1, seg_free1,
                    [&](const TcStep& w, const TcSeg&) {
                        const int t = w.j & 1, rt = w.row_tile();
                        const bool mine = C::kTiles == 1 || t == own;
                        if (w.opens_tile()) {
                            if (!tree_wait(bar(kQFull + qring.slot), qring.phase, abort_flag, a.flags)) return false;
                            qtile[rt] = qring.slot;
                            qring.next();
                        }
                        if (w.first_use() && !take(&kslot)) return false;
                        const int qs = rt == 0 ? qtile[0] : qtile[1];
                        if (!mine) {
                            if (!w.wide) mbar_arrive(bar(kEmptyB + kslot));
                            if (w.closes_tile()) tc_commit(bar(kQEmpty + qs));
                            return true;
                        }
                        tc_fence_after();
                        const uint64_t kb = kdesc + uint32_t(kslot * (C::kSlotBytes / 16)), qb = qdesc + uint32_t(qs * (C::kQBytes / 16));
                        const uint32_t d = tmem + C::kSCol + t * C::kKeys;
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            tc_mma_f16(d, qb + ((k / 4) * (C::kRows * 128) + (k % 4) * 32) / 16,
                                       kb + ((k / 4) * (C::kKeys * 128) + (k % 4) * 32) / 16, idesc_s, k > 0);
                        tc_commit(bar(kSFull + t));
                        tc_commit(bar(kEmptyB + kslot));
                        if (w.closes_tile()) tc_commit(bar(kQEmpty + qs));
                        return true;
                    },
                    [&](const TcStep& w, const TcSeg&) {
                        const int t = w.j & 1;
                        if (w.first_use()) {
                            if (!take(&vslot)) return false;
                            if (w.tail()) {
                                if (!tree_wait(bar(kVokB + vslot), (vok >> vslot) & 1u, abort_flag, a.flags)) return false;
                                vok ^= 1u << vslot;
                            }
                        }
                        if (C::kTiles == 2 && t != own) {
                            if (!w.wide) mbar_arrive(bar(kEmptyB + vslot));
                            return true;
                        }
                        if (!tree_wait(bar(kPFull + t), (p_phase >> t) & 1u, abort_flag, a.flags)) return false;
                        p_phase ^= 1u << t;
                        tc_fence_after();
                        const uint64_t vb = vdesc + uint32_t(vslot * (C::kSlotBytes / 16));
                        const uint32_t d = tmem + (C::kTiles == 2 ? t * C::kOCols : 0);
                        const bool fresh = C::kTiles == 2 ? w.j < 2 : w.j == 0;
#pragma unroll
                        for (int k = 0; k < C::kKeys / 16; ++k)
                            tc_mma_f16_ta(d, tmem + C::kSCol + t * C::kKeys + 8 * k, vb + k * 128, idesc_o, !fresh || k > 0);
                        tc_commit(bar(kPvDone + t));
                        tc_commit(bar(kEmptyB + vslot));
                        return true;
                    });
                // every mma has completed before the tensor memory is released
                tc_commit(bar(kAllDone + own));
                mbar_wait_bounded(bar(kAllDone + own), 0u);
            }
        } else if (wid >= 14) {
            // ============================================================ V inspectors
            // They see every load land and give every slot back, so that no
            // barrier gets two phases ahead of them.
            Ring<C::kSlots> ring;
            const int t = tid - 448;
            auto landed = [&](int* slot) {
                *slot = ring.slot;
                const bool ok = tree_wait_warp(bar(kFullB + ring.slot), ring.phase, abort_flag, a.flags);
                ring.next();
                return ok;
            };
            tc_steps(
                seg_wait, seg_free,
                [&](const TcStep& w, const TcSeg&) {
                    if (!w.first_use()) return true;
                    int slot;
                    if (!landed(&slot)) return false;
                    if (lane == 0) mbar_arrive(bar(kEmptyB + slot));
                    return true;
                },
                [&](const TcStep& w, const TcSeg& s) {
                    if (!w.first_use()) return true;
                    const int blk = w.block();
                    int slot;
                    if (!landed(&slot)) return false;
                    if (!w.tail()) {
                        if (lane == 0) mbar_arrive(bar(kEmptyB + slot));
                        return true;
                    }
                    uint8_t* vb = smem + C::kRingOff + slot * C::kSlotBytes;
                    constexpr uint32_t kExp = kBf16 ? 0x7f807f80u : 0x7c007c00u;
                    bool found = false;
                    for (int row = t; row < C::kKeys; row += 32 * C::kInspectors) {
                    const int tok = tree_token(a, blk, row);
                    const bool dead = tok < 0 || tok >= s.len, node = tok >= s.len - s.n;
                    if (dead || node) {
                        for (int hf = 0; hf < C::kHalves; ++hf) {
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                uint4* at = reinterpret_cast<uint4*>(vb + hf * (C::kKeys * 128) + row * 128 + ((c ^ (row & 7)) << 4));
                                uint4 x = dead ? make_uint4(0u, 0u, 0u, 0u) : *at;
                                const uint32_t bx = __vcmpeq2(x.x & kExp, kExp), by = __vcmpeq2(x.y & kExp, kExp),
                                               bz = __vcmpeq2(x.z & kExp, kExp), bw = __vcmpeq2(x.w & kExp, kExp);
                                if ((bx | by | bz | bw) != 0u) {
                                    found = true;
                                    x = make_uint4(x.x & ~bx, x.y & ~by, x.z & ~bz, x.w & ~bw);
                                    *at = x;
                                } else if (dead) {
                                    *at = x;
                                }
                            }
                        }
                    }
                    }
                    if (found) bad_v[w.seg & 3] = w.seg + 1;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(kVokB + slot));
                        mbar_arrive(bar(kEmptyB + slot));
                    }
                    return true;
                });
        }
    } else {
        regs_inc<192>();
        // ================================================================ softmax
        const int t = wid >> 2, row = tid & 127;
        if (C::kTiles == 2 || t == 0) {
            const uint32_t lanes = uint32_t(32 * (wid & 3)) << 16;
            const uint32_t to = tmem + lanes + (C::kTiles == 2 ? t * C::kOCols : 0);
            const float scale = a.scale_log2 == 0.f ? 1e-38f : fabsf(a.scale_log2);
            const int per_slot = a.slot_rows < 32 ? a.slot_rows : 32;
            const bool packed = a.page_size % a.slot_rows == 0;
            int n_s[2] = {0, 0}, n_one = 0, n_seg = 0;  // n_s[b]: jobs so far in S buffer b
            int last = 0;                               // S buffer of the last job
            bool dead = false;
            int kblocks = 0;  // K blocks before this segment
            while (!dead) {
                const TcSeg* sp = seg_wait(n_seg);
                TcStep w;
                if (sp == nullptr || !w.enter(*sp)) break;
                const TcSeg& s = *sp;
                const TreeReq r = s.req();
                const int seg = n_seg++;
                const bool joint = C::kTiles == 2 && !w.wide;  // both pipelines hold parts of the same rows
                const int node = s.node0 + (w.wide ? t * a.npt : 0) + row / a.hpt;
                const long long at = tree_row(a, s.row0, s.nodes, s.hh, row + (w.wide ? t * C::kRows : 0));
                const bool live = __any_sync(kFull, at >= 0);  // a warp without rows only keeps step
                float m = kNegInf, l = 0.f;
                // pipeline 1 leaves the last joint segment's O to pipeline 0 until it has been read
                if (t == 1 && n_one > 0 && !tree_wait_warp(bar(kOneFree), uint32_t(n_one - 1) & 1u, abort_flag, a.flags)) break;
                const int step = C::kTiles == 2 ? 2 : 1;
                const int first = C::kTiles == 2 ? t : 0;
                for (int j = first; j < w.jobs; j += step) {
                    w.j = j;
                    const int blk = w.block(), sb = j & 1;
                    if (!tree_wait_warp(bar(kSFull + sb), uint32_t(n_s[sb]++) & 1u, abort_flag, a.flags)) {
                        dead = true;
                        break;
                    }
                    if (live) {
                        tc_fence_after();
                        const uint32_t ts = tmem + lanes + C::kSCol + sb * C::kKeys;
                        uint32_t x[C::kKeys];
#pragma unroll
                        for (int c = 0; c < C::kKeys; c += 32) tmem_ld32(ts + c, x + c);
                        const unsigned bad_pages = bad_slots[(kblocks + blk - s.blk0) % C::kBadRing];
                        tmem_wait_ld();
                        if (!packed || bad_pages != 0u || w.tail()) {
                            const int nd = min(node, r.n - 1);
#pragma unroll
                            for (int c = 0; c < C::kKeys; c += 32) {
                                uint32_t allow = 0;
                                if (packed && bad_pages == 0u) {
                                    allow = tree_allow(a, r, nd, (blk * a.spb) * a.slot_rows + c, 32);
                                } else {
                                    for (int e = 0; e < 32; e += per_slot) {
                                        const int col = c + e, p = blk * a.spb + col / a.slot_rows;
                                        const int r0 = p % a.cpp * a.slot_rows + col % a.slot_rows;
                                        const int count = min(per_slot, a.page_size - r0);
                                        if ((bad_pages >> (col / a.slot_rows)) & 1u) continue;
                                        allow |= tree_allow(a, r, nd, p / a.cpp * a.page_size + r0, count) << e;
                                    }
                                }
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (((allow >> e) & 1u) == 0u) x[c + e] = __float_as_uint(kNegInf);
                            }
                        }
                        float top = __uint_as_float(x[0]);
#pragma unroll
                        for (int c = 1; c < C::kKeys; ++c) top = fmaxf(top, __uint_as_float(x[c]));
                        top *= scale;
                        const bool fresh = C::kTiles == 2 ? j < 2 : j == 0;
                        if (fresh) {
                            m = top;
                        } else {
                            const bool rise = top > m + 8.f;
                            if (__any_sync(kFull, rise)) {
                                const float f = rise ? ex2(m - top) : 1.f;
                                if (rise) m = top;
                                l *= f;
                                // O holds every block before this one once the last P V is done. A
                                // barrier per S buffer: S of this job was issued after the P V before
                                // in its buffer, so no barrier is more than one phase behind.
                                if (!tree_wait_warp(bar(kPvDone + last), uint32_t(n_s[last] - (last == sb ? 2 : 1)) & 1u, abort_flag,
                                                  a.flags)) {
                                    dead = true;
                                    break;
                                }
                                tc_fence_after();
#pragma unroll 1
                                for (int c = 0; c < D; c += 16) {
                                    uint32_t o[16];
                                    tmem_ld16(to + c, o);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                    tmem_st16(to + c, o);
                                }
                            }
                        }
                        const float mu = m == kNegInf ? 0.f : m;
                        float2 sum = make_float2(0.f, 0.f);
                        const float2 sc2 = make_float2(scale, scale), mu2 = make_float2(-mu, -mu);
#pragma unroll
                        for (int c = 0; c < C::kKeys; c += 64) {
                            uint32_t p[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                float2 y = make_float2(__uint_as_float(x[c + 2 * e]), __uint_as_float(x[c + 2 * e + 1]));
                                y = __ffma2_rn(y, sc2, mu2);
                                y = make_float2(ex2(y.x), ex2(y.y));
                                sum = __fadd2_rn(sum, y);
                                p[e] = Elt<T>::pack(y.x, y.y);
                            }
                            tmem_st32(ts + c / 2, p);
                        }
                        l += sum.x + sum.y;
                        tmem_wait_st();
                        tc_fence_before();
                    }
                    last = sb;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kPFull + sb));
                }
                if (dead) break;
                kblocks += s.blk1 - s.blk0;
                // ---- the segment's end
                const int mine = C::kTiles == 2 ? (w.jobs + 1 - t) / 2 : w.jobs;  // jobs of this pipeline
                if (mine > 0 && !tree_wait_warp(bar(kPvDone + last), uint32_t(n_s[last] - 1) & 1u, abort_flag, a.flags)) break;
                tc_fence_after();
                float2 other = make_float2(kNegInf, 0.f);
                if (joint) {
                    if (t == 1) {
                        stat[row] = make_float2(m, l);
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(kOneDone));
                        ++n_one;
                        seg_free(seg);
                        continue;
                    }
                    if (!tree_wait_warp(bar(kOneDone), uint32_t(n_one++) & 1u, abort_flag, a.flags)) break;
                    tc_fence_after();
                    if (w.jobs > 1) other = stat[row];
                }
                const bool two = joint && w.jobs > 1;
                const float mm = fmaxf(m, other.x), mu = mm == kNegInf ? 0.f : mm;
                const float f0 = ex2(m - mu), f1 = ex2(other.x - mu);
                const float L = l * f0 + other.y * f1;
                const float inv = mm == kNegInf ? 0.f : 1.f / L;
                const float lse2 = mm == kNegInf ? kNegInf : mm + log2f(L);
                const float i0 = f0 * inv, i1 = f1 * inv;
                const bool fix = bad_v[seg & 3] == seg + 1;
                if (live) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(to + c, o);
                        float f[32];
                        if (two) {
                            uint32_t o1[32];
                            tmem_ld32(to + C::kOCols + c, o1);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                f[e] = __uint_as_float(o[e]) * i0 + __uint_as_float(o1[e]) * i1;
                        } else {
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]) * i0;
                        }
                        if (fix && at >= 0) {
                            // non-finite elements of the node rows in these blocks, for the rows that attend them
                            for (int i = 0; i < r.n; ++i) {
                                const int tok = r.ctx() + i;
                                const int blk = tree_slots(a, tok + 1) - 1;
                                if (blk / a.spb < s.blk0 || blk / a.spb >= s.blk1) continue;
                                if ((tree_allow(a, r, node, tok, 1) & 1u) == 0u) continue;
                                const int page = __ldg(a.indices + r.lo + tok / a.page_size);
                                if (page < 0 || page >= a.num_total_pages) continue;
                                const T* v = static_cast<const T*>(a.v) +
                                             ((size_t(page) * a.num_kv_heads + s.kvh) * a.page_size + tok % a.page_size) * D + c;
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    const float y = float(v[e]);
                                    if (!isfinite(y)) f[e] += y;
                                }
                            }
                        }
                        if (at >= 0) {
                            if (s.slot >= 0) {
                                float4* po = reinterpret_cast<float4*>(
                                    a.part_o + (size_t(s.slot) * a.seg_rows + row + (w.wide ? t * C::kRows : 0)) * D + c);
#pragma unroll
                                for (int e = 0; e < 8; ++e) po[e] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
                            } else {
                                uint4* po = reinterpret_cast<uint4*>(static_cast<T*>(a.o) + at * D + c);
#pragma unroll
                                for (int e = 0; e < 4; ++e) po[e] = Elt<T>::from_f32(f + 8 * e);
                            }
                        }
                    }
                    if (at >= 0) {
                        if (s.slot >= 0)
                            a.part_lse[size_t(s.slot) * a.seg_rows + row + (w.wide ? t * C::kRows : 0)] = lse2;
                        else
                            a.lse[at] = lse2 == kNegInf ? kNegInf : lse2 * kLn2;
                    }
                }
                if (joint) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kOneFree));
                }
                seg_free(seg);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (wid == 9) tmem_dealloc(tmem, 512);
}

}  // namespace pd
