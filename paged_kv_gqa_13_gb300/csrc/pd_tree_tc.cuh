// Tree decode on the 5th-generation tensor cores (tcgen05.mma kind::f16, f32
// accumulators in tensor memory) for 16-bit q over 16-bit paged pools.
//
// A row tile is up to 128 rows (nodes x q heads of one kv head): the M of both
// products. Per job of 64 keys and row tile: S = Q K^T (A = Q and B = K from
// shared memory, K-major as they lie), then the softmax warps turn S into
// weights P in place (tensor memory), then O += P V (A = P from tensor memory,
// B = V from shared memory, MN-major as it lies).
//
// A pipeline has a row tile's O, two S buffers, an mma warp and 4 softmax
// warps: its next S is computed while its softmax works on the one before.
// Two pipelines share the tensor cores. Where requests have more rows than a
// row tile (kWide) they hold the two row tiles of a segment over the same K and
// V; elsewhere they are lines of their own, each with a range of the work, a
// ring and producers of its own (head_dim 256: one line, for tensor memory
// holds one O).
//
// K and V come in blocks of kKeys keys through a ring of slots, K and V of
// block n as loads 2 n and 2 n + 1 of the line. A wait tells the phases of a
// barrier apart by parity only, so no barrier may get two phases ahead of a
// role that waits on it: whoever waits on a barrier takes part in its next
// phase. The mma warps and inspectors wait for every load and give every slot
// back; a slot is refilled by one producer alone (TreeProducers), which is the
// only one that waits for it to be empty.
//
// Roles beside the softmax warps, per line: an mma warp per pipeline; producers
// (TMA, several: a box of 16 rows x 128 bytes costs its issuing warp about 75
// cycles, and one warp alone kept the ring from filling); inspectors, which make V safe where weights can be zero: a zero
// weight does not undo a NaN or an infinity, so in blocks that hold tokens some
// row does not attend, rows past the end are zeroed and non-finite elements of
// node rows are replaced by zero, to be added to the rows that attend them at
// the end. The first inspector also walks the segments.
//
// E4M3 pools (kFp8): copies bring codes into stages, and converters, in the
// inspectors' place, widen them into the operand slots. Every code is an f16
// value, one conversion per pair of codes (a bf16 value takes four
// instructions), so both products run in f16 for bf16 q too: the softmax warps
// write q rows as f16 times a power of two each.
//
// Rounding. S, maxima, sums and O are f32. The weights are rounded to the
// operand type, at most half a step each, because both operands of a product
// have one type and V is 16-bit in memory: f32 weights would take V widened to
// tf32, twice its bytes in shared memory at half the rate, or two products of
// a weight's two parts. Sums take the weights before rounding, so that lse is
// that of f32 weights. Against 64 bits: bf16 0.0023 of the outputs' norm (f32
// sums rounded once: 0.0017), f16 0.0003 (0.0002).
//
// The running maximum of a row moves only when it rises by more than 2^8 (the
// weights then stay below 2^8, and O, in tensor memory, is rescaled rarely).
//
// What bounds it. Few rows per request: the K and V bytes (32 chains of 4 over
// 512 to 4096 tokens, bf16: 58 us, 65% of the DRAM cycles; 16 requests of head_dim
// 256: 181 us, 78%). Many rows: S, P and O pass through tensor memory once per 64
// keys, so the softmax warps and the two products take turns at 48% tensor
// cycles (64 nodes over 131,072 tokens, f16: 466 to 490 us against 318 for the
// bytes; chunks of 1021 tokens: 414 to 422 us against 245 for the products). E4M3: converting
// and the padding of ragged row tiles (64 trees: 134 us, 39% tensor cycles).
#pragma once

#include "pd_decode_tc.cuh"
#include "pd_tree.cuh"
#include "pd_tree_kernels.h"

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

// Instruction descriptor of kind::f16: 16-bit A and B of one type, f32
// accumulator; b_mn: B is MN-major. kIdescNegA, set in it, negates A.
__host__ __device__ constexpr uint32_t tc_idesc_f16(bool bf16, int M, int N, bool b_mn) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | (uint32_t(N >> 3) << 17) |
           (uint32_t(M >> 4) << 24);
}
constexpr uint32_t kIdescNegA = 1u << 13;

// The tcgen05 instructions of an mma warp: the whole warp runs its code, so
// that descriptors stay in uniform registers, and lane 0 (`lead`) issues.
// D = A * B (+ D when acc), A and B from shared memory.
__device__ __forceinline__ void tc_mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc, bool lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(acc)), "r"(uint32_t(lead))
        : "memory");
}

// The same with A in tensor memory (two 16-bit elements per column).
__device__ __forceinline__ void tc_mma_f16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc, bool lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(acc)), "r"(uint32_t(lead))
        : "memory");
}

__device__ __forceinline__ void tc_commit_if(uint32_t bar, bool lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(uint32_t(lead))
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

// 32 bytes at once: a thread that owns a row writes whole sectors.
__device__ __forceinline__ void store32(void* p, const uint32_t (&r)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// ---------------------------------------------------------------- configuration

// Lines are independent: each walks a range of work of its own through a ring
// of its own. kWide: one line, two pipelines over the same blocks. Otherwise
// two lines of one pipeline (head_dim 256: one, for tensor memory holds one O).
template <int D, bool kWide, bool kFp8>
struct CfgTree {
    static constexpr int kRows = 128;
    static constexpr int kLines = kWide || D == 256 ? 1 : 2;
    static constexpr int kPipes = kWide ? 2 : 1;       // pipelines (row tiles) per line
    static constexpr int kKeys = kWide ? 128 : 64;     // keys per K or V block
    static constexpr int kJobKeys = 64;
    static constexpr int kJobs = kKeys / kJobKeys;     // jobs per block
    static constexpr int kHalves = D / 64;             // 128-byte column blocks of a row
    static constexpr int kSlotBytes = kKeys * D * 2;   // one K or V block
    static constexpr int kQBytes = kRows * D * 2;      // one row tile of q
    static constexpr int kSlots = kFp8 ? (D == 64 ? 4 : 3) : D == 64 ? 10 : 5;
    static constexpr int kStages = kFp8 ? 4 : 0;       // E4M3 pools: blocks of codes on their way
    static constexpr int kStageBytes = kKeys * D;
    // warps of a line after the softmax warps of all lines: mma, producers, inspectors (E4M3 pools: converters)
    static constexpr int kProducers = kFp8 ? (kLines == 2 ? 1 : 2) : kLines == 2 ? 2 : 4;
    static constexpr int kInspectors = kFp8 ? (kLines == 2 ? 2 : 4) : kLines == 2 ? 1 : 2;
    static constexpr int kOthers = kPipes + kProducers + kInspectors;
    static constexpr int kSoftWarps = 4 * kLines * kPipes;
    static constexpr int kThreads = round_up(32 * (kSoftWarps + kLines * kOthers), 128);
    static constexpr int kWalkers = kOthers + 4 * kPipes;  // warps that read a line's segments
    static constexpr int kSegRing = 8;
    // Tags of segments with non-finite V: more than inspectors can be ahead of the softmax warps at a segment's end.
    // V of the next segment is then still in its slot, so that V of at most (kSlots - 1) / 2 more has landed. (Eight
    // tags everywhere: 64 trees over an E4M3 pool 145.0 -> 147.6 us, by other registers.)
    static constexpr int kTags = kSlots > 5 ? kSegRing : 4;
    static_assert(1 + (kSlots - 1) / 2 < kTags, "tags");
    static constexpr int kClaimAhead = kWide ? 3 : 5;
    static constexpr int kSegCost = kWide ? (kFp8 ? 3 : 0) : 3;       // see TreeArgs::seg_cost: an output takes about 5,000 cycles
    static constexpr int kBadRing = 16;  // more than the K blocks that the producers are ahead of the softmax warps
    // a line's barriers (8 bytes each); those of S buffer b of pipeline p at 2 p + b
    static constexpr int kFull = 0, kEmpty = kFull + kSlots, kVok = kEmpty + kSlots, kQFull = kVok + kSlots,
                         kQEmpty = kQFull + kPipes, kQRaw = kQEmpty + kPipes, kSFull = kQRaw + kPipes, kPFull = kSFull + 2 * kPipes,
                         kPvDone = kPFull + 2 * kPipes, kAllDone = kPvDone + 2 * kPipes, kSegFull = kAllDone + kPipes,
                         kSegFree = kSegFull + kSegRing, kStFull = kSegFree + kSegRing, kStEmpty = kStFull + kStages,
                         kBars = kStEmpty + kStages;
    // a line's shared memory: q, ring | barriers, bad-V tags, bad slots, segments (of all lines, after the data)
    static constexpr int kRingOff = kPipes * kQBytes;
    static constexpr int kStageOff = kRingOff + kSlots * kSlotBytes;
    static constexpr int kLineBytes = kStageOff + kStages * kStageBytes;
    static constexpr int kTagOff = round_up(kBars * 8, 16);
    static constexpr int kBadOff = kTagOff + 4 * kTags;
    static constexpr int kSegOff = kBadOff + 4 * kBadRing;
    static constexpr int kCtlBytes = round_up(kSegOff + kSegRing * 68, 8);
    static constexpr int kCtlOff = kLines * kLineBytes;
    static constexpr int kMiscOff = kCtlOff + kLines * kCtlBytes;  // tensor-memory address, abort flag
    static constexpr int kBytes = kMiscOff + 16 + 1024;            // 1024: alignment of the base
    // tensor memory: O of every pipeline, then its two S buffers
    static constexpr int kSCol = kLines * kPipes * D;
    static_assert(kSCol + kLines * kPipes * 2 * kJobKeys <= 512, "tensor memory");
    static_assert(kBytes <= 232448, "shared memory");
    static_assert(kLineBytes % 1024 == 0 && kSlotBytes % 1024 == 0, "operand tiles stay 1024-byte aligned");
};

// Load i of a line goes to place i % kPlaces of its ring, and each place belongs
// to one of the line's producers. That producer has issued every load of the
// place and waits for the one before to be used up, so that the place's empty
// barrier cannot pass the phase that it waits for; a producer that waited for
// places of others could be overtaken by two phases and then see the wrong one.
template <int kPlaces, int kProducers>
struct TreeProducers {
    static_assert(kProducers <= kPlaces, "every producer has a place");
    __host__ __device__ static constexpr bool mine(int place, int me) { return place % kProducers == me; }
};

// Segments come to a line's roles through a ring in shared memory, filled by
// the warp that walks them. blk1 = blk0 ends the line.
struct TcSeg {
    int blk0, blk1, tail0, slots;     // blocks; first block with node tokens; slots of the request
    int slot, row0, node0, nodes;     // partial slot or -1; q rows and nodes of the segment
    int hh, head0, kvh, lo;           // head tile, its first q head and kv head; first entry of indices
    int len, n, start;                // the request: tokens, nodes, first q row
    float k_scale, v_scale;           // of the kv head (E4M3 pools)
    __device__ __forceinline__ TreeReq req() const {
        return TreeReq{n, start, len, lo, 0};
    }
};

static_assert(sizeof(TcSeg) == 68, "CfgTree::kCtlBytes");

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

// Token of column col of block blk; -1 for a row past its page.
__device__ __forceinline__ int tree_token(const TreeArgs& a, int blk, int col) {
    if (a.packed) return (((blk << a.spb_shift)) << a.slot_shift) + col;
    const int s = (blk << a.spb_shift) + (col >> a.slot_shift), page = a.by_cpp.div(s);
    const int row = ((s - page * a.cpp) << a.slot_shift) + col - (col >> a.slot_shift << a.slot_shift);
    return row < a.page_size ? page * a.page_size + row : -1;
}

// ---------------------------------------------------------------- the kernel

template <typename T, int D, bool kWide, bool kFp8>
__global__ void __launch_bounds__(CfgTree<D, kWide, kFp8>::kThreads, 1)
    tree_tc_kernel(const TreeArgs a, const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                   const __grid_constant__ CUtensorMap tmv) {
    using C = CfgTree<D, kWide, kFp8>;
    using M = typename std::conditional<kFp8, __half, T>::type;  // operand type
    constexpr bool kBf16 = std::is_same<M, __nv_bfloat16>::value;
    const float kNegInf = -__int_as_float(0x7f800000);
    extern __shared__ __align__(16) uint8_t tree_tc_smem[];
    uint8_t* base = tree_tc_smem + ((1024u - (smem_u32(tree_tc_smem) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31, wid = __shfl_sync(kFull, tid >> 5, 0);
    // role: softmax warps first; then each line's mma, producers and inspectors
    const bool soft = wid < C::kSoftWarps;
    const int rest = wid - C::kSoftWarps;
    const int line = soft ? wid / (4 * C::kPipes) : rest / C::kOthers;
    // (E4M3 pools: the first line's converters come first, so that both lines' spread over all four schedulers)
    const int part = soft ? 0 : kFp8 && C::kLines == 2 && line == 0 ? (rest + 2) % C::kOthers : rest % C::kOthers;
    const bool idle = line >= C::kLines;
    uint8_t* smem = base + (idle ? 0 : line) * C::kLineBytes;
    uint8_t* ctl = base + C::kCtlOff + (idle ? 0 : line) * C::kCtlBytes;
    const uint32_t sbase = smem_u32(smem), bars = smem_u32(ctl);
    auto bar = [&](int i) { return bars + 8u * uint32_t(i); };
    // of segment i, at i % kTags: i + 1 once non-finite V elements were found
    volatile int* bad_v = reinterpret_cast<volatile int*>(ctl + C::kTagOff);
    // slots of each K block whose page id is bad, by the K block's number in this line
    volatile uint32_t* bad_slots = reinterpret_cast<volatile uint32_t*>(ctl + C::kBadOff);
    TcSeg* segs = reinterpret_cast<TcSeg*>(ctl + C::kSegOff);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(base + C::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(base + C::kMiscOff + 4);
    TreePlanScratch* plan = reinterpret_cast<TreePlanScratch*>(base);  // before the first copy lands there

    if (!soft && !idle && part == 0) {
        if (lane == 0) {
            for (int i = 0; i < C::kSlots; ++i) {
                mbar_init(bar(C::kFull + i), kFp8 ? C::kInspectors : 1);
                mbar_init(bar(C::kEmpty + i), kFp8 ? C::kPipes : C::kPipes + C::kInspectors);  // mma warps and inspectors
                mbar_init(bar(C::kVok + i), C::kInspectors);
            }
            for (int i = 0; i < C::kStages; ++i) {
                mbar_init(bar(C::kStFull + i), 1);
                mbar_init(bar(C::kStEmpty + i), C::kInspectors);
            }
            for (int i = 0; i < C::kPipes; ++i) {
                mbar_init(bar(C::kQFull + i), kFp8 ? 4 : 1);
                mbar_init(bar(C::kQEmpty + i), 1);
                mbar_init(bar(C::kQRaw + i), 1);
                mbar_init(bar(C::kAllDone + i), 1);
            }
            for (int i = 0; i < 2 * C::kPipes; ++i) {
                mbar_init(bar(C::kSFull + i), 1);
                mbar_init(bar(C::kPFull + i), 4);
                mbar_init(bar(C::kPvDone + i), 1);
            }
            for (int i = 0; i < C::kSegRing; ++i) {
                mbar_init(bar(C::kSegFull + i), 1);
                mbar_init(bar(C::kSegFree + i), C::kWalkers);
            }
            fence_mbar_init();
            *abort_flag = 0;
            for (int i = 0; i < C::kTags; ++i) bad_v[i] = 0;
        }
        __syncwarp();
        if (line == 0) tmem_alloc(smem_u32(tslot), 512);
    }
    if (!soft && line == 0 && part == C::kPipes && lane == 0) {
        prefetch_tensormap(&tmq);
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
    }
    tree_plan<C::kLines>(a, plan);
    TreeWalk walk;
    const bool walker = !soft && !idle && part == C::kPipes + C::kProducers;
    const TreeLine cuts = tree_line<C::kLines>(a, plan);
    if (walker) walk = tree_start<C::kLines>(cuts, plan, line);
    tc_fence_before();
    __syncthreads();  // the walks have been read: copies may land
    tc_fence_after();
    launch_dependents();
    const uint32_t tmem = *tslot;

    auto test = [&](int b, uint32_t phase) { return __all_sync(kFull, mbar_test_wait(bar(b), phase)) != 0; };
    auto wait = [&](int b, uint32_t phase) { return tree_wait_warp(bar(b), phase, abort_flag, a.flags); };
    // Segment i, waiting for it, and giving it back.
    auto seg_at = [&](int i) -> const TcSeg& { return segs[i % C::kSegRing]; };
    auto seg_phase = [&](int i) { return uint32_t(i / C::kSegRing) & 1u; };
    auto seg_wait = [&](int i) { return wait(C::kSegFull + i % C::kSegRing, seg_phase(i)); };
    auto seg_free = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kSegFree + i % C::kSegRing));
    };

    if (idle) {
    } else if (!soft && part < C::kPipes) {
        // ================================================================ mma of pipeline `part`
        {
            const bool lead = lane == 0;
            const uint32_t idesc_s = tc_idesc_f16(kBf16, C::kRows, C::kJobKeys, false) | (!kFp8 && a.scale_log2 < 0.f ? kIdescNegA : 0u);
            constexpr uint32_t idesc_o = tc_idesc_f16(kBf16, C::kRows, D, true);
            // operand descriptors of slot 0 (K K-major, V MN-major) and of the row tile's q; addresses count 16 bytes
            const uint64_t kdesc = smem_desc_sw128(sbase + C::kRingOff, 16, 1024);
            const uint64_t vdesc = smem_desc_sw128(sbase + C::kRingOff, C::kKeys * 128, 1024);
            const uint64_t qb = smem_desc_sw128(sbase + part * C::kQBytes, 16, 1024);
            const int pipe = line * C::kPipes + part;
            const uint32_t s_cols = tmem + C::kSCol + pipe * 2 * C::kJobKeys, o_cols = tmem + pipe * D;
            Ring<C::kSlots> ring;
            uint32_t vok = 0;        // phase of each slot's vok barrier
            int n_qk = 0, n_pv = 0;  // jobs issued; job x is in S buffer x & 1
            // The place of the S products: segment and block.
            int seg = -1, blk = 0, blk1 = 0, tail0 = 0, kslot = 0;
            bool first = false;
            auto land = [&](int* slot) {
                *slot = ring.slot;
                const bool ok = wait(C::kFull + ring.slot, ring.phase);
                ring.next();
                return ok;
            };
            // To the next block, waiting until its K has landed (1). 0: none left, -1: stop.
            auto advance = [&]() -> int {
                if (++blk >= blk1) {
                    ++seg;
                    if (!wait(C::kSegFull + seg % C::kSegRing, seg_phase(seg))) return -1;
                    const TcSeg& s = seg_at(seg);
                    if (s.blk0 == s.blk1) return 0;
                    blk = s.blk0;
                    blk1 = s.blk1;
                    tail0 = s.tail0;
                    if (!wait(C::kQFull + part, uint32_t(seg) & 1u)) return -1;
                    first = true;
                }
                return land(&kslot) ? 1 : -1;
            };
            // Whether advance() would not wait.
            auto ready = [&]() {
                if (blk + 1 >= blk1) {
                    const int i = seg + 1;
                    if (!test(C::kSegFull + i % C::kSegRing, seg_phase(i))) return false;
                    if (seg_at(i).blk0 == seg_at(i).blk1) return true;
                    if (!test(C::kQFull + part, uint32_t(i) & 1u)) return false;
                }
                return test(C::kFull + ring.slot, ring.phase);
            };
            auto issue_s = [&](int half) {
                tc_fence_after();
                const uint64_t kb = kdesc + uint32_t(kslot * (C::kSlotBytes / 16) + half * (C::kJobKeys * 8));
                const uint32_t d = s_cols + (n_qk & 1) * C::kJobKeys;
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tc_mma_f16(d, qb + ((k / 4) * (C::kRows * 128) + (k % 4) * 32) / 16,
                               kb + ((k / 4) * (C::kKeys * 128) + (k % 4) * 32) / 16, idesc_s, k > 0, lead);
                tc_commit_if(bar(C::kSFull + 2 * part + (n_qk & 1)), lead);
                if (half == C::kJobs - 1) {
                    tc_commit_if(bar(C::kEmpty + kslot), lead);
                    if (blk + 1 == blk1) {  // the segment's last S
                        tc_commit_if(bar(C::kQEmpty + part), lead);
                        if (lead) mbar_arrive(bar(C::kSegFree + seg % C::kSegRing));
                    }
                }
                ++n_qk;
            };
            int more = advance();
            if (more == 1) issue_s(0);
            while (more == 1) {
                int vs;
                const bool tail = blk >= tail0, fresh = first;
                first = false;
                bool ok = true;
                if (C::kJobs > 1) issue_s(1);
                if (!land(&vs)) break;
                if (!kFp8 && tail) {
                    if (!wait(C::kVok + vs, (vok >> vs) & 1u)) break;
                    vok ^= 1u << vs;
                }
#pragma unroll
                for (int half = 0; half < C::kJobs; ++half) {
                    const int buf = n_pv & 1;
                    const int pfull = C::kPFull + 2 * part + buf;
                    const uint32_t phase = uint32_t(n_pv >> 1) & 1u;
                    bool moved = true;
                    // The next job's S before this job's P V, unless its K comes later than this job's weights.
                    if (half + 1 == C::kJobs) {
                        const long long t0 = clock64();
                        while (!(moved = ready()) && !test(pfull, phase) && !__any_sync(kFull, *abort_flag != 0 || clock64() - t0 > kWaitCycles)) {
                        }
                        if (moved && (more = advance()) == 1) issue_s(0);
                        if (more < 0) {
                            ok = false;
                            break;
                        }
                    }
                    if (!wait(pfull, phase)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t vb = vdesc + uint32_t(vs * (C::kSlotBytes / 16) + half * (C::kJobKeys * 8));
#pragma unroll
                    for (int k = 0; k < C::kJobKeys / 16; ++k)
                        tc_mma_f16_ta(o_cols, s_cols + buf * C::kJobKeys + 8 * k, vb + k * 128, idesc_o,
                                      !fresh || half > 0 || k > 0, lead);
                    tc_commit_if(bar(C::kPvDone + 2 * part + buf), lead);
                    if (half == C::kJobs - 1) tc_commit_if(bar(C::kEmpty + vs), lead);
                    ++n_pv;
                    if (!moved && (more = advance()) == 1) issue_s(0);
                }
                if (!ok) break;
            }
            // every mma has completed before the tensor memory is released
            tc_commit_if(bar(C::kAllDone + part), lead);
            mbar_wait_bounded(bar(C::kAllDone + part), 0u);
        }
    } else if (!soft && part < C::kPipes + C::kProducers) {
        // ================================================================ producers
        const uint64_t once = l2_evict_first_policy(), again = l2_evict_normal_policy();
        const int me = part - C::kPipes;
        // the ring that the copies land in: operand slots, or stages of codes
        constexpr int kPlaces = kFp8 ? C::kStages : C::kSlots, kPlaceFull = kFp8 ? C::kStFull : C::kFull,
                      kPlaceEmpty = kFp8 ? C::kStEmpty : C::kEmpty, kPlaceOff = kFp8 ? C::kStageOff : C::kRingOff,
                      kPlaceBytes = kFp8 ? C::kStageBytes : C::kSlotBytes, kQLanded = kFp8 ? C::kQRaw : C::kQFull;
        using Own = TreeProducers<kPlaces, C::kProducers>;
        Ring<kPlaces> ring;
        int loads = 0, qloads = 0, segments = 0, kblocks = 0;  // loads: of all producers
        bool ok = true;
        // one box per lane: slot_rows rows x 64 columns (codes: x head_dim columns)
        constexpr int kBoxes = kFp8 ? 1 : C::kHalves, kRowBytes = kFp8 ? D : 128;
        const int sl = lane / kBoxes, hf = lane % kBoxes, spb = 1 << a.spb_shift;
        auto load_block = [&](const TcSeg& s, int blk, const CUtensorMap* tm, bool is_k) -> bool {
            if (Own::mine(ring.slot, me)) {
                const int p = (blk << a.spb_shift) + sl;
                int page = a.num_total_pages, row = 0;  // page out of range: the copy fills zeros
                bool bad = false;
                if (sl < spb && p < s.slots) {
                    const int at = a.by_cpp.div(p);
                    row = (p - at * a.cpp) << a.slot_shift;
                    page = __ldg(a.indices + s.lo + at);
                    bad = page < 0 || page >= a.num_total_pages;
                    if (bad) page = a.num_total_pages;
                }
                if (loads >= kPlaces && !wait(kPlaceEmpty + ring.slot, ring.phase ^ 1u)) return false;
                if (is_k) {
                    const unsigned found = __ballot_sync(kFull, bad);
                    if (lane == 0) {
                        unsigned bits = 0;
                        for (unsigned f = found; f != 0u; f &= f - 1u) bits |= 1u << ((__ffs(f) - 1) / kBoxes);
                        bad_slots[kblocks % C::kBadRing] = bits;
                        if (bits != 0u) atomicOr(a.flags, kFlagBadPage);
                    }
                }
                // (test-only: the first copy of all waits for bytes that never arrive)
                const int extra = loads == 0 && blockIdx.x == 0 && line == 0 ? a.test_extra_tx : 0;
                if (lane == 0) mbar_arrive_expect_tx(bar(kPlaceFull + ring.slot), uint32_t(kPlaceBytes + extra));
                __syncwarp();
                if (sl < spb)
                    tma_load_4d(sbase + kPlaceOff + ring.slot * kPlaceBytes + hf * (C::kKeys * 128) + (sl << a.slot_shift) * kRowBytes,
                                tm, hf * 64, row, s.kvh, page, bar(kPlaceFull + ring.slot), s.n > a.nps ? again : once);
            }
            ++loads;
            ring.next();
            return true;
        };
        for (; ok; ++segments) {
            if (!seg_wait(segments)) break;
            const TcSeg& s = seg_at(segments);
            const int blk0 = s.blk0, blk1 = s.blk1;
            if (blk0 == blk1) break;
            for (int p = 0; me == 0 && p < C::kPipes && ok; ++p) {
                // a row tile past the segment's nodes is copied like another (rows of other requests, or zeros) and not used
                ok = segments == 0 || wait(C::kQEmpty + p, uint32_t(segments - 1) & 1u);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(kQLanded + p), uint32_t(a.npt * a.hpt) * D * 2);
                    for (int h = 0; h < C::kHalves; ++h)
                        tma_load_3d(sbase + p * C::kQBytes + h * (C::kRows * 128), &tmq, h * 64, s.head0, s.row0 + p * a.npt,
                                    bar(kQLanded + p));
                }
                __syncwarp();
                ++qloads;
            }
            for (int blk = blk0; blk < blk1 && ok; ++blk, ++kblocks)
                ok = load_block(s, blk, &tmk, true) && load_block(s, blk, &tmv, false);
            if (!ok) break;
            seg_free(segments);
        }
        // copies issued last may still be landing when another role has stopped early
        for (int i = max(0, loads - kPlaces); i < loads; ++i)
            if (Own::mine(i % kPlaces, me)) mbar_wait_bounded(bar(kPlaceFull + i % kPlaces), uint32_t(i / kPlaces) & 1u);
        for (int i = max(0, qloads - C::kPipes); i < qloads; ++i)
            mbar_wait_bounded(bar(kQLanded + i % C::kPipes), uint32_t(i / C::kPipes) & 1u);
    } else if (!soft) {
        // ================================================================ inspectors / converters; the first also walks the segments
        constexpr uint32_t kExp = kBf16 ? 0x7f807f80u : 0x7c007c00u;
        const int me = part - C::kPipes - C::kProducers;
        Ring<C::kSlots> ring;
        Ring<kFp8 ? C::kStages : 1> stage;
        int loads = 0;
        bool ok = true, more = walker;
        int walked = 0;
        // The next segment into its place of the ring (which is free): of this range, or (claim) of the
        // next one that nobody has asked for, or the end. false: this range has no more.
        auto publish = [&](bool claim) -> bool {
            TreeWalk::Seg s;
            TcSeg x{};
            while (!walk.next(a, &s)) {
                if (!claim) return false;
                int range;
                if (!tree_claim(a, cuts, &range)) {
                    more = false;
                    break;
                }
                walk.locate(a, cuts, range);
                if (lane == 0) walk.write_split(a, cuts);
            }
            if (lane == 0) {
                if (more) {
                    x = TcSeg{s.blk0, s.blk1,  s.tail0, s.slots, s.slot,  s.row0, s.node0,   s.nodes,
                              s.hh,   s.head0, s.kvh,   s.r.lo,  s.r.len, s.r.n,  s.r.start, 1.f, 1.f};
                    if (kFp8) {
                        x.k_scale = __ldg(a.k_scale + s.kvh);
                        x.v_scale = __ldg(a.v_scale + s.kvh);
                    }
                }
                segs[walked % C::kSegRing] = x;
                mbar_arrive(bar(C::kSegFull + walked % C::kSegRing));
            }
            __syncwarp();
            ++walked;
            return true;
        };
        // A place for it in the ring; wait for one only when fewer than four segments are ahead of segment i.
        auto place = [&](int i) -> bool {
            if (walked < C::kSegRing) return true;
            const int b = C::kSegFree + walked % C::kSegRing;
            const uint32_t phase = seg_phase(walked) ^ 1u;
            return walked > i + 3 ? test(b, phase) : (ok = wait(b, phase));
        };
        const TreeWalk share = walk;
        for (int i = 0; ok; ++i) {
            while (more && walked < i + C::kSegRing && place(i) && publish(walked == i)) {
            }
            if (walker && i == 0 && lane == 0) share.write_split(a, cuts);
            if (!ok || !seg_wait(i)) break;
            const TcSeg& s = seg_at(i);
            const int blk1 = s.blk1, tail0 = s.tail0, len = s.len, ctx = s.len - s.n;
            if (s.blk0 == blk1) break;
            for (int blk = s.blk0; blk < blk1; ++blk) {
                // ask for more work a few blocks before the last segment's end, so that its copies follow on
                if (more && walked == i + 1 && blk + C::kClaimAhead >= blk1 && place(i)) publish(true);
                if (!ok) break;
                if constexpr (kFp8) {
                    // codes to f16 (exact), 8 at a time, into the operand layout: K, then V
                    for (int kv = 0; kv < 2; ++kv, ++loads, ring.next(), stage.next()) {
                        if (!(ok = wait(C::kStFull + stage.slot, stage.phase))) break;
                        if (loads >= C::kSlots && !(ok = wait(C::kEmpty + ring.slot, ring.phase ^ 1u))) break;
                        const uint8_t* from = smem + C::kStageOff + stage.slot * C::kStageBytes;
                        uint8_t* to = smem + C::kRingOff + ring.slot * C::kSlotBytes;
                        constexpr int kPerRow = D / 8, kStep = 32 * C::kInspectors / kPerRow;  // lanes per row, rows per round
                        const int at = 32 * me + lane, piece = at % kPerRow;
                        const bool guard = kv == 1 && blk >= tail0;
                        bool found = false;
                        const int row0 = at / kPerRow;
                        // rounds of eight rows per lane: all loads, then the conversions and stores
                        constexpr int kRound = C::kKeys / kStep < 8 ? C::kKeys / kStep : 8;
                        const uint8_t* src = from + row0 * D + piece * 8;
                        // row & 7 of the rows of a round: all the same, or (steps of four rows) in turn row0 and row0 + 4
                        static_assert(kStep == 4 || kStep % 8 == 0, "rows of a round");
                        uint8_t* dst = to + piece / 8 * (C::kKeys * 128) + row0 * 128;
                        const uint32_t in_row = uint32_t(((piece & 7) ^ (row0 & 7)) << 4);
#pragma unroll 1
                        for (int r0 = row0; r0 < C::kKeys; r0 += kRound * kStep, src += kRound * kStep * D, dst += kRound * kStep * 128) {
                            uint2 w[kRound];
#pragma unroll
                            for (int x = 0; x < kRound; ++x) w[x] = *reinterpret_cast<const uint2*>(src + x * kStep * D);
                            if (guard) {
#pragma unroll
                                for (int x = 0; x < kRound; ++x) {
                                    const int tok = tree_token(a, blk, r0 + x * kStep);
                                    if (tok >= 0 && tok < ctx) continue;
                                    if (tok < 0 || tok >= len) {
                                        w[x] = make_uint2(0u, 0u);
                                    } else {
                                        const uint32_t nx = __vcmpeq4(w[x].x & 0x7f7f7f7fu, 0x7f7f7f7fu),
                                                       ny = __vcmpeq4(w[x].y & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                        found |= (nx | ny) != 0u;
                                        w[x] = make_uint2(w[x].x & ~nx, w[x].y & ~ny);
                                    }
                                }
                            }
#pragma unroll
                            for (int x = 0; x < kRound; ++x) {
                                *reinterpret_cast<uint4*>(dst + x * kStep * 128 + (in_row ^ (kStep == 4 && x % 2 == 1 ? 64u : 0u))) =
                                    make_uint4(e4m3x2_to_f16x2(w[x].x), e4m3x2_to_f16x2(w[x].x >> 16), e4m3x2_to_f16x2(w[x].y),
                                               e4m3x2_to_f16x2(w[x].y >> 16));
                            }
                        }
                        if (found) bad_v[i % C::kTags] = i + 1;
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(bar(C::kFull + ring.slot));
                            mbar_arrive(bar(C::kStEmpty + stage.slot));
                        }
                    }
                    if (!ok) break;
                } else {
                    if (!(ok = wait(C::kFull + ring.slot, ring.phase))) break;
                    if (lane == 0) mbar_arrive(bar(C::kEmpty + ring.slot));  // K
                    ring.next();
                    if (!(ok = wait(C::kFull + ring.slot, ring.phase))) break;
                    if (blk >= tail0) {
                        uint8_t* vb = smem + C::kRingOff + ring.slot * C::kSlotBytes;
                        bool found = false;
                        for (int row = 32 * me + lane; row < C::kKeys; row += 32 * C::kInspectors) {
                            const int tok = tree_token(a, blk, row);
                            const bool dead = tok < 0 || tok >= len, node = tok >= ctx;
                            if (!dead && !node) continue;
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
                        if (found) bad_v[i % C::kTags] = i + 1;
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(C::kVok + ring.slot));
                    }
                    if (lane == 0) mbar_arrive(bar(C::kEmpty + ring.slot));
                    ring.next();
                }
            }
            seg_free(i);
        }
    } else {
        // ================================================================ softmax of pipeline p
        // f16 weights are 2^7 times larger than their maximum-relative value: still below 2^15, and normal down
        // to 2^-21 of the largest (bf16 has the range of f32)
        constexpr float kShift = kBf16 ? 0.f : 7.f;
        const int pipe = wid >> 2, p = pipe % C::kPipes, row = tid & 127;
        const uint32_t lanes = uint32_t(32 * (wid & 3)) << 16;
        const uint32_t to = tmem + lanes + pipe * D, ts0 = tmem + lanes + C::kSCol + pipe * 2 * C::kJobKeys;
        float scale = a.scale_log2 == 0.f ? 1e-38f : fabsf(a.scale_log2);
        const int per_slot = min(1 << a.slot_shift, 32);
        const bool packed = a.packed != 0, o_wide = (reinterpret_cast<uintptr_t>(a.o) & 31u) == 0;
        int jobs = 0, kblocks = 0;  // kblocks: K blocks before this segment
        bool ok = true;
        auto turn_q = [&](const TcSeg& s, int seg) -> bool {
            // This thread's q row, where the copy put it, as f16 times a power of two that brings its
            // largest element near 2^14 (exact but for elements more than 2^28 below it) and the sign of
            // the score scale.
            const float ks = a.scale_log2 * s.k_scale;
            uint8_t* tile = smem + p * C::kQBytes + row * 128;
            auto piece = [&](int c) { return reinterpret_cast<uint4*>(tile + c / 8 * (C::kRows * 128) + (((c & 7) ^ (row & 7)) << 4)); };
            if (!wait(C::kQRaw + p, uint32_t(seg) & 1u)) return false;
            float big = 0.f;
            if (!std::is_same<T, __half>::value) {
#pragma unroll 8
                for (int c = 0; c < D / 8; ++c) {
                    float f[8];
                    Elt<T>::to_f32(*piece(c), f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(f[e]));
                }
            }
            int up = 0;
            if (big > 0.f) up = max(-126, min(126, 141 - int(__float_as_uint(big) >> 23)));
            const float by = __uint_as_float(uint32_t(127 + up) << 23) * (ks < 0.f ? -1.f : 1.f);
#pragma unroll 8
            for (int c = 0; c < D / 8; ++c) {
                float f[8];
                Elt<T>::to_f32(*piece(c), f);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] *= by;
                *piece(c) = Elt<__half>::from_f32(f);
            }
            scale = ks == 0.f ? 1e-38f : fabsf(ks) * __uint_as_float(uint32_t(127 - up) << 23);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::kQFull + p));
            return true;
        };
        for (int seg = 0; ok; ++seg) {
            if (!seg_wait(seg)) break;
            const TcSeg& s = seg_at(seg);
            const int blk0 = s.blk0, blk1 = s.blk1, tail0 = s.tail0;
            if (blk0 == blk1) break;
            const TreeReq r = s.req();
            const int node = s.node0 + p * a.npt + a.by_hpt.div(row);
            const long long at = tree_row(a, s.row0, s.nodes, s.hh, row + p * C::kRows);
            const bool live = __any_sync(kFull, at >= 0);  // a warp without rows only keeps step
            float m = kNegInf, l = 0.f;
            if (kFp8) {
                if (!(ok = turn_q(s, seg))) break;
            }
            for (int blk = blk0; blk < blk1 && ok; ++blk) {
#pragma unroll 1
                for (int half = 0; half < C::kJobs; ++half) {
                    const int buf = jobs & 1;
                    if (!(ok = wait(C::kSFull + 2 * p + buf, uint32_t(jobs >> 1) & 1u))) break;
                    if (live) {
                        tc_fence_after();
                        const uint32_t ts = ts0 + buf * C::kJobKeys;
                        uint32_t x[C::kJobKeys];
                        tmem_ld32(ts, x);
                        tmem_ld32(ts + 32, x + 32);
                        const unsigned bad_pages = bad_slots[(kblocks + blk - blk0) % C::kBadRing];
                        tmem_wait_ld();
                        if (!packed || bad_pages != 0u || blk >= tail0) {
                            const int nd = min(node, r.n - 1);
#pragma unroll
                            for (int c = 0; c < C::kJobKeys; c += 32) {
                                const int c0 = half * C::kJobKeys + c;
                                uint32_t allow = 0;
                                if (packed && bad_pages == 0u) {
                                    allow = tree_allow(a, r, nd, tree_token(a, blk, c0), 32);
                                } else {
                                    for (int e = 0; e < 32; e += per_slot) {
                                        const int col = c0 + e, x0 = col >> a.slot_shift, q = (blk << a.spb_shift) + x0;
                                        const int page = a.by_cpp.div(q);
                                        const int r0 = ((q - page * a.cpp) << a.slot_shift) + col - (x0 << a.slot_shift);
                                        const int count = min(per_slot, a.page_size - r0);
                                        if ((bad_pages >> x0) & 1u) continue;
                                        allow |= tree_allow(a, r, nd, page * a.page_size + r0, count) << e;
                                    }
                                }
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (((allow >> e) & 1u) == 0u) x[c + e] = __float_as_uint(kNegInf);
                            }
                            __syncwarp();  // tensor-memory accesses are the whole warp's
                        }
                        float tops[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) tops[c] = __uint_as_float(x[c]);
#pragma unroll
                        for (int c = 4; c < C::kJobKeys; ++c) tops[c % 4] = fmaxf(tops[c % 4], __uint_as_float(x[c]));
                        const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * scale;
                        if (blk == blk0 && half == 0) {
                            m = top;
                        } else {
                            const bool rise = top > m + 8.f;
                            if (__any_sync(kFull, rise)) {
                                const float f = rise ? ex2(m - top) : 1.f;
                                if (rise) m = top;
                                l *= f;
                                // O holds every job before this one once the last P V is done. S of this
                                // job was issued after the P V before in its buffer, so that no barrier is
                                // more than one phase behind.
                                if (!(ok = wait(C::kPvDone + 2 * p + (buf ^ 1), uint32_t((jobs - 1) >> 1) & 1u))) break;
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
                        const float mu = m == kNegInf ? 0.f : m - kShift;
                        float2 sums[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                        const float2 sc2 = make_float2(scale, scale), mu2 = make_float2(-mu, -mu);
                        uint32_t w[C::kJobKeys / 2];
#pragma unroll
                        for (int e = 0; e < C::kJobKeys / 2; ++e) {
                            float2 y = make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
                            y = __ffma2_rn(y, sc2, mu2);
                            y = make_float2(ex2(y.x), ex2(y.y));
                            sums[e % 2] = __fadd2_rn(sums[e % 2], y);
                            w[e] = Elt<M>::pack(y.x, y.y);
                        }
                        tmem_st32(ts, w);
                        sums[0] = __fadd2_rn(sums[0], sums[1]);
                        l += sums[0].x + sums[0].y;
                        tmem_wait_st();
                        tc_fence_before();
                    }
                    ++jobs;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::kPFull + 2 * p + buf));
                }
            }
            if (!ok) break;
            kblocks += blk1 - blk0;
            // ---- the segment's end
            if (!wait(C::kPvDone + 2 * p + ((jobs - 1) & 1), uint32_t((jobs - 1) >> 1) & 1u)) break;
            tc_fence_after();
            if (live) {
                // empty by the sum: the maximum passes over scores of NaN, the sum does not
                const float inv = (l == 0.f ? 0.f : 1.f / l) * s.v_scale;
                const float lse2 = l == 0.f ? kNegInf : m - kShift + log2f(l);
                const bool fix = bad_v[seg % C::kTags] == seg + 1;
                const size_t prow = size_t(s.slot) * a.seg_rows + row + p * C::kRows;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    float f[32];
                    __syncwarp();
                    tmem_ld32(to + c, o);
                    tmem_wait_ld();
                    if (at < 0) continue;
#pragma unroll
                    for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]) * inv;
                    if (fix) {
                        // non-finite elements of the node rows in these blocks, for the rows that attend them
                        for (int i = 0; i < r.n; ++i) {
                            const int tok = r.ctx() + i;
                            const int blk = tree_slot_of(a, tok) >> a.spb_shift;
                            if (blk < blk0 || blk >= blk1) continue;
                            if ((tree_allow(a, r, node, tok, 1) & 1u) == 0u) continue;
                            const int page = __ldg(a.indices + r.lo + tok / a.page_size);
                            if (page < 0 || page >= a.num_total_pages) continue;
                            const size_t vrow = ((size_t(page) * a.num_kv_heads + s.kvh) * a.page_size + tok % a.page_size) * D + c;
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                float y;
                                if constexpr (kFp8)  // the only non-finite codes are NaN
                                    y = (static_cast<const uint8_t*>(a.v)[vrow + e] & 0x7f) == 0x7f ? __int_as_float(0x7fc00000) : 0.f;
                                else
                                    y = float(static_cast<const T*>(a.v)[vrow + e]);
                                if (!isfinite(y)) f[e] += y;
                            }
                        }
                    }
                    if (s.slot >= 0) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint32_t v[8];
#pragma unroll
                            for (int x = 0; x < 8; ++x) v[x] = __float_as_uint(f[e + x]);
                            store32(a.part_o + prow * D + c + e, v);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 16) {
                            uint32_t v[8];
#pragma unroll
                            for (int x = 0; x < 8; ++x) v[x] = Elt<T>::pack(f[e + 2 * x], f[e + 2 * x + 1]);
                            T* po = static_cast<T*>(a.o) + at * D + c + e;
                            if (o_wide) {
                                store32(po, v);
                            } else {
                                reinterpret_cast<uint4*>(po)[0] = make_uint4(v[0], v[1], v[2], v[3]);
                                reinterpret_cast<uint4*>(po)[1] = make_uint4(v[4], v[5], v[6], v[7]);
                            }
                        }
                    }
                }
                if (at >= 0) {
                    if (s.slot >= 0)
                        a.part_lse[prow] = tree_part_lse(lse2);
                    else
                        a.lse[at] = lse2 == kNegInf ? kNegInf : lse2 * kLn2;
                }
                tc_fence_before();
            }
            seg_free(seg);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (!soft && line == 0 && part == 0) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- lookup

template <typename T, int D, bool kWide, bool kFp8>
TreeKernels tree_tc_kernels() {
    using C = CfgTree<D, kWide, kFp8>;
    TreeKernels k{};
    k.main = reinterpret_cast<const void*>(tree_tc_kernel<T, D, kWide, kFp8>);
    k.merge = reinterpret_cast<const void*>(tree_merge_kernel<T, D>);
    k.threads = C::kThreads;
    k.smem = C::kBytes;
    k.per_sm = 1;
    k.tile_rows = C::kRows;
    k.tiles = C::kPipes;
    k.workers = C::kLines;
    k.block_tokens = C::kKeys;
    k.seg_cost = C::kSegCost;
    k.tensor = true;
    return k;
}

template <typename T, bool kFp8>
bool tree_tc_lookup(int D, bool wide, TreeKernels* k) {
    switch (D) {
        case 64: *k = wide ? tree_tc_kernels<T, 64, true, kFp8>() : tree_tc_kernels<T, 64, false, kFp8>(); return true;
        case 128: *k = wide ? tree_tc_kernels<T, 128, true, kFp8>() : tree_tc_kernels<T, 128, false, kFp8>(); return true;
        case 256: *k = tree_tc_kernels<T, 256, false, kFp8>(); return true;
    }
    return false;
}

}  // namespace pd
