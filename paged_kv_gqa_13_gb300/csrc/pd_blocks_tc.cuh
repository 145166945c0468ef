// Attention over block-scaled E4M3 pools on the 5th-generation tensor cores
// (tcgen05.mma kind::f8f6f4, accumulators in tensor memory), for one query row
// per request or many, reading the codes where the copies put them.
//
// A code is never widened. The pool is the A operand of both products: per tile
// of 128 tokens S^T[128 tokens][R rows] = K Q^T (A = K as it lies, K-major), and
// O^T[head_dim][R] += V^T P^T (A = V as it lies, MN-major). Rows (nodes x q heads
// of one kv head) are the N of the products, 16 or 32 of them, so that no
// column is spent on rows that are not there, and a token is a lane of tensor memory: its two scales
// are one register each of the thread that owns it,
//
//   x_r = S_r * k_scale * c_r          e_r = 2^(x_r - m_r)          p_r = e_r * v_scale
//
// c_r the row's score scale and m_r the running maximum of x_r + log2 v_scale: of
// what a token can bring to the output, not of its weight alone, so that the
// weights that meet the codes keep their precision whatever the scales are. l_r
// sums e_r, and the output is O_r / l_r.
//
// Parts. Both operands of a product have 8 bits. q goes in as E4M3, which has 4
// significant bits: it is scaled by a power of two for each row (its largest element
// into [128, 256)) and split into parts, each the code nearest to 16 times what the
// part before leaves: two hold a bf16 row and three an f16 row exactly, but for elements
// more than 2^13 (2^14) below the row's largest, which lose at most 2^-21 of it. The
// weights go in as E5M2, 3 significant bits a part but f16's range: p_r, 2^9.5 to 2^15.5
// at the row's maximum, is rounded to f16 and split into parts, each the code nearest to 8
// times what the part before leaves: for a bf16 output three, p_r to 2^-9 of itself
// beside the f16's 2^-11, for an f16 output four, which hold an f16 exactly. What is lost absolutely is 2^-23
// (2^-25) of a weight, 2^-32.5 (2^-34.5) of the largest: a tail of many small weights keeps
// its mass. (As two and three E4M3 parts a weight 2^-16.5 of the largest became
// zero: beside one key 12 above the mean of 16,384, in natural units of the score,
// more than half of their mass was gone.) Parts are further columns of a product (an instruction
// takes as long for 16 columns as for 128), added up in f32: those of S when it is read, those
// of O at the end. l takes the f32 weights before rounding. S, x, sums and O are f32.
//
// The maximum of a row moves only when it is passed by more than 6 (a factor of
// 64), or when a row that has attended nothing so far has its first score; whether one is, is a
// vote of the four warps of a tile. A row then takes the
// new maximum over all 128 tokens, and O is rescaled in tensor memory.
//
// Lines, segments, ranges, tails and the merge are those of the tree decode
// (pd_tree.cuh, pd_tree_tc.cuh), with blocks of 128 tokens and a ring of K and V
// slots for each line. Roles of a line: four softmax warps (a thread owns a token),
// an mma warp, producers (TMA copies of the codes, cp.async of the scales), and a
// warp that walks the segments and writes the parts of a segment's q ahead of time.
//
// What bounds it. Not the products: one instruction takes 80 to 90 cycles to issue
// whatever N is up to 128, 4 for S and 4 for O of a tile at head_dim 128, about 14 TB/s of
// codes on 152 SMs, and the tensor pipe is 3 % busy. What does not grow with the work
// (partition, q's parts, first copies, the slowest line, the merge), 45 to 50 us between
// events: 58 us over a floor of 11 (32 requests of 512 to 4096 tokens, 4 kv heads of 128, 16
// rows, bf16), 93 over 40 (4 of 65,536), 208 over 158 (4 of 131,072, 8 kv heads, 4 rows), 91
// over 44 (32 short ones, 16 kv heads, one row; widened codes: 209). Which part of it is not
// measured; one CTA over one tile takes 13. From 17 rows on see pick_blocks.
//
// Whoever waits on a barrier takes part in its next phase, or waits for a load
// whose slot cannot be filled again before it has given its weights.
#pragma once

#include "pd_tree_tc.cuh"

namespace pd {

// ---------------------------------------------------------------- PTX wrappers

// Matrix descriptor; mode 2: 128-byte swizzle, 4: 64-byte swizzle, 0: none. For an MN-major operand without swizzle: 16
// bytes along N, 8 rows of K, sbo between blocks of 16 along N, lbo between groups of 8 along K.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, int mode) {
    return uint64_t((addr >> 4) & 0x3fffu) | (uint64_t((lbo >> 4) & 0x3fffu) << 16) |
           (uint64_t((sbo >> 4) & 0x3fffu) << 32) | (uint64_t(1) << 46) | (uint64_t(mode) << 61);
}

// A of E4M3, B of E4M3 or E5M2
__host__ __device__ constexpr uint32_t tc_idesc_codes(int M, int N, bool a_mn, bool b_mn, bool b_e5m2) {
    return (1u << 4) | (b_e5m2 ? 1u << 10 : 0u) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

// D (tensor memory) = A * B (+ D when acc), issued by lane 0 (`lead`) of a warp.
__device__ __forceinline__ void tc_mma_codes(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc, bool lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(acc)), "r"(uint32_t(lead))
        : "memory");
}

// The largest of a warp's values (NaN has no say).
__device__ __forceinline__ float redux_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// The E5M2 codes nearest to a pair, and their values: an E5M2 code is the upper byte of an f16.
__device__ __forceinline__ uint32_t half2_e5m2(__half2 h) {
    __half2_raw r;
    memcpy(&r, &h, 4);
    return uint32_t(__nv_cvt_halfraw2_to_fp8x2(r, __NV_SATFINITE, __NV_E5M2));
}
__device__ __forceinline__ __half2 e5m2_half2(uint32_t w) {
    const uint32_t x = __byte_perm(w, 0u, 0x1404);
    __half2 h;
    memcpy(&h, &x, 4);
    return h;
}
__device__ __forceinline__ __half2 codes_half2(uint32_t w) {
    const uint32_t x = e4m3x2_to_f16x2(w);
    __half2 h;
    memcpy(&h, &x, 4);
    return h;
}

// ---------------------------------------------------------------- configuration

// kParts: of an element of q (f16: 3, bf16: 2). A weight has one more.
template <int D, int R, int kParts>
struct CfgBlocks {
    static constexpr int kKeys = 128;                     // tokens of a tile, the M of S^T
    static_assert(R == 16 || R == 32, "rows of a segment");
    static constexpr int kLines = D <= 128 && kParts * R <= 64 ? 2 : 1;  // what tensor memory holds
    static constexpr int kRowBytes = D < 128 ? D : 128;   // of a column block of codes
    static constexpr int kColBlocks = D / kRowBytes;
    static constexpr int kMode = kRowBytes == 128 ? 2 : 4;
    static constexpr int kSlotBytes = kKeys * D;
    static constexpr int kQRows = kParts * R, kQBytes = kQRows * D;  // part p of row r is row p R + r
    static constexpr int kQBufs = 2;
    static constexpr int kPParts = kParts + 1, kPPart = kKeys * R, kPBytes = kPParts * kPPart, kPBufs = 2;
    static constexpr int kProducers = kLines == 2 ? 2 : 4;
    static constexpr int kOthers = 2 + kProducers;        // mma, producers, walker
    static constexpr int kSoftWarps = 4;                  // of a line
    static constexpr int kThreads = 32 * kLines * (kSoftWarps + kOthers);
    static constexpr int kWalkers = 1 + kProducers + kSoftWarps;  // warps that read a line's segments
    static constexpr int kSegRing = 8, kBadRing = 16, kMaxSlots = 10;
    static constexpr int kScales = kMaxSlots / 2 + 3;     // tiles whose scales are held: see load_block
    // a line's barriers (8 bytes each)
    static constexpr int kFull = 0, kEmpty = kFull + kMaxSlots, kScFull = kEmpty + kMaxSlots, kQFull = kScFull + kScales,
                         kQEmpty = kQFull + 2, kSFull = kQEmpty + 2, kPFull = kSFull + 2, kPvDone = kPFull + 2,
                         kVote = kPvDone + 2, kSegFull = kVote + 1, kSegFree = kSegFull + kSegRing,
                         kAllDone = kSegFree + kSegRing, kBars = kAllDone + 1;
    // a line's small shared memory
    static constexpr int kRowcOff = round_up(kBars * 8, 16);              // [kQBufs][R] score scale of a row
    static constexpr int kRowAtOff = kRowcOff + kQBufs * R * 4;           // [kQBufs][R] its q row, -1: none
    static constexpr int kNodeOff = kRowAtOff + kQBufs * R * 8;           // [kQBufs][R] its node
    static constexpr int kWarpOff = round_up(kNodeOff + kQBufs * R * 4, 16);  // per softmax warp: c, -m, a factor, a rise [R] each
    static constexpr int kRedOff = kWarpOff + kSoftWarps * 4 * R * 4;     // [maxima, sums][warp][R]
    static constexpr int kVoteOff = kRedOff + 2 * kSoftWarps * R * 4;     // [2]
    static constexpr int kTagOff = kVoteOff + 2 * 4;                          // [2] segment with non-finite V
    static constexpr int kBadOff = kTagOff + 2 * 4;
    static constexpr int kProgressOff = kBadOff + kBadRing * 4;
    static constexpr int kSegOff = round_up(kProgressOff + 4, 8);
    static constexpr int kScaleOff = round_up(kSegOff + kSegRing * 68, 16);   // [kScales][K, V][kKeys]
    static constexpr int kCtlBytes = round_up(kScaleOff + kScales * 2 * kKeys * 4, 16);
    // a line's operands: q parts, P parts, ring
    static constexpr int kFixed = kQBufs * kQBytes + kPBufs * kPBytes;
    static constexpr int kRoom = (232448 - 1024 - 16) / kLines - kCtlBytes - kFixed;
    static constexpr int kFits = kRoom / kSlotBytes;
    static constexpr int kSlots = kFits < kMaxSlots ? kFits : kMaxSlots;
    static constexpr int kPOff = kQBufs * kQBytes;
    static constexpr int kRingOff = kFixed;
    static constexpr int kLineBytes = kFixed + kSlots * kSlotBytes;
    static constexpr int kCtlOff = kLines * kLineBytes;
    static constexpr int kMiscOff = kCtlOff + kLines * kCtlBytes;  // tensor-memory address, abort flag
    static constexpr int kBytes = kMiscOff + 16 + 1024;            // 1024: alignment of the base
    // tensor memory of a line: two S buffers (a column for each part of a row), then for each column block O of each part
    // of the weights
    static constexpr int kOCol = 2 * kQRows;
    static constexpr int kLineCols = kOCol + kColBlocks * kPParts * R;
    static_assert(kLines * kLineCols <= 512, "tensor memory");
    static_assert(kSlots >= 3 && kBytes <= 232448, "shared memory");
    static_assert(kLineBytes % 1024 == 0 && kQBytes % 1024 == 0 && kPBytes % 1024 == 0 && kSlotBytes % 1024 == 0, "alignment");
    // In tiles. (At 6, 8, 12 or 24 some shapes are 4 to 7 us faster and others 10 slower: where the work is small, the first
    // lines then have a segment's cost and no tile.)
    static constexpr int kSegCost = 2;
    static constexpr int kClaimAhead = 4;
};

// ---------------------------------------------------------------- the kernel

template <typename T, int D, int R>
__global__ void __launch_bounds__(CfgBlocks<D, R, std::is_same<T, __half>::value ? 3 : 2>::kThreads, 1)
    blocks_tc_kernel(const TreeArgs a, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
    constexpr int kParts = std::is_same<T, __half>::value ? 3 : 2;
    using C = CfgBlocks<D, R, kParts>;
    constexpr int kPParts = C::kPParts;
    constexpr float kShift = 9.5f, kRise = 6.f;  // weights: 2^kShift at the maximum, at most 2^(kShift + kRise) < 57344
    const float kNegInf = -__int_as_float(0x7f800000);
    extern __shared__ __align__(16) uint8_t blocks_smem[];
    uint8_t* base = blocks_smem + ((1024u - (smem_u32(blocks_smem) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31, wid = __shfl_sync(kFull, tid >> 5, 0);
    const bool soft = wid < C::kLines * C::kSoftWarps;
    const int rest = wid - C::kLines * C::kSoftWarps;
    const int line = soft ? wid / C::kSoftWarps : rest / C::kOthers;
    const int part = soft ? 0 : rest % C::kOthers;  // 0: mma, then producers, last: walker
    uint8_t* smem = base + line * C::kLineBytes;
    uint8_t* ctl = base + C::kCtlOff + line * C::kCtlBytes;
    const uint32_t sbase = smem_u32(smem), bars = smem_u32(ctl);
    auto bar = [&](int i) { return bars + 8u * uint32_t(i); };
    float* rowc = reinterpret_cast<float*>(ctl + C::kRowcOff);
    long long* rowat = reinterpret_cast<long long*>(ctl + C::kRowAtOff);
    int* rownode = reinterpret_cast<int*>(ctl + C::kNodeOff);
    volatile int* tag = reinterpret_cast<volatile int*>(ctl + C::kTagOff);
    volatile uint32_t* bad_slots = reinterpret_cast<volatile uint32_t*>(ctl + C::kBadOff);
    volatile int* progress = reinterpret_cast<volatile int*>(ctl + C::kProgressOff);
    TcSeg* segs = reinterpret_cast<TcSeg*>(ctl + C::kSegOff);
    const float* scales = reinterpret_cast<const float*>(ctl + C::kScaleOff);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(base + C::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(base + C::kMiscOff + 4);
    TreePlanScratch* plan = reinterpret_cast<TreePlanScratch*>(base);  // before the first copy lands there

    if (!soft && part == 0) {
        if (lane == 0) {
            for (int i = 0; i < C::kSlots; ++i) {
                mbar_init(bar(C::kFull + i), 1);
                mbar_init(bar(C::kEmpty + i), 1);
            }
            for (int i = 0; i < C::kScales; ++i) mbar_init(bar(C::kScFull + i), 32);
            for (int i = 0; i < 2; ++i) {
                mbar_init(bar(C::kQFull + i), 1);
                mbar_init(bar(C::kQEmpty + i), 1 + C::kSoftWarps);
                mbar_init(bar(C::kSFull + i), 1);
                mbar_init(bar(C::kPFull + i), C::kSoftWarps);
                mbar_init(bar(C::kPvDone + i), 1);
                tag[i] = 0;
            }
            mbar_init(bar(C::kVote), C::kSoftWarps);
            for (int i = 0; i < C::kSegRing; ++i) {
                mbar_init(bar(C::kSegFull + i), 1);
                mbar_init(bar(C::kSegFree + i), C::kWalkers);
            }
            mbar_init(bar(C::kAllDone), 1);
            fence_mbar_init();
            int* votes = reinterpret_cast<int*>(ctl + C::kVoteOff);
            votes[0] = votes[1] = 0;
            *progress = 0;
            *abort_flag = 0;
        }
        __syncwarp();
        if (line == 0) tmem_alloc(smem_u32(tslot), 512);
    }
    if (!soft && line == 0 && part == 1 && lane == 0) {
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
    }
    tree_plan<C::kLines>(a, plan);
    const TreeLine cuts = tree_line<C::kLines>(a, plan);
    const bool walker = !soft && part == C::kOthers - 1;
    TreeWalk walk;
    if (walker) walk = tree_start<C::kLines>(cuts, plan, line);
    tc_fence_before();
    __syncthreads();  // the walks have been read: copies may land
    tc_fence_after();
    launch_dependents();
    const uint32_t tmem = *tslot + uint32_t(line * C::kLineCols);

    auto test = [&](int b, uint32_t phase) { return __all_sync(kFull, mbar_test_wait(bar(b), phase)) != 0; };
    auto wait = [&](int b, uint32_t phase) { return tree_wait_warp(bar(b), phase, abort_flag, a.flags); };
    auto seg_at = [&](int i) -> const TcSeg& { return segs[i % C::kSegRing]; };
    auto seg_phase = [&](int i) { return uint32_t(i / C::kSegRing) & 1u; };
    auto seg_wait = [&](int i) { return wait(C::kSegFull + i % C::kSegRing, seg_phase(i)); };
    auto seg_free = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kSegFree + i % C::kSegRing));
    };
    auto q_buf = [&](int seg) { return seg % C::kQBufs; };
    auto q_phase = [&](int seg) { return uint32_t(seg / C::kQBufs) & 1u; };

    if (!soft && part == 0) {
        // ================================================================ mma
        const bool lead = lane == 0;
        constexpr uint32_t idesc_s = tc_idesc_codes(C::kKeys, C::kQRows, false, false, false), idesc_o = tc_idesc_codes(128, kPParts * R, true, true, true);
        constexpr uint32_t kGroup = 8 * C::kRowBytes;  // bytes of 8 rows
        const uint64_t kdesc = smem_desc(sbase + C::kRingOff, 16, kGroup, C::kMode);
        // (head_dim 64: M is 128 all the same, its second half the first once more, at no step)
        const uint64_t vdesc = smem_desc(sbase + C::kRingOff, 0, kGroup, C::kMode);
        const uint64_t qdesc = smem_desc(sbase, 16, kGroup, C::kMode);
        const uint64_t pdesc = smem_desc(sbase + C::kPOff, 128, 2048, 0);
        Ring<C::kSlots> ring;
        int n_qk = 0, n_pv = 0;
        int seg = -1, blk = 0, blk1 = 0, kslot = 0;
        bool first = false;
        auto land = [&](int* slot) {
            *slot = ring.slot;
            const bool ok = wait(C::kFull + ring.slot, ring.phase);
            ring.next();
            return ok;
        };
        // To the next tile, waiting until its K has landed (1). 0: none left, -1: stop.
        auto advance = [&]() -> int {
            if (++blk >= blk1) {
                ++seg;
                if (!seg_wait(seg)) return -1;
                const TcSeg& s = seg_at(seg);
                if (s.blk0 == s.blk1) return 0;
                blk = s.blk0;
                blk1 = s.blk1;
                if (!wait(C::kQFull + q_buf(seg), q_phase(seg))) return -1;
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
                if (!test(C::kQFull + q_buf(i), q_phase(i))) return false;
            }
            return test(C::kFull + ring.slot, ring.phase);
        };
        auto issue_s = [&]() {
            tc_fence_after();
            const uint64_t kb = kdesc + uint32_t(kslot * (C::kSlotBytes / 16)), qb = qdesc + uint32_t(q_buf(seg) * (C::kQBytes / 16));
            const uint32_t d = tmem + (n_qk & 1) * C::kQRows;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                const int cb = k * 32 / C::kRowBytes, in = k * 32 % C::kRowBytes;
                tc_mma_codes(d, kb + (cb * C::kKeys * C::kRowBytes + in) / 16, qb + (cb * C::kQRows * C::kRowBytes + in) / 16, idesc_s, k > 0, lead);
            }
            tc_commit_if(bar(C::kSFull + (n_qk & 1)), lead);
            if (blk + 1 == blk1) {  // the segment's last S
                tc_commit_if(bar(C::kQEmpty + q_buf(seg)), lead);
                if (lead) mbar_arrive(bar(C::kSegFree + seg % C::kSegRing));
            }
            ++n_qk;
            if (lead) *progress = n_qk;
        };
        int more = advance();
        if (more == 1) issue_s();
        while (more == 1) {
            int vs;
            const bool fresh = first;
            first = false;
            if (!land(&vs)) break;
            const int buf = n_pv % C::kPBufs;
            const int pfull = C::kPFull + buf;
            const uint32_t phase = uint32_t(n_pv / C::kPBufs) & 1u;
            // The next tile's S before this tile's P V, unless its K comes later than this tile's weights.
            bool moved;
            const long long t0 = clock64();
            while (!(moved = ready()) && !test(pfull, phase) && !__any_sync(kFull, *abort_flag != 0 || clock64() - t0 > kWaitCycles)) {
            }
            if (moved && (more = advance()) == 1) issue_s();
            if (more < 0) break;
            if (!wait(pfull, phase)) break;
            tc_fence_after();
            const uint64_t vb = vdesc + uint32_t(vs * (C::kSlotBytes / 16)), pb = pdesc + uint32_t(buf * (C::kPBytes / 16));
#pragma unroll
            for (int cb = 0; cb < C::kColBlocks; ++cb)
#pragma unroll
                for (int k = 0; k < C::kKeys / 32; ++k)
                    tc_mma_codes(tmem + C::kOCol + cb * kPParts * R, vb + (cb * C::kKeys * C::kRowBytes + k * 32 * C::kRowBytes) / 16,
                                 pb + k * 512 / 16, idesc_o, !fresh || k > 0, lead);
            tc_commit_if(bar(C::kPvDone + buf), lead);
            tc_commit_if(bar(C::kEmpty + vs), lead);
            ++n_pv;
            if (!moved && (more = advance()) == 1) issue_s();
        }
        // every mma has completed before the tensor memory is released
        tc_commit_if(bar(C::kAllDone), lead);
        mbar_wait_bounded(bar(C::kAllDone), 0u);
    } else if (!soft && !walker) {
        // ================================================================ producers
        const uint64_t once = l2_evict_first_policy(), again = l2_evict_normal_policy();
        const int me = part - 1;
        using Own = TreeProducers<C::kSlots, C::kProducers < C::kSlots ? C::kProducers : C::kSlots>;
        const bool idle = me >= C::kSlots;
        Ring<C::kSlots> ring;
        Ring<C::kScales> sc;
        int loads = 0, kblocks = 0;  // of all producers
        bool ok = true;
        // one box per lane: slot_rows rows x kRowBytes codes
        const int sl = lane / C::kColBlocks, cb = lane % C::kColBlocks, spb = 1 << a.spb_shift;
        // The page and row of this lane's box in block blk; a page out of range makes the copy fill zeros.
        struct Box {
            int page, row;
            bool bad;
        };
        auto look_up = [&](const TcSeg& s, int blk) {
            const int p = (blk << a.spb_shift) + sl;
            Box x{a.num_total_pages, 0, false};
            if (sl < spb && p < s.slots) {
                const int at = a.by_cpp.div(p);
                x.row = (p - at * a.cpp) << a.slot_shift;
                x.page = __ldg(a.indices + s.lo + at);
            }
            return x;
        };
        auto load_block = [&](const TcSeg& s, int blk, const Box& box, const CUtensorMap* tm, bool is_k) -> bool {
            if (!idle && Own::mine(ring.slot, me)) {
                if (loads >= C::kSlots && !wait(C::kEmpty + ring.slot, ring.phase ^ 1u)) return false;
                if (is_k) {
                    const unsigned found = __ballot_sync(kFull, box.bad);
                    if (lane == 0) {
                        unsigned bits = 0;
                        for (unsigned f = found; f != 0u; f &= f - 1u) bits |= 1u << ((__ffs(f) - 1) / C::kColBlocks);
                        bad_slots[kblocks % C::kBadRing] = bits;
                        if (bits != 0u) atomicOr(a.flags, kFlagBadPage);
                    }
                }
                // (test-only: the first copy of all waits for bytes that never arrive)
                const int extra = loads == 0 && blockIdx.x == 0 && line == 0 ? a.test_extra_tx : 0;
                if (lane == 0) mbar_arrive_expect_tx(bar(C::kFull + ring.slot), uint32_t(C::kSlotBytes + extra));
                __syncwarp();
                if (sl < spb)
                    tma_load_4d(sbase + C::kRingOff + ring.slot * C::kSlotBytes + cb * (C::kKeys * C::kRowBytes) + (sl << a.slot_shift) * C::kRowBytes,
                                tm, cb * C::kRowBytes, box.row, s.kvh, box.page, bar(C::kFull + ring.slot), s.n > a.nps ? again : once);
                if (!is_k) {
                    // The place is free: the copy before in this slot was of K or V of a tile kSlots / 2 before at least, its
                    // product is done, and so are the weights of the tile two before that one.
                    copy_scales<C::kKeys, C::kColBlocks>(a, s.kvh, s.len, blk, box.page, box.row, smem_u32(scales) + uint32_t(sc.slot * 2 * C::kKeys * 4),
                                                         bar(C::kScFull + sc.slot));
                }
            }
            ++loads;
            ring.next();
            if (!is_k) sc.next();
            return true;
        };
        for (int i = 0; ok; ++i) {
            if (!seg_wait(i)) break;
            const TcSeg& s = seg_at(i);
            const int blk0 = s.blk0, blk1 = s.blk1;
            if (blk0 == blk1) break;
            Box next = look_up(s, blk0);
            for (int blk = blk0; blk < blk1 && ok; ++blk, ++kblocks) {
                Box box = next;
                box.bad = box.page < 0 || box.page > a.num_total_pages || (box.page == a.num_total_pages && sl < spb && (blk << a.spb_shift) + sl < s.slots);
                if (box.bad) box.page = a.num_total_pages;
                if (blk + 1 < blk1) next = look_up(s, blk + 1);  // one block ahead of its use
                ok = load_block(s, blk, box, &tmk, true) && load_block(s, blk, box, &tmv, false);
            }
            if (!ok) break;
            seg_free(i);
        }
        // copies issued last may still be landing when another role has stopped early
        for (int i = max(0, loads - C::kSlots); !idle && i < loads; ++i)
            if (Own::mine(i % C::kSlots, me)) mbar_wait_bounded(bar(C::kFull + i % C::kSlots), uint32_t(i / C::kSlots) & 1u);
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (walker) {
        // ================================================================ segments, and the parts of their q
        constexpr int kPer = D / 32;  // elements of a row per lane
        int walked = 0, tiles = 0;    // published; tiles of them
        bool more = true, own = true, ok = true;
        const TreeWalk share = walk;
        // The next segment into its place of the ring; `claim`: of a range nobody has asked for where this one has no more
        // (asked for when few of the published tiles are left), or the end. false: nothing published.
        auto publish = [&](bool claim) -> bool {
            if (walked >= C::kSegRing && !wait(C::kSegFree + walked % C::kSegRing, seg_phase(walked) ^ 1u)) return ok = false;
            TreeWalk::Seg s;
            TcSeg x{};
            while (!walk.next(a, &s)) {
                own = false;
                if (!claim) return false;
                if (cuts.tail != 0) {
                    const long long t0 = clock64();
                    while (*progress < tiles - C::kClaimAhead) {
                        if (__any_sync(kFull, *abort_flag != 0 || clock64() - t0 > kWaitCycles)) return ok = false;
                        __nanosleep(100);
                    }
                    __syncwarp();
                }
                int range;
                if (!tree_claim(a, cuts, &range)) {
                    more = false;
                    break;
                }
                walk.locate(a, cuts, range);
                if (lane == 0) walk.write_split(a, cuts);
            }
            if (more) {
                x = TcSeg{s.blk0, s.blk1,  s.tail0, s.slots, s.slot,  s.row0, s.node0,   s.nodes,
                          s.hh,   s.head0, s.kvh,   s.r.lo,  s.r.len, s.r.n,  s.r.start, 1.f, 1.f};
                tiles += s.blk1 - s.blk0;
            }
            if (lane == 0) {
                segs[walked % C::kSegRing] = x;
                mbar_arrive(bar(C::kSegFull + walked % C::kSegRing));
            }
            __syncwarp();
            ++walked;
            return true;
        };
        for (int i = 0; ok; ++i) {
            while (ok && more && walked <= i && publish(true)) {
            }
            if (i == 0 && lane == 0) share.write_split(a, cuts);
            // segments of this range ahead, for the producers
            while (ok && more && own && walked < i + 3 && publish(false)) {
            }
            if (!ok) break;
            const TcSeg s = seg_at(i);
            if (s.blk0 == s.blk1) break;
            const int qb = q_buf(i), rows = min(R, (s.nodes * a.hpt + 7) & ~7);
            if (i >= C::kQBufs && !wait(C::kQEmpty + qb, q_phase(i) ^ 1u)) break;
            uint8_t* to = smem + qb * C::kQBytes;
            for (int r0 = 0; r0 < rows; r0 += 8) {
                uint32_t w[8][kPer / 2];
                long long mine = -1;  // lane x: the q row of row r0 + x
                if (lane < 8) mine = tree_row(a, s.row0, s.nodes, s.hh, r0 + lane);
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const long long at = __shfl_sync(kFull, mine, x);
                    const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.q) + (at < 0 ? 0 : at) * D) + lane * (kPer / 2);
#pragma unroll
                    for (int y = 0; y < kPer / 2; ++y) w[x][y] = at >= 0 ? __ldg(src + y) : 0u;
                }
                float mine_c = 0.f;
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int r = r0 + x;
                    float f[kPer];
#pragma unroll
                    for (int y = 0; y < kPer / 2; ++y) {
                        const float2 v = unpack_pair<T>(w[x][y]);
                        f[2 * y] = v.x;
                        f[2 * y + 1] = v.y;
                    }
                    float big = 0.f;
#pragma unroll
                    for (int y = 0; y < kPer; ++y) big = fmaxf(big, fabsf(f[y]));
                    big = redux_max(big);
                    // 2^-e brings the largest element into [128, 256)
                    const int e = max(-119, min(120, int(__float_as_uint(big) >> 23) - 127 - 7));
                    const float by = __uint_as_float(uint32_t(127 - e) << 23);
                    if (lane == x) mine_c = big <= 3.402823466e38f ? a.scale_log2 * __uint_as_float(uint32_t(127 + e) << 23) : __int_as_float(0x7fc00000);
#pragma unroll
                    for (int y = 0; y < kPer; ++y) f[y] *= by;
#pragma unroll
                    for (int p = 0; p < kParts; ++p) {
                        uint32_t codes[(kPer + 3) / 4] = {};
#pragma unroll
                        for (int y = 0; y < kPer; y += 2) {
                            const uint32_t c2 = uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(f[y], f[y + 1]), __NV_SATFINITE, __NV_E4M3));
                            codes[y / 4] |= c2 << (8 * (y % 4));
                            const float2 got = __half22float2(codes_half2(c2));
                            f[y] = (f[y] - got.x) * 16.f;
                            f[y + 1] = (f[y + 1] - got.y) * 16.f;
                        }
                        const int x0 = lane * kPer, col = x0 / C::kRowBytes, in = x0 % C::kRowBytes;
                        const int sw = C::kMode == 2 ? r & 7 : (r >> 1) & 3;
                        uint8_t* dst = to + col * (C::kQRows * C::kRowBytes) + (p * R + r) * C::kRowBytes + (((in >> 4) ^ sw) << 4) + (in & 15);
                        if constexpr (kPer == 2)
                            *reinterpret_cast<uint16_t*>(dst) = uint16_t(codes[0]);
                        else if constexpr (kPer == 4)
                            *reinterpret_cast<uint32_t*>(dst) = codes[0];
                        else
                            *reinterpret_cast<uint2*>(dst) = make_uint2(codes[0], codes[1]);
                    }
                }
                if (lane < 8) {
                    rowc[qb * R + r0 + lane] = mine_c;
                    rowat[qb * R + r0 + lane] = mine;
                    rownode[qb * R + r0 + lane] = s.node0 + a.by_hpt.div(r0 + lane);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::kQFull + qb));
        }
    } else {
        // ================================================================ softmax: a thread owns a token of every tile
        const int quad = wid & 3, tok = 32 * quad + lane;
        const uint32_t lanes = uint32_t(32 * quad) << 16;
        const uint32_t ts0 = tmem + lanes, to = tmem + lanes + C::kOCol;
        float* wc = reinterpret_cast<float*>(ctl + C::kWarpOff) + quad * 4 * R;  // c of this warp's rows
        float* wm = wc + R;                                                      // kShift - m
        float* wf = wm + R;                                                      // a factor
        float* wd = wf + R;                                                      // what wm rose by
        // Exchanged maxima and, apart from them, sums: a segment's first maxima are written while a slow warp may still be
        // reading the sums of the segment before.
        float* red = reinterpret_cast<float*>(ctl + C::kRedOff);
        float* sums = red + 4 * R;
        volatile int* votes = reinterpret_cast<volatile int*>(ctl + C::kVoteOff);
        int exchanges = 0;
        // All four warps of the line have come here, with what their lanes wrote.
        auto exchange = [&]() -> bool {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::kVote));
            const bool got = wait(C::kVote, uint32_t(exchanges) & 1u);
            ++exchanges;
            return got;
        };
        int jobs = 0;
        Ring<C::kScales> sc;
        Ring<C::kSlots> ring;  // of the loads; V of a tile is the second
        bool ok = true;
        const bool packed = a.packed != 0;
        for (int seg = 0; ok; ++seg) {
            if (!seg_wait(seg)) break;
            const TcSeg& s = seg_at(seg);
            const int blk0 = s.blk0, blk1 = s.blk1, tail0 = s.tail0;
            if (blk0 == blk1) break;
            const TreeReq r = s.req();
            const int qb = q_buf(seg), cols = min(R, s.nodes * a.hpt);  // rows
            if (!(ok = wait(C::kQFull + qb, q_phase(seg)))) break;
            __syncwarp();
            if (lane < R) {
                wc[lane] = lane < ((cols + 7) & ~7) ? rowc[qb * R + lane] : 0.f;
                wm[lane] = 0.f;
            }
            __syncwarp();
            float m = kNegInf;  // lane: the running maximum of row `lane`
            unsigned unset = 0u;  // rows that have none yet: they attended no token of the tiles so far
            float l[R];
#pragma unroll
            for (int c = 0; c < R; ++c) l[c] = 0.f;
            for (int blk = blk0; blk < blk1; ++blk, ++jobs, sc.next(), ring.next(), ring.next()) {
                const int buf = jobs & 1, pbuf = jobs % C::kPBufs;
                if (!(ok = wait(C::kSFull + buf, uint32_t(jobs >> 1) & 1u))) break;
                tc_fence_after();
                float x[R], part[16], last[16];
                auto load_parts = [&](int c) {
                    const uint32_t at = ts0 + buf * C::kQRows + c;
                    tmem_ld16(at, *reinterpret_cast<uint32_t(*)[16]>(x + c));
                    tmem_ld16(at + R, *reinterpret_cast<uint32_t(*)[16]>(part));
                    if (kParts > 2) tmem_ld16(at + 2 * R, *reinterpret_cast<uint32_t(*)[16]>(last));
                };
                load_parts(0);
                if (quad == 0 && lane == 0) mbar_arrive(bar(C::kEmpty + ring.slot));  // S is there: K has been read
                if (!(ok = wait(C::kScFull + sc.slot, sc.phase))) break;
                const float* sk = scales + sc.slot * 2 * C::kKeys;
                const int sat = a.run > 1 ? tok >> 2 : tok;
                const float ks = sk[sat], vs = sk[C::kKeys + sat];
                const float lv = log2f(fmaxf(vs, kLeastV));  // (smaller scales count so for the maximum)
                const unsigned bad_pages = bad_slots[jobs % C::kBadRing];
                // the sums of the parts, the smallest first
#pragma unroll
                for (int c = 0; c < R; c += 16) {
                    if (c >= cols) break;
                    if (c > 0) load_parts(c);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float2 by = make_float2(0.0625f, 0.0625f);
                        float2 y = make_float2(part[e], part[e + 1]);
                        if (kParts > 2) y = __ffma2_rn(make_float2(last[e], last[e + 1]), by, y);
                        y = __ffma2_rn(y, by, make_float2(x[c + e], x[c + e + 1]));
                        x[c + e] = y.x;
                        x[c + e + 1] = y.y;
                    }
                }
                const bool fresh = blk == blk0;
                const bool guard = !packed || bad_pages != 0u || blk >= tail0;
                unsigned allow = ~0u;  // rows that attend the token
                if (guard) {
                    const int t = (bad_pages >> (tok >> a.slot_shift)) & 1u ? -1 : tree_token(a, blk, tok), ctx = r.ctx(), i = t - ctx;
                    allow = t < 0 || t >= r.len ? 0u : ~0u;
                    if (allow != 0u && i >= 0) {
#pragma unroll 4
                        for (int c = 0; c < cols; ++c) {
                            const int node = min(rownode[qb * R + c], r.n - 1);
                            bool sees;
                            if (a.mask == nullptr)
                                sees = i <= node;
                            else
                                sees = i / 32 < a.mask_words && ((__ldg(a.mask + size_t(r.start + node) * a.mask_words + i / 32) >> (i % 32)) & 1u) != 0u;
                            if (!sees) allow &= ~(1u << c);
                        }
                    }
                    if ((t < 0 || t >= ctx)) {
                        // V of a token that some row does not attend: a weight of zero does not undo NaN
                        uint8_t* vrow = smem + C::kRingOff + (ring.slot + 1 == C::kSlots ? 0 : ring.slot + 1) * C::kSlotBytes + tok * C::kRowBytes;
                        const uint32_t vphase = ring.phase ^ (ring.slot + 1 == C::kSlots ? 1u : 0u);
                        const bool dead = t < 0 || t >= r.len;
                        const bool landed = tree_wait(bar(C::kFull + (ring.slot + 1 == C::kSlots ? 0 : ring.slot + 1)), vphase, abort_flag, a.flags);
                        bool found = false;
                        for (int x0 = 0; landed && x0 < D / 16; ++x0) {
                            // (lanes in turn from another 16 bytes on: all banks)
                            constexpr int kIn = C::kRowBytes / 16;
                            const int in = (x0 + lane) % kIn;
                            uint4* at = reinterpret_cast<uint4*>(vrow + x0 / kIn * (C::kKeys * C::kRowBytes) + in * 16);
                            uint4 w = *at;
                            uint4 n = make_uint4(~0u, ~0u, ~0u, ~0u);
                            if (!dead)
                                n = make_uint4(__vcmpeq4(w.x & 0x7f7f7f7fu, 0x7f7f7f7fu), __vcmpeq4(w.y & 0x7f7f7f7fu, 0x7f7f7f7fu),
                                               __vcmpeq4(w.z & 0x7f7f7f7fu, 0x7f7f7f7fu), __vcmpeq4(w.w & 0x7f7f7f7fu, 0x7f7f7f7fu));
                            if ((n.x | n.y | n.z | n.w) != 0u) {
                                found |= !dead;
                                *at = make_uint4(w.x & ~n.x, w.y & ~n.y, w.z & ~n.z, w.w & ~n.w);
                            }
                        }
                        if (found) tag[seg & 1] = seg + 1;
                    }
                    __syncwarp();
                }
                // ---- exponents against the running maximum (the scores themselves in a segment's first tile); minus
                // infinity where a row does not attend the token
                float top = kNegInf;
                const float2 ks2 = make_float2(ks, ks);
#pragma unroll
                for (int c = 0; c < R; c += 4) {
                    if (c % 8 == 0 && c >= cols) break;
                    const float4 cc = *reinterpret_cast<const float4*>(wc + c), mm = *reinterpret_cast<const float4*>(wm + c);
                    float2 y = __fmul2_rn(make_float2(x[c], x[c + 1]), ks2), z = __fmul2_rn(make_float2(x[c + 2], x[c + 3]), ks2);
                    y = __ffma2_rn(y, make_float2(cc.x, cc.y), make_float2(mm.x, mm.y));
                    z = __ffma2_rn(z, make_float2(cc.z, cc.w), make_float2(mm.z, mm.w));
                    x[c] = y.x, x[c + 1] = y.y, x[c + 2] = z.x, x[c + 3] = z.y;
                    if (guard) {
#pragma unroll
                        for (int e = c; e < c + 4; ++e)
                            if (((allow >> e) & 1u) == 0u) x[e] = kNegInf;
                    }
                    top = fmaxf(fmaxf(top, fmaxf(x[c], x[c + 1])), fmaxf(x[c + 2], x[c + 3]));
                }
                // ---- does a weight pass its limit?
                bool over = fresh;
                if (!over) {
                    const int id = exchanges + 1;
                    bool passed = top + lv > kShift + kRise;
                    if (unset != 0u) {
#pragma unroll
                        for (int c = 0; c < R; ++c) passed |= ((unset >> c) & 1u) != 0u && x[c] > kNegInf;
                    }
                    if (__any_sync(kFull, passed) && lane == 0) votes[(id - 1) & 1] = id;
                    if (!(ok = exchange())) break;
                    over = votes[(id - 1) & 1] == id;
                }
                if (over) {
                    float mine = kNegInf;
#pragma unroll
                    for (int c = 0; c < R; ++c) {
                        if (c >= cols) break;
                        const float t = redux_max(isnan(x[c]) ? kNegInf : x[c] + lv);
                        if (lane == c) mine = t;
                    }
                    const float was = lane < R ? wm[lane] : 0.f;
                    if (lane < R) red[quad * R + lane] = mine - was;
                    if (!(ok = exchange())) break;
                    if (lane < R) {
                        const float best = fmaxf(fmaxf(red[lane], red[R + lane]), fmaxf(red[2 * R + lane], red[3 * R + lane]));
                        const float to_m = fmaxf(m, best), now = to_m == kNegInf ? kShift : kShift - to_m;
                        wf[lane] = m == kNegInf ? 1.f : ex2(m - to_m);
                        wd[lane] = now - was;
                        wm[lane] = now;
                        m = to_m;
                    }
                    unset = __ballot_sync(kFull, lane < cols && m == kNegInf);
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < R; ++c) x[c] += wd[c];
                    if (!fresh) {
                        // O holds every tile before this one once the last P V is done
                        if (!(ok = wait(C::kPvDone + (jobs - 1) % C::kPBufs, uint32_t((jobs - 1) / C::kPBufs) & 1u))) break;
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < R; ++c) l[c] *= wf[c];
#pragma unroll 1
                        for (int cb = 0; cb < kPParts * C::kColBlocks; ++cb)  // each part's O of each column block
#pragma unroll
                            for (int c = 0; c < R; c += 16) {
                                uint32_t o[16];
                                tmem_ld16(to + cb * R + c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * wf[c + e]);
                                tmem_st16(to + cb * R + c, o);
                            }
                        tmem_wait_st();
                    }
                }
                // ---- weights and their parts, each 8 times what the one before leaves
                if (jobs >= C::kPBufs && !(ok = wait(C::kPvDone + pbuf, uint32_t((jobs - C::kPBufs) / C::kPBufs) & 1u))) break;
                uint8_t* pp = smem + C::kPOff + pbuf * C::kPBytes + tok * 16;
                const float2 vs2 = make_float2(vs, vs);
                auto weights = [&](auto guarded) {
#pragma unroll
                    for (int c = 0; c < R; c += 8) {
                        if (c >= cols) break;
                        uint32_t parts[kPParts][4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 y = make_float2(ex2(x[c + 2 * e]), ex2(x[c + 2 * e + 1]));
                            float2 w = __fmul2_rn(y, vs2);
                            if constexpr (decltype(guarded)::value) {  // (a scale that is not a number)
                                if (((allow >> (c + 2 * e)) & 1u) == 0u) w.x = 0.f;
                                if (((allow >> (c + 2 * e + 1)) & 1u) == 0u) w.y = 0.f;
                            }
                            float2 sum = __fadd2_rn(make_float2(l[c + 2 * e], l[c + 2 * e + 1]), y);
                            l[c + 2 * e] = sum.x;
                            l[c + 2 * e + 1] = sum.y;
                            __half2 left = __floats2half2_rn(w.x, w.y);
#pragma unroll
                            for (int p = 0; p < kPParts; ++p) {
                                parts[p][e] = half2_e5m2(left);
                                left = __hmul2(__hsub2(left, e5m2_half2(parts[p][e])), __float2half2_rn(8.f));
                            }
                        }
                        uint8_t* at = pp + c / 16 * 2048 + c % 16;
#pragma unroll
                        for (int p = 0; p < kPParts; ++p)
                            *reinterpret_cast<uint2*>(at + p * C::kPPart) =
                                make_uint2(__byte_perm(parts[p][0], parts[p][1], 0x5410), __byte_perm(parts[p][2], parts[p][3], 0x5410));
                    }
                };
                if (guard)
                    weights(std::true_type{});
                else
                    weights(std::false_type{});
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::kPFull + pbuf));
            }
            if (!ok) break;
            // ---- the segment's end
            if (!(ok = wait(C::kPvDone + (jobs - 1) % C::kPBufs, uint32_t((jobs - 1) / C::kPBufs) & 1u))) break;
            tc_fence_after();
            // sums of the rows over the four warps, in their order
            ReduceScatter<R, 16>::run(l, lane);
            sums[quad * R + ReduceScatter<R, 16>::index(0, lane)] = l[0];
            if (!(ok = exchange())) break;
            if (lane < R) {
                const float sum = (sums[lane] + sums[R + lane]) + (sums[2 * R + lane] + sums[3 * R + lane]);
                wf[lane] = sum == 0.f ? 0.f : 1.f / sum;
                // empty by the sum: the maximum passes over scores of NaN, the sum does not
                const float lse2 = sum == 0.f ? kNegInf : (m == kNegInf ? 0.f : m) - kShift + log2f(sum);
                const long long at = lane < cols ? rowat[qb * R + lane] : -1;
                if (quad == 0 && at >= 0) {
                    if (s.slot >= 0)
                        a.part_lse[size_t(s.slot) * a.seg_rows + lane] = tree_part_lse(lse2);
                    else
                        a.lse[at] = lse2 == kNegInf ? kNegInf : lse2 * kLn2;
                }
            }
            __syncwarp();
            const bool fix = tag[seg & 1] == seg + 1;
#pragma unroll 1
            for (int x = 0; x < C::kColBlocks * (R / 16); ++x) {
                const int cb = x / (R / 16), c = x % (R / 16) * 16;
                if (c >= cols) continue;
                uint32_t o[kPParts][16];  // of each part of the weights
                __syncwarp();
#pragma unroll
                for (int p = 0; p < kPParts; ++p) tmem_ld16(to + (cb * kPParts + p) * R + c, o[p]);
                tmem_wait_ld();
                const int dim = cb * 128 + tok;
                if (dim >= D) continue;  // (head_dim 64: the second half of M)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const long long at = c + e < cols ? rowat[qb * R + c + e] : -1;
                    if (at < 0) continue;
                    float f = __uint_as_float(o[kPParts - 1][e]);
#pragma unroll
                    for (int p = kPParts - 2; p >= 0; --p) f = fmaf(f, 0.125f, __uint_as_float(o[p][e]));  // the smallest first
                    f *= wf[c + e];
                    if (fix) {
                        // NaN of node rows in these blocks, for the rows that attend them
                        const int node = rownode[qb * R + c + e];
                        for (int i = 0; i < r.n; ++i) {
                            const int t = r.ctx() + i, b = tree_slot_of(a, t) >> a.spb_shift;
                            if (b < blk0 || b >= blk1) continue;
                            if ((tree_allow(a, r, node, t, 1) & 1u) == 0u) continue;
                            const int page = __ldg(a.indices + r.lo + t / a.page_size);
                            if (page < 0 || page >= a.num_total_pages) continue;
                            const size_t vrow = ((size_t(page) * a.num_kv_heads + s.kvh) * a.page_size + t % a.page_size) * D;
                            if ((static_cast<const uint8_t*>(a.v)[vrow + dim] & 0x7f) == 0x7f) f = __int_as_float(0x7fc00000);
                        }
                    }
                    if (s.slot >= 0)
                        a.part_o[(size_t(s.slot) * a.seg_rows + c + e) * D + dim] = f;
                    else
                        static_cast<T*>(a.o)[at * D + dim] = T(f);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::kQEmpty + qb));
            seg_free(seg);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (!soft && line == 0 && part == 0) tmem_dealloc(*tslot, 512);
}

// ---------------------------------------------------------------- lookup

template <typename T, int D, int R>
TreeKernels blocks_tc_kernels() {
    using C = CfgBlocks<D, R, std::is_same<T, __half>::value ? 3 : 2>;
    TreeKernels k{};
    k.main = reinterpret_cast<const void*>(blocks_tc_kernel<T, D, R>);
    k.merge = reinterpret_cast<const void*>(tree_merge_kernel<T, D>);
    k.threads = C::kThreads;
    k.smem = C::kBytes;
    k.per_sm = 1;
    k.tile_rows = R;
    k.tiles = 1;
    k.workers = C::kLines;
    k.block_tokens = C::kKeys;
    k.seg_cost = C::kSegCost;
    k.tensor = k.codes = true;
    return k;
}

template <typename T, int R>
bool blocks_tc_lookup(int D, TreeKernels* k) {
    switch (D) {
        case 64: *k = blocks_tc_kernels<T, 64, R>(); return true;
        case 128: *k = blocks_tc_kernels<T, 128, R>(); return true;
    }
    if constexpr (R == 16) {
        if (D == 256) {
            *k = blocks_tc_kernels<T, 256, R>();
            return true;
        }
    }
    return false;
}

}  // namespace pd
