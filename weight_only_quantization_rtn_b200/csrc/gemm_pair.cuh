// Tensor-core kernels that share one staged operand between two dequantized tiles:
// the gated feed-forward block's two projections, and the gradient of a quantized
// linear layer (or of the block) with respect to its input.
//
//   GATED   G = X·Ŵgᵀ, U = X·Ŵuᵀ (reduction over K); H = act(G) ⊙ U in the epilogue
//   DGRAD   dX = Σ_p dY_p·Ŵ_p   (reduction over N; p = 1 for a linear layer, 2 for the
//           gated block, whose two products are one sum: dG·Ŵg + dU·Ŵu)
//
// As in gemm_tc_kernel the dequantized weights are the A operand (128 rows of the
// accumulator per CTA) and the tokens are B.  Each CTA holds two accumulators in tensor
// memory, fed by two A tiles and one token tile: gate and up rows of the same 128
// features, or two blocks of 128 input channels of the same weight rows.  So a token
// tile that was loaded once is multiplied twice, and shared memory, whose bandwidth a
// 128 x 256 tile with one accumulator uses up (loads, dequantized stores and operand
// reads together), has room left.
//
// PAIR (more than 96 tokens): two CTAs of a cluster compute one tile together
// (cta_group::2): each holds its own 128 rows of both A tiles and half of the tokens, one
// thread of the even CTA issues the MMAs (M = 256) for both, and each SM reads half of
// the B operand.  The token tile is the batch divided evenly (at most 256 tokens), in
// steps of 16, not a power of two: 333 tokens are two tiles of 176.
//
// DGRAD needs Ŵ with the reduction along its rows.  The codes stay as they are stored:
// a block is 64 weight rows x 256 input channels, dequantized into the "MN-major" layout
// (64 channels contiguous per 128-byte swizzled line, lines along the rows), which the
// tensor core reads as the transposed A operand; nothing is transposed in memory.
//
// Warps: 0 loads tokens (TMA, 128-byte swizzle), 2 loads codes (TMA), 1 issues the MMAs
// and owns the tensor memory, 3 brings scales and zero points (GATED), 4 and up dequantize and
// run the epilogue (8, 12 or 16 warps: 168, 128 or 96 registers).  Three rings of
// shared memory, because the three have different sizes and lead times: token blocks,
// code units (GATED with 4 bits: 128 input channels, so that a row is 64 bytes; loaded as
// 32-byte rows the TMA engine's row rate, not bandwidth, paced the kernel) and dequantized
// A tiles.  Scales and zero points of GATED have a small ring of their own, four groups
// a slot; DGRAD's go from global memory to registers two blocks ahead.  Both read rows of any
// number of groups and any alignment.
//
// The kernel is persistent, one CTA (or pair) per SM (or two).  Either whole tiles are
// dealt in turn, or (when that would leave CTAs idle for longer than it costs) all tiles'
// code units, in order, are divided evenly over the CTAs.  Then a tile may belong to
// several CTAs: each owner but the first leaves its binary32 part in the workspace, with a
// ready flag per warp, and the first owner adds the parts in order and finishes the tile.
// A CTA leaves a part for its first tile only and waits only in its last one, so a part
// has usually been there for a while, nothing waits in a circle, and the epilogues of the
// CTAs are spread over time instead of all writing at once.
//
// Measured on the device (K = 4096, N = 11008, both 4-bit): M = 2048 with G and U kept 265 us =
// 1395 TFLOP/s in a short run and 305 to 317 us in a long one, bound by the tensor cores and then by
// the power limit, its backward pass (with the elementwise half) 265 and 313 us; M = 61 29 us,
// 13 to 16 us of it dequantization (0.35 to 0.44 us per block and SM).
#pragma once

#include "activation.cuh"
#include "common.cuh"

namespace w4a16 {

// ------------------------------------------------------------------ CTA pairs
__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The address of this CTA's shared-memory location `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t mapa_u32(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// mbar_wait for a barrier that the other CTA of the pair arrives on (bounded).
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity) {
    uint64_t t0 = 0;
    for (uint32_t tries = 1;; ++tries) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if ((tries & 63u) == 0u) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0) {
                t0 = now;
            } else if (now - t0 > kWaitTimeoutNs) {
                report_error(kErrMbarTimeout);
                return false;
            }
        }
    }
}

template <bool PAIR>
__device__ __forceinline__ void tmem_alloc_g(uint32_t holder, uint32_t ncols) {
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(holder),
                     "r"(ncols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tmem_alloc(holder, ncols);
        tmem_relinquish();
    }
}

template <bool PAIR>
__device__ __forceinline__ void tmem_dealloc_g(uint32_t taddr, uint32_t ncols) {
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                     : "memory");
    else
        tmem_dealloc(taddr, ncols);
}

template <bool PAIR>
__device__ __forceinline__ void tc_mma_bf16_g(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                              uint32_t idesc, uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        tc_mma_bf16(tmem_d, adesc, bdesc, idesc, accumulate);
}

// D += A·B with A (128 rows x 16 of the reduction, 8 columns) in tensor memory.
__device__ __forceinline__ void tc_mma_bf16_ta(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
        "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// This thread's 32 columns of its lane of tensor memory.
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]), "r"(r[1]),
        "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
        "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}

// Arrive on the barrier at `bar` (PAIR: on the same barrier of both CTAs) once all MMAs
// issued so far have completed.
template <bool PAIR>
__device__ __forceinline__ void tc_commit_g(uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
            "[%0], %1;" ::"r"(bar),
            "h"((uint16_t)3)
            : "memory");
    else
        tc_commit(bar);
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0u;
}

// Shared-memory descriptor of an MN-major operand in the 128-byte swizzle layout: lines
// of 64 contiguous bf16 along M (or N), one line per step of K; groups of 8 lines are
// 1024 bytes apart, the next 64 along M (or N) lie `block_bytes` further.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr, uint32_t block_bytes) {
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)((block_bytes >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

constexpr uint32_t kIdescAMnMajor = 1u << 15;
constexpr uint32_t kIdescBMnMajor = 1u << 16;

// ------------------------------------------------------------------ configuration
constexpr int kPairCodeWarp = 2;
constexpr int kPairScaleWarp = 3;       // GATED
constexpr int kPairBlock = 64;          // reduction per block
constexpr int kPairRows = 128;          // rows of one A tile per CTA
constexpr int kPairABytes = 2 * kPairRows * kPairBlock * 2;   // both A tiles of a block: 32 KB
constexpr int kPairQuadBytes = 2 * 2 * kPairRows * 8;        // four groups' [scale, zero][matrix][row]: 4 KB
constexpr int kPairMaxQuads = 4;
constexpr int kPairMaxX = 8;
constexpr int kPairMaxWarps = 16;       // dequantizing warps, at most

// A pair's MMAs take longer than two groups of dequantizing warps need for a block; a single
// CTA's small tiles do not, so its 4-bit gradient has a third group (M = 77, K = 37888,
// N = 8192: 157 us with two groups, 133 us with three); three gained nothing with 8-bit codes.
// With kTmemA a group costs no A buffer and 96 registers do, so there are four (M = 61,
// K = 8192, N = 18944: 66.6 us with two, 60.7 with three, 56.1 with four).
//
// kTmemA: a single CTA's GATED tiles leave tensor memory free, and what paced them with the A
// tiles in shared memory was its bandwidth (0.57 us per block at any token count, 0.39 us
// without the stores).  So there the dequantized weights go to tensor memory (a lane is a
// weight row, K-major as the MMA reads A from there) and never touch shared memory, which
// holds deep rings of loads instead.  DGRAD cannot: its A is the transpose of what a thread has.
constexpr int kPairMaxA = 6;
template <bool PAIR, int BITS, bool DGRAD>
struct PairConfig {
    static constexpr bool kPair = PAIR;
    static constexpr bool kTmemA = !PAIR && !DGRAD;
    static constexpr int kGroups = kTmemA ? 4 : (!PAIR && DGRAD && BITS == 4 ? 3 : 2);
    static constexpr int kWarps = 4 * kGroups;                 // warps 4 .. 4 + kWarps - 1
    static constexpr int kThreads = (4 + kWarps) * 32;
    static constexpr int kSmemA = kTmemA ? 0 : (kGroups + 1) * kPairABytes;   // A ring
    static constexpr int kStage = kWarps * 1024;               // epilogue staging, 1 KB per warp
    static constexpr int kQuads = DGRAD ? 0 : (kTmemA ? 4 : 2);  // ring of scales, four groups a slot
    static constexpr int kLoads = kTmemA ? 225 * 1024 - kStage - kQuads * kPairQuadBytes
                                         : (kGroups == 2 ? 112 * 1024 : 84 * 1024);
    static constexpr int kSmem = kSmemA + kStage + kQuads * kPairQuadBytes + kLoads + 1024 + 1024;
    static_assert(kSmem <= 232448, "shared memory");
    // 64-wide blocks per code unit, and its bytes: two boxes (gate, up) of 128 rows, of 128 bytes
    // with kTmemA and 64 bytes in a pair's tighter ring; DGRAD: 64 rows x 256 channels.
    static constexpr int kUnitBlocks = DGRAD ? 1 : (kTmemA ? 2 : 1) * 8 / BITS;
    static constexpr int kUnitBytes = 2 * kPairRows * kPairBlock * BITS / 8 * kUnitBlocks;
};

// Most tokens of a tile of one CTA: its token ring must hold a block for each A buffer.
constexpr int kPairMaxSingle = 96;

// A slots, code units and token blocks that the rings hold.
//
// A barrier's wait tells two successive phases apart, no more: a warp that awaits a slot's
// next phase has to know that the phase before it has completed.  Blocks are numbered
// through all segments of a CTA's share, group k dequantizes the blocks ≡ k modulo the number
// of groups (pair_first), and a group waits for the A slot of its block first.
//   A slot of block j, freed by the MMAs of block j − NA: those of block j − 2·NA are complete,
//     because the group's last block, at most NA before this one, waited for no older ones.
//   Code unit and tokens of block j: what their slots held before was loaded, because all
//     blocks up to j − NA are multiplied and the rings cover at least NA blocks
//     (a unit that ends a tile may hold as little as one block: `cover` below).
struct PairRings {
    int na, sp, sx;
};

// Fewest blocks that `units` consecutive code units of `per_unit` blocks hold, when a tile has
// `blocks` (units do not cross tiles, so a tile's last may be short).
__host__ __device__ inline int pair_cover(int units, int per_unit, int blocks) {
    return blocks <= per_unit ? units * blocks : units / 2 * (per_unit + 1) + units % 2;
}

// First block of group `grp` in a segment, counted from the segment's first, which `before`
// blocks of the share precede.
__host__ __device__ inline int pair_first(int before, int grp, int groups) {
    const int d = grp - before % groups;
    return d < 0 ? d + groups : d;
}

template <typename Cfg>
__host__ __device__ inline PairRings pair_rings(int bt, int acc_cols, int blocks) {
    const int x_bytes = bt * kPairBlock * 2;
    PairRings r;
    if (Cfg::kTmemA) {
        r.na = (512 - 2 * acc_cols) / 64;
        if (r.na > kPairMaxA) r.na = kPairMaxA;
        r.sx = (Cfg::kLoads - 4 * Cfg::kUnitBytes) / x_bytes;
        if (r.sx > kPairMaxX) r.sx = kPairMaxX;
        r.sp = (Cfg::kLoads - r.sx * x_bytes) / Cfg::kUnitBytes;
        const int cover = pair_cover(r.sp, Cfg::kUnitBlocks, blocks);
        if (r.na > cover) r.na = cover;              // (tiles of a single block)
    } else {
        r.na = Cfg::kGroups + 1;
        // tokens come from L2 and need less of a lead than codes do
        r.sx = Cfg::kPair ? r.na + 1 : r.na;
        r.sp = (Cfg::kLoads - r.sx * x_bytes) / Cfg::kUnitBytes;
        if (r.sp > kPairMaxX) r.sp = kPairMaxX;
        r.sx = (Cfg::kLoads - r.sp * Cfg::kUnitBytes) / x_bytes;
        if (r.sx > kPairMaxX) r.sx = kPairMaxX;
    }
    if (r.sp > kPairMaxX) r.sp = kPairMaxX;
    return r;
}

struct PairArgs {
    const uint16_t* scales[2];   // GATED: gate, up; DGRAD: one per product
    const uint16_t* zeros[2];
    uint16_t* out;               // GATED: H [M, N]; DGRAD: dX [M, K]
    uint16_t* G;                 // GATED: kept outputs, or null
    uint16_t* U;
    float* partials;             // split: [slots][CTAs of a slot] binary32 parts
    int M, N, K;
    int gshift;                  // log2 g; 31 for per-channel (one group per row)
    int groups;                  // groups per row
    uint32_t flip;               // symmetric codes: 0x88888888 or 0x80808080, else 0
    int act;
    int products;                // DGRAD: 1 or 2
    int bt;                      // tokens of a CTA's tile (PAIR: half of the tile's)
    int acc_cols;                // tensor-memory columns of one accumulator (power of two)
    int blocks;                  // reduction blocks of a tile
    int tiles_m;
    int tiles;
    int split;                   // 1: the tiles' code units are divided evenly over the CTAs
    uint64_t* flags;             // [slots][CTAs of a slot][kPairMaxWarps] ready flags of the parts
    uint64_t ready;              // the flags' value in this launch
};

// Ready flag of a part: the launch's own 64-bit value (launch_flag), which neither data nor a
// flag that an earlier launch left behind holds, so the workspace needs no clearing before its
// first use.  The first owner clears a flag that it consumed: a captured launch, which keeps its
// value, finds its flags clear.

// A CTA's (pair's) share of the work, as segments (tile, first unit, units).  The host
// refuses problems of 2^31 units and more.
template <int UB>
struct PairWalk {
    int tile, u0, units;
    int at, end;                 // split: this share's units still to do
    __host__ __device__ __forceinline__ static int upt(const PairArgs& a) { return (a.blocks + UB - 1) / UB; }
    // First unit of a slot's share.
    __host__ __device__ __forceinline__ static int start(const PairArgs& a, int c, int slots) {
        return (int)((int64_t)a.tiles * upt(a) * c / slots);
    }
    __host__ __device__ __forceinline__ void init(const PairArgs& a, int slot, int slots) {
        tile = slot - slots;
        at = a.split ? start(a, slot, slots) : 0;
        end = a.split ? start(a, slot + 1, slots) : 0;
    }
    __host__ __device__ __forceinline__ bool next(const PairArgs& a, int slots) {
        const int per = upt(a);
        if (!a.split) {
            tile += slots;
            u0 = 0;
            units = per;
            return tile < a.tiles;
        }
        if (at >= end) return false;
        tile = at / per;
        u0 = at - tile * per;
        units = end - at < per - u0 ? end - at : per - u0;
        at += units;
        return true;
    }
    __host__ __device__ __forceinline__ int first_block() const { return u0 * UB; }
    __host__ __device__ __forceinline__ int count(const PairArgs& a) const {
        return ((u0 + units) * UB < a.blocks ? (u0 + units) * UB : a.blocks) - u0 * UB;
    }
    // Slots [slot + 1, followers_end) hold the rest of the tile that this share begins.
    __host__ __device__ __forceinline__ int followers_end(const PairArgs& a, int slot, int slots) const {
        const int per = upt(a);
        int c = slot + 1;
        if (u0 == 0 && units < per)
            while (c < slots && start(a, c, slots) < (tile + 1) * per) ++c;
        return c;
    }
};

// Wait for another CTA's part (bounded: about one second).
__device__ __forceinline__ bool pair_wait_flag(const uint64_t* flag, uint64_t ready) {
    uint64_t t0 = 0;
    for (uint32_t tries = 1;; ++tries) {
        if (ld_acquire_u64(flag) == ready) return true;
        __nanosleep(100);
        if ((tries & 63u) == 0u) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0) {
                t0 = now;
            } else if (now - t0 > kWaitTimeoutNs) {
                report_error(kErrMbarTimeout);
                return false;
            }
        }
    }
}

// A scale and zero point as the dequantization wants them, from bf16 pairs (s, s), (z, z):
// s·2^6 and −z·2^-6 (see below; exact while s < 2^122).  Symmetric codes are flipped to
// offset form and take z = 8 or 128.  `worst` keeps the largest s·2^6: where it is no finite number,
// s·2^6 does not exist, the results are none either and the kernel says so.  (A second form of the
// conversion for such blocks, s and 2^6 multiplied one after the other, gave the right numbers and
// cost every short batch 2 to 6%: dX, M = 77, 8192 x 8192 28.9 us instead of 27.5.)
__device__ __forceinline__ uint32_t pair_scale(uint32_t ss, uint32_t& worst) {
    const uint32_t scaled = bf16x2_mul(ss, 0x42804280u);
    worst = max(worst, scaled & 0x7FFFFFFFu);
    return scaled;
}
constexpr uint32_t kPairNoScale = 0x7F800000u;      // an infinity or no number in the upper half

template <int BITS>
__device__ __forceinline__ uint32_t pair_zero(uint32_t zz, bool sym) {
    constexpr uint32_t kSym = BITS == 4 ? 0xBE00BE00u : 0xC000C000u;             // −8·2^-6, −128·2^-6
    return sym ? kSym : bf16x2_mul(zz, 0xBC80BC80u);
}

// Eight codes -> four bf16 pairs in natural order.
// A code q of 4 or 8 bits alone in a 16-bit half is, as bf16, q·2^-133 exactly (subnormal, or
// in the first normal binade, which continues the same steps).  One fma with 2^127 and
// −z·2^-6 gives (q − z)·2^-6 exactly (an integer of at most 8 bits), one multiplication by
// s·2^6 rounds (q − z)·s once.  PRMT brings the codes into the halves: 4 bits (w0) from
// the two nibbles of each byte, masked where they are (the upper one is 16·q and takes 2^123),
// 8 bits (w0, w1) from the bytes themselves.  14 instructions; with the exponent set by a
// LOP3 and a subtraction 17 for 4 bits, and with 8-bit codes formed in binary32 30.
template <int BITS>
__device__ __forceinline__ void pair_dequant8(uint32_t w0, uint32_t w1, uint32_t flip, uint32_t zz,
                                              uint32_t ss, uint32_t out[4]) {
    uint32_t lo, hi;
    if constexpr (BITS == 4) {
        lo = (w0 ^ flip) & 0x0F0F0F0Fu;
        hi = (w0 ^ flip) & 0xF0F0F0F0u;          // 16·q, as bf16 16·q·2^-133
    } else {
        lo = w0 ^ flip;
        hi = w1 ^ flip;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t q;
        if constexpr (BITS == 4) {
            // bytes [lo.j, 0, hi.j, 0]: selector 8 | x replicates byte x's sign bit (of a byte of
            // lo: zero), which the PTX instruction does and __byte_perm does not
            const uint32_t sel = (uint32_t)j | 0x80u | ((uint32_t)(4 + j) << 8) | 0x8000u;
            asm("prmt.b32 %0, %1, %2, %3;" : "=r"(q) : "r"(lo), "r"(hi), "r"(sel));
        } else {
            q = __byte_perm(j < 2 ? lo : hi, 0u, (j & 1) ? 0x4342u : 0x4140u);
        }
        out[j] = bf16x2_mul(bf16x2_fma(q, BITS == 4 ? 0x7D007F00u : 0x7F007F00u, zz), ss);
    }
}

__device__ __forceinline__ void sts128_addr(uint32_t addr, const uint32_t v[4]) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3])
                 : "memory");
}

// The same at a constant offset.
template <int OFF>
__device__ __forceinline__ void sts128_at(uint32_t addr, const uint32_t v[4]) {
    asm volatile("st.shared.v4.u32 [%0 + %5], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "n"(OFF)
                 : "memory");
}

template <int OFF>
__device__ __forceinline__ uint4 lds128_at(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4 + %5];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr), "n"(OFF));
    return v;
}

__device__ __forceinline__ uint4 lds128_addr(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}

// ------------------------------------------------------------------ epilogue
// A strip is 32 rows (a warp's quarter of tensor memory) x 16 tokens.  tcgen05.ld
// 16x256b gives it as MMA fragments (lane t: rows t/4 and t/4 + 8, tokens 2(t%4), + 1), so
// that stmatrix can transpose it: the strip goes through 1 KB of shared memory as 16
// token rows of 32 contiguous outputs and leaves in 16-byte stores.  Storing a
// lane's row directly took 32 two-byte stores per lane and output instead of 2.
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, uint32_t r[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r0),
                 "r"(r1), "r"(r2), "r"(r3)
                 : "memory");
}

// Rounds a strip to bf16 and writes it to out[m0 .. m0+15][c0 .. c0+31] (rows of `ld`
// elements, `cols` of them valid, M rows).  v[8h + i]: register i of row half h.
__device__ __forceinline__ void strip_store(const float v[16], uint32_t stage, uint16_t* __restrict__ out, int m0, int M,
                                            int c0, int cols, int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        // matrices: (rows 0-7, tokens 0-7), (rows 8-15, tokens 0-7), then tokens 8-15
        const int token = (lane & 7) + 8 * (lane >> 4);
        const int chunk = 2 * h + ((lane >> 3) & 1);
        stmatrix_x4_trans(stage + (uint32_t)(token * 64 + ((chunk ^ ((token >> 1) & 3)) * 16)),
                          pack_bf16(v[8 * h], v[8 * h + 1]), pack_bf16(v[8 * h + 2], v[8 * h + 3]),
                          pack_bf16(v[8 * h + 4], v[8 * h + 5]), pack_bf16(v[8 * h + 6], v[8 * h + 7]));
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int token = (lane >> 2) + 8 * i, chunk = lane & 3;
        const uint4 d = lds128_addr(stage + (uint32_t)(token * 64 + ((chunk ^ ((token >> 1) & 3)) * 16)));
        const int m = m0 + token, c = c0 + 8 * chunk;
        if (m < M && c < cols) {
            uint16_t* o = out + (int64_t)m * cols + c;
            if ((cols & 7) == 0) {
                *reinterpret_cast<uint4*>(o) = d;
            } else {
                const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c + e < cols) o[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
            }
        }
    }
    __syncwarp();                                   // the staging bytes are free again
}

// Both accumulators' strips of rows row0 + 32·quarter .. + 31.
template <bool DGRAD>
__device__ __forceinline__ void pair_emit(const PairArgs& a, float v0[16], float v1[16], uint32_t stage, int r0, int rank,
                                          int quarter, int m, int lane) {
    if constexpr (DGRAD) {
        const int c = r0 + rank * 2 * kPairRows + 32 * quarter;
        strip_store(v0, stage, a.out, m, a.M, c, a.K, lane);
        strip_store(v1, stage, a.out, m, a.M, c + kPairRows, a.K, lane);
    } else {
        const int c = r0 + rank * kPairRows + 32 * quarter;
        if (a.G != nullptr) {
            strip_store(v0, stage, a.G, m, a.M, c, a.N, lane);
            strip_store(v1, stage, a.U, m, a.M, c, a.N, lane);
        }
        // (the choice of the activation outside the loop)
        switch (a.act) {
            case W4A16_ACT_SILU:
#pragma unroll
                for (int i = 0; i < 16; ++i) v0[i] = act_value(W4A16_ACT_SILU, v0[i]) * v1[i];
                break;
            case W4A16_ACT_GELU:
#pragma unroll
                for (int i = 0; i < 16; ++i) v0[i] = act_value(W4A16_ACT_GELU, v0[i]) * v1[i];
                break;
            case W4A16_ACT_GELU_TANH:
#pragma unroll
                for (int i = 0; i < 16; ++i) v0[i] = act_value(W4A16_ACT_GELU_TANH, v0[i]) * v1[i];
                break;
            default:
#pragma unroll
                for (int i = 0; i < 16; ++i) v0[i] = act_value(W4A16_ACT_RELU, v0[i]) * v1[i];
        }
        strip_store(v0, stage, a.out, m, a.M, c, a.N, lane);
    }
}

// Scale group of half h of the reduction block (GATED).
__device__ __forceinline__ int pair_group(const PairArgs& a, int block, int h) {
    return min((block * kPairBlock + 32 * h) >> a.gshift, a.groups - 1);
}

// First row of a tile (features or input channels) and its first token.
template <bool DGRAD>
__device__ __forceinline__ int pair_row0(const PairArgs& a, int tile, int ctas) {
    return tile / a.tiles_m * (DGRAD ? 2 : 1) * ctas * kPairRows;
}

// Floats of one CTA's part: [strip of 16 tokens][quarter][accumulator][4][lane] float4.
__host__ __device__ inline int64_t pair_part_floats(int tokens) {
    return (int64_t)((tokens + 15) / 16) * 4 * 2 * 16 * 32;
}

// A tile (or a CTA's share of one) whose MMAs have been issued.
struct PairTileDone {
    int r0, m0;
    bool publish;                // leave the sums as a part
    int slot, followers_end;     // parts of slots [slot + 1, followers_end) belong to the tile
    uint32_t accf, phase;        // barrier: accumulators complete
    uint32_t accempty;           // barrier (of the even CTA): accumulators read
    uint32_t tmem, stage;
};

__device__ __forceinline__ void pair_add(float (&f0)[16], float (&f1)[16], const float4 (&p)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f0[4 * e] += p[e].x; f0[4 * e + 1] += p[e].y; f0[4 * e + 2] += p[e].z; f0[4 * e + 3] += p[e].w;
        f1[4 * e] += p[4 + e].x; f1[4 * e + 1] += p[4 + e].y; f1[4 * e + 2] += p[4 + e].z; f1[4 * e + 3] += p[4 + e].w;
    }
}

// The epilogue of one warp: its strips of the accumulators, finished or left as a part.
template <bool PAIR, int GROUPS, bool DGRAD>
__device__ __forceinline__ bool pair_epilogue(const PairArgs& a, const PairTileDone& t, int rank, int w) {
    constexpr int kCtas = PAIR ? 2 : 1, kGroups = GROUPS;
    const int lane = threadIdx.x & 31;
    const int mma_n = kCtas * a.bt;
    bool ok = mbar_wait_cluster(t.accf, t.phase);
    if (!ok) return false;
    tc_fence_after();
    const int quarter = w & 3;                         // the lanes this warp may read
    const int strips = (min(mma_n, a.M - t.m0) + 15) / 16;
    const uint32_t t_lane = t.tmem + ((uint32_t)(quarter * 32) << 16);
    const int64_t part_floats = pair_part_floats(mma_n);
    for (int c = t.slot + 1; c < t.followers_end && ok; ++c)
        ok = pair_wait_flag(a.flags + ((int64_t)c * kCtas + rank) * kPairMaxWarps + w, a.ready);
    if (!__all_sync(0xffffffffu, ok ? 1 : 0)) return false;
    // strips of this warp: the quarter's strips are dealt over its warps
#pragma unroll 1
    for (int sidx = w >> 2; sidx < strips; sidx += kGroups) {
        uint32_t v0[16], v1[16];
        const uint32_t t0 = t_lane + 16 * sidx;
        tmem_ld_16x256b_x2(t0, v0);
        tmem_ld_16x256b_x2(t0 + (16u << 16), v0 + 8);
        tmem_ld_16x256b_x2(t0 + a.acc_cols, v1);
        tmem_ld_16x256b_x2(t0 + a.acc_cols + (16u << 16), v1 + 8);
        tmem_wait_ld();
        if (sidx + kGroups >= strips) {
            // the last of them is in registers: the next tile may have the accumulators
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) mbar_arrive_cluster(t.accempty);
                else mbar_arrive(t.accempty);
            }
        }
        float f0[16], f1[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            f0[e] = __uint_as_float(v0[e]);
            f1[e] = __uint_as_float(v1[e]);
        }
        // place of the strip in a CTA's part: 8 float4 per lane, lanes side by side
        const int64_t in_part = (int64_t)(sidx * 4 + quarter) * (2 * 16 * 32);
        if (t.publish) {
            float4* part =
                reinterpret_cast<float4*>(a.partials + ((int64_t)t.slot * kCtas + rank) * part_floats + in_part);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                part[e * 32 + lane] = make_float4(f0[4 * e], f0[4 * e + 1], f0[4 * e + 2], f0[4 * e + 3]);
                part[(4 + e) * 32 + lane] = make_float4(f1[4 * e], f1[4 * e + 1], f1[4 * e + 2], f1[4 * e + 3]);
            }
            continue;
        }
        // the followers' parts in order, two in flight at a time
        const float4* part =
            reinterpret_cast<const float4*>(a.partials + ((int64_t)(t.slot + 1) * kCtas + rank) * part_floats + in_part) + lane;
        const int64_t next_part = kCtas * part_floats / 4;
        int left = t.followers_end - t.slot - 1;
        for (; left > 1; left -= 2, part += 2 * next_part) {
            float4 p[8], q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                p[e] = __ldcg(part + e * 32);
                q[e] = __ldcg(part + next_part + e * 32);
            }
            pair_add(f0, f1, p);
            pair_add(f0, f1, q);
        }
        if (left > 0) {
            float4 p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = __ldcg(part + e * 32);
            pair_add(f0, f1, p);
        }
        pair_emit<DGRAD>(a, f0, f1, t.stage, t.r0, rank, quarter, t.m0 + 16 * sidx, lane);
    }
    if ((w >> 2) >= strips && lane == 0) {             // no strip for this warp
        if constexpr (PAIR) mbar_arrive_cluster(t.accempty);
        else mbar_arrive(t.accempty);
    }
    if (t.publish) {
        __threadfence();                               // every lane's part before the flag
        __syncwarp();
        if (lane == 0)
            st_release_u64(a.flags + ((int64_t)t.slot * kCtas + rank) * kPairMaxWarps + w, a.ready);
    } else if (t.followers_end > t.slot + 1) {
        __syncwarp();
        if (lane == 0)                                 // the parts were read: their flags are free again
            for (int c = t.slot + 1; c < t.followers_end; ++c)
                a.flags[((int64_t)c * kCtas + rank) * kPairMaxWarps + w] = 0ull;
    }
    return true;
}

template <bool PAIR, int BITS, bool DGRAD>
__global__ void __launch_bounds__(PairConfig<PAIR, BITS, DGRAD>::kThreads, 1)
    gemm_pair_kernel(const __grid_constant__ CUtensorMap tmX0, const __grid_constant__ CUtensorMap tmX1,
                     const __grid_constant__ CUtensorMap tmP0, const __grid_constant__ CUtensorMap tmP1,
                     const __grid_constant__ PairArgs a) {
    using Cfg = PairConfig<PAIR, BITS, DGRAD>;
    constexpr int UB = Cfg::kUnitBlocks, NG = Cfg::kGroups;
    constexpr int kCtas = PAIR ? 2 : 1;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const PairRings rings = pair_rings<Cfg>(a.bt, a.acc_cols, a.blocks);
    const int NA = rings.na, SP = rings.sp, SX = rings.sx, x_bytes = a.bt * kPairBlock * 2;
    const uint32_t as = smem_u32(smem);              // NA x kPairABytes (not with kTmemA)
    const uint32_t ps = as + Cfg::kSmemA;            // SP code units
    const uint32_t xs = ps + SP * Cfg::kUnitBytes;   // SX token blocks
    const uint32_t st = ps + Cfg::kLoads;            // epilogue staging
    const uint32_t qs = st + Cfg::kStage;            // kQuads scale slots
    const uint32_t bars = qs + Cfg::kQuads * kPairQuadBytes;
    const uint32_t xfull = bars, xempty = xfull + 8 * kPairMaxX;
    const uint32_t pfull = xempty + 8 * kPairMaxX, pempty = pfull + 8 * kPairMaxX;
    const uint32_t afull = pempty + 8 * kPairMaxX, aempty = afull + 8 * kPairMaxA;
    const uint32_t accf = aempty + 8 * kPairMaxA, accempty = accf + 8;
    const uint32_t qfull = accempty + 8, qempty = qfull + 8 * kPairMaxQuads;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + (qempty + 8 * kPairMaxQuads - as));

    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);   // uniform
    const int lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)cluster_ctarank() : 0;
    // Split: shares are numbered from the last CTA to the first, so that a first owner waits for
    // CTAs of lower index only, which are on the machine before it: however few SMs other
    // work leaves, every wait ends.
    const int slots = (int)gridDim.x / kCtas;
    const int slot = a.split ? slots - 1 - (int)blockIdx.x / kCtas : (int)blockIdx.x / kCtas;
    const int per_product = a.blocks / a.products;
    const int mma_n = kCtas * a.bt;

    if (threadIdx.x == 0) {
        for (int s = 0; s < SX; ++s) {
            mbar_init(xfull + 8 * s, 1);
            mbar_init(xempty + 8 * s, 1);
        }
        for (int s = 0; s < SP; ++s) {
            mbar_init(pfull + 8 * s, 1);
            mbar_init(pempty + 8 * s, 4 * UB);
        }
        for (int s = 0; s < NA; ++s) {
            mbar_init(afull + 8 * s, kCtas * 4);
            mbar_init(aempty + 8 * s, 1);
        }
        for (int s = 0; s < Cfg::kQuads; ++s) {
            mbar_init(qfull + 8 * s, 32);
            mbar_init(qempty + 8 * s, Cfg::kWarps);
        }
        mbar_init(accf, 1);
        mbar_init(accempty, kCtas * Cfg::kWarps);
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmX0);
        if (DGRAD && a.products > 1) prefetch_tensormap(&tmX1);
    }
    if (warp == kPairCodeWarp && lane == 0) {
        prefetch_tensormap(&tmP0);
        if (!DGRAD || a.products > 1) prefetch_tensormap(&tmP1);
    }
    const int tmem_cols = Cfg::kTmemA ? 512 : 2 * a.acc_cols;
    if (warp == 1) tmem_alloc_g<PAIR>(smem_u32(tmem_holder), tmem_cols);
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();      // the pair's barriers are set up before either arrives
    tc_fence_after();
    const uint32_t tmem_d = *tmem_holder;
    const uint32_t tmem_a = tmem_d + (uint32_t)(512 - 64 * NA);      // kTmemA: NA x (gate 32, up 32 columns)
    PairWalk<UB> walk;
    walk.init(a, slot, slots);

    if (warp == 0) {
        // ------------------------------------------------------------ token loads
        if (lane == 0) {
            int s = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            while (ok && walk.next(a, slots)) {
                const int b0 = walk.first_block(), nb = walk.count(a);
                const int m0 = walk.tile % a.tiles_m * mma_n + rank * a.bt;
                for (int i = 0; i < nb; ++i) {
                    ok = mbar_wait_backoff(xempty + 8 * s, ph ^ 1u, 128u);
                    if (!ok) break;
                    mbar_arrive_expect_tx(xfull + 8 * s, x_bytes);
                    int b = b0 + i;
                    const CUtensorMap* tx = &tmX0;
                    if (DGRAD && b >= per_product) {
                        b -= per_product;
                        tx = &tmX1;
                    }
                    tma_load_2d(xs + s * x_bytes, tx, b * kPairBlock, m0, xfull + 8 * s);
                    ++issued;
                    if (++s == SX) { s = 0; ph ^= 1u; }
                }
            }
            // Do not leave while copies into this CTA's shared memory are in flight.
            for (int i = (issued > SX ? issued - SX : 0); i < issued; ++i)
                if (!mbar_wait(xfull + 8 * (i % SX), (uint32_t)(i / SX) & 1u)) break;
        }
        __syncwarp();
    } else if (warp == kPairCodeWarp) {
        // ------------------------------------------------------------ code loads
        if (lane == 0) {
            int s = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            while (ok && walk.next(a, slots)) {
                const int r0 = pair_row0<DGRAD>(a, walk.tile, kCtas);
                for (int u = 0; u < walk.units; ++u) {
                    ok = mbar_wait_backoff(pempty + 8 * s, ph ^ 1u, 128u);
                    if (!ok) break;
                    const uint32_t bar = pfull + 8 * s, p = ps + s * Cfg::kUnitBytes;
                    mbar_arrive_expect_tx(bar, Cfg::kUnitBytes);
                    if constexpr (DGRAD) {
                        int b = walk.u0 + u;
                        const CUtensorMap* tp = &tmP0;
                        if (b >= per_product) {
                            b -= per_product;
                            tp = &tmP1;
                        }
                        const int c0 = (r0 + rank * 2 * kPairRows) / (8 / BITS);   // code bytes; boxes of 128
#pragma unroll
                        for (int h = 0; h < BITS / 4; ++h)
                            tma_load_2d(p + h * kPairBlock * 128, tp, c0 + 128 * h, b * kPairBlock, bar);
                    } else {
                        const int k = (walk.u0 + u) * UB * kPairBlock, n = r0 + rank * kPairRows;
                        tma_load_2d(p, &tmP0, k / (8 / BITS), n, bar);
                        tma_load_2d(p + Cfg::kUnitBytes / 2, &tmP1, k / (8 / BITS), n, bar);
                    }
                    ++issued;
                    if (++s == SP) { s = 0; ph ^= 1u; }
                }
            }
            for (int i = (issued > SP ? issued - SP : 0); i < issued; ++i)
                if (!mbar_wait(pfull + 8 * (i % SP), (uint32_t)(i / SP) & 1u)) break;
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issue (even CTA)
        // The whole warp runs the loop and one elected lane issues, so that the descriptors
        // live in uniform registers: formed in one lane's registers, eight MMAs took 1100
        // cycles to issue beside busy dequantizing warps, more than they take to run.
        if (rank == 0) {
            const uint32_t idesc = idesc_bf16_f32(kCtas * kPairRows, mma_n) | (DGRAD ? kIdescAMnMajor : 0u);
            const uint64_t ad0 = DGRAD ? sw128_mnmajor_desc(as, 8192) : sw128_kmajor_desc(as);
            const uint64_t bd0 = sw128_kmajor_desc(xs);
            constexpr uint32_t kStepA = DGRAD ? 2048 / 16 : 32 / 16;     // 16 of the reduction, in 16-byte units
            const uint32_t acc1 = tmem_d + (uint32_t)a.acc_cols;
            int s = 0, ab = 0, seg = 0;
            uint32_t pa = 0;
            bool ok = true;
            while (ok && walk.next(a, slots)) {
                const int nb = walk.count(a);
                // both CTAs' warps have read the previous tile's accumulators
                if (seg > 0) ok = mbar_wait_cluster(accempty, (uint32_t)(seg - 1) & 1u);
                ++seg;
                for (int i = 0; i < nb && ok; ++i) {
                    // (a dequantizing warp of each CTA arrives after the tokens landed there too)
                    ok = mbar_wait_cluster(afull + 8 * ab, pa);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ad = ad0 + (uint32_t)(ab * (kPairABytes / 16));
                    const uint64_t bd = bd0 + (uint32_t)(s * (x_bytes / 16));
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < kPairBlock / 16; ++kk) {
                            const uint32_t acc = (i | kk) != 0 ? 1u : 0u;
                            if constexpr (Cfg::kTmemA) {
                                const uint32_t at = tmem_a + (uint32_t)(64 * ab + 8 * kk);
                                tc_mma_bf16_ta(tmem_d, at, bd + kk * 2, idesc, acc);
                                tc_mma_bf16_ta(acc1, at + 32, bd + kk * 2, idesc, acc);
                            } else {
                                tc_mma_bf16_g<PAIR>(tmem_d, ad + kk * kStepA, bd + kk * 2, idesc, acc);
                                tc_mma_bf16_g<PAIR>(acc1, ad + (kPairABytes / 32 + kk * kStepA), bd + kk * 2, idesc, acc);
                            }
                        }
                        tc_commit_g<PAIR>(xempty + 8 * s);
                        tc_commit_g<PAIR>(aempty + 8 * ab);
                        if (i == nb - 1) tc_commit_g<PAIR>(accf);
                    }
                    __syncwarp();
                    if (++s == SX) s = 0;
                    if (++ab == NA) { ab = 0; pa ^= 1u; }
                }
            }
            if (!ok && elect_one()) tc_commit_g<PAIR>(accf);     // error: no MMA outlives the CTA
        }
        __syncwarp();
    } else if (!DGRAD && warp == kPairScaleWarp) {
        // ------------------------------------------------------------ scales and zeros
        // A slot holds four consecutive groups of the tile's rows; the slots of a segment follow its
        // reduction.  (Fetched by the dequantizing warps into registers ahead of their use,
        // a quarter of their time went to issuing these scattered loads and to the moves
        // that awaited them: M = 61, K = 8192, N = 18944 took 73 us instead of 66.6.)
        if constexpr (!DGRAD) {
            // rows of scales are aligned to 8 or 4 bytes (copied asynchronously), or to 2
            const int align = (a.groups & 3) == 0 ? 8 : ((a.groups & 1) == 0 ? 4 : 2);
            const int arrays = a.flip != 0u ? 1 : 2;
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            while (ok && walk.next(a, slots)) {
                const int b0 = walk.first_block(), last = b0 + walk.count(a) - 1;
                const int q0 = pair_group(a, b0, 0) >> 2, q1 = pair_group(a, last, 1) >> 2;
                const int n0 = pair_row0<DGRAD>(a, walk.tile, kCtas) + rank * kPairRows + lane;
                int64_t row[4];                               // this lane's rows, 32 apart
                // (a row behind the last reads the last row's scales: its results are dropped)
#pragma unroll
                for (int k = 0; k < 4; ++k) row[k] = (int64_t)min(n0 + 32 * k, a.N - 1) * a.groups;
                for (int qd = q0; qd <= q1; ++qd) {
                    if (lane == 0) ok = mbar_wait_backoff(qempty + 8 * s, ph ^ 1u, 128u);
                    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                    if (!ok) break;
                    const uint32_t dst = qs + (uint32_t)(s * kPairQuadBytes + 8 * lane);
                    const bool half = 4 * qd + 2 < a.groups;   // the slot's third group exists
                    for (int t = 0; t < arrays; ++t) {
                        uint32_t v[2][4][4];
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const uint16_t* base = (t == 0 ? a.scales[m] : a.zeros[m]) + 4 * qd;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint16_t* src = base + row[k];
                                const uint32_t d = dst + (uint32_t)(((2 * t + m) * kPairRows + 32 * k) * 8);
                                if (align == 8) {
                                    cp_async_8(d, src, 8u);
                                } else if (align == 4) {
                                    cp_async_4(d, src, 4u);
                                    cp_async_4(d + 4, half ? src + 2 : src, half ? 4u : 0u);
                                } else {
#pragma unroll
                                    for (int e = 0; e < 4; ++e) v[m][k][e] = ldg_u16(src + min(e, a.groups - 1 - 4 * qd));
                                }
                            }
                        }
                        if (align == 2)
#pragma unroll
                            for (int m = 0; m < 2; ++m)
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(
                                                     dst + (uint32_t)(((2 * t + m) * kPairRows + 32 * k) * 8)),
                                                 "r"(v[m][k][0] | v[m][k][1] << 16), "r"(v[m][k][2] | v[m][k][3] << 16)
                                                 : "memory");
                    }
                    if (align > 2) cp_async_arrive_noinc(qfull + 8 * s);
                    else mbar_arrive(qfull + 8 * s);
                    if (++s == Cfg::kQuads) { s = 0; ph ^= 1u; }
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");     // no copy outlives the CTA
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ------------------------------------------------------------ dequantize, epilogue
        // Groups of four warps take the blocks in turn, so that one group's waits, fences and
        // loads hide behind the others' arithmetic and each warp pays its per-block overhead
        // for sixteen chunks of codes.
        const int w = warp - 4, grp = w >> 2, wg = w & 3;
        const bool sym = a.flip != 0u;
        const uint32_t afull_r = PAIR ? mapa_u32(afull, 0) : afull;
        int cnt = 0, ucnt = 0, seg = 0;              // blocks and units of the segments before
        // GATED: scale slots of the segments before, the one at hand (counted through all), its place
        int quads = 0, quad = -1, qslot = -1;
        uint32_t qph = 0, worst = 0;
        bool ok = true;
        // A finished tile's epilogue runs after the next segment's first NA blocks were
        // dequantized, while its own last MMAs complete: the pipeline is full again when the
        // accumulators are free.
        bool pending = false, e_publish = false;
        int e_r0 = 0, e_m0 = 0, e_f1 = 0;

        auto epilogue = [&]() {
            PairTileDone t;
            t.r0 = e_r0;
            t.m0 = e_m0;
            t.publish = e_publish;
            t.slot = slot;
            t.followers_end = e_f1;
            t.accf = accf;
            t.phase = (uint32_t)seg & 1u;
            t.accempty = PAIR ? mapa_u32(accempty, 0) : accempty;
            t.tmem = tmem_d;
            t.stage = st + w * 1024;
            ok = pair_epilogue<PAIR, NG, DGRAD>(a, t, rank, w);
            ++seg;
        };

        while (ok) {
            const bool more = walk.next(a, slots);
            if (!more && !pending) break;
            const int nb = more ? walk.count(a) : 0, b0 = more ? walk.first_block() : 0;
            const int r0 = more ? pair_row0<DGRAD>(a, walk.tile, kCtas) : 0;
            // this group's first block of the segment (the turns go on from segment to segment: see
            // PairRings), and its slot and phase in each ring
            int i = pair_first(cnt, grp, NG);
            int ab = (cnt + i) % NA, xslot = (cnt + i) % SX;
            uint32_t aph = (uint32_t)((cnt + i) / NA) & 1u, xph = (uint32_t)((cnt + i) / SX) & 1u;
            const int ufirst = ucnt + i / UB;
            int pslot = ufirst % SP;
            uint32_t pph = (uint32_t)(ufirst / SP) & 1u;
            cnt += nb;
            if (more) ucnt += walk.units;
            // The A tiles of a block are written: visible to the tensor core, then counted; the
            // codes were used, so their slot is given back.
            auto release = [&]() {
                if constexpr (Cfg::kTmemA) {
                    tmem_wait_st();
                    tc_fence_before();
                } else {
                    fence_proxy_async_smem();
                }
                __syncwarp();
                // one warp of the group also vouches for the block's tokens
                if (wg == 0) {
                    ok = mbar_wait(xfull + 8 * xslot, xph) && ok;
                    xslot += NG;
                    const bool wrap = xslot >= SX;       // NG <= SX
                    xslot -= wrap ? SX : 0;
                    xph ^= wrap ? 1u : 0u;
                }
                if (lane == 0) {
                    if constexpr (PAIR) mbar_arrive_cluster(afull_r + 8 * ab);
                    else mbar_arrive(afull + 8 * ab);
                    // (a segment's last unit may have fewer blocks: the last one arrives for them too)
                    if (UB > 1 && i == nb - 1) mbar_arrive_n(pempty + 8 * pslot, (uint32_t)(UB - i % UB));
                    else mbar_arrive(pempty + 8 * pslot);
                }
                ab += NG;
                const bool awrap = ab >= NA;
                ab -= awrap ? NA : 0;
                aph ^= awrap ? 1u : 0u;
                pslot += (i % UB + NG) / UB;
                const bool pwrap = pslot >= SP;          // a step is at most SP
                pslot -= pwrap ? SP : 0;
                pph ^= pwrap ? 1u : 0u;
            };
            if constexpr (!DGRAD) {
                // thread = row r of both matrices
                const int r = wg * 32 + lane;
                const uint32_t sts0 = (uint32_t)(r * 128 + ((r & 7) * 16));               // chunk c: ^ 16·c
                // this row's codes in a unit; logical chunk c is at ^ 16·c (128- or 64-byte swizzle)
                const uint32_t lds0 = ps + (Cfg::kTmemA ? (uint32_t)(r * 128 + (r & 7) * 16)
                                                        : (uint32_t)(r * 64 + ((r >> 1) & 3) * 16));
                // The slot of scales at hand: every warp walks through all of a segment's, in order,
                // and gives one back when it goes on (what it read there was used by then).
                const int quad0 = pair_group(a, b0, 0) >> 2;
                auto advance = [&](int to) {
                    while (quad < to && ok) {
                        if (quad >= 0) {
                            __syncwarp();
                            if (lane == 0) mbar_arrive(qempty + 8 * qslot);
                        }
                        ++quad;
                        if (++qslot == Cfg::kQuads) { qslot = 0; qph ^= 1u; }
                        ok = mbar_wait(qfull + 8 * qslot, qph) && ok;
                    }
                };
                uint32_t sc[2][2], zc[2][2];                  // pairs of [matrix][half of the block]
                int have = -1;
                for (int phase = pending ? 0 : 1; phase < 2; ++phase) {
                    const int hi = phase == 0 ? min(nb, NA) : nb;
                    for (; i < hi && ok; i += NG) {
                        const int ga = pair_group(a, b0 + i, 0), gb = pair_group(a, b0 + i, 1);
                        if (ga != have || gb != ga) {
                            advance(quads + (ga >> 2) - quad0);
                            if (!ok) break;
                            const uint32_t at = qs + (uint32_t)(qslot * kPairQuadBytes + 8 * r + 2 * (ga & 3));
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                sc[j][0] = sc[j][1] = pair_scale(dup16(lds_u16(at + j * 8 * kPairRows)), worst);
                                zc[j][0] = zc[j][1] = pair_zero<BITS>(sym ? 0u : dup16(lds_u16(at + (2 + j) * 8 * kPairRows)), sym);
                            }
                            if (gb != ga) {                   // (g = 32: the next group, of the same four)
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    sc[j][1] = pair_scale(dup16(lds_u16(at + 2 + j * 8 * kPairRows)), worst);
                                    zc[j][1] = pair_zero<BITS>(sym ? 0u : dup16(lds_u16(at + 2 + (2 + j) * 8 * kPairRows)), sym);
                                }
                            }
                            have = ga;
                        }
                        // (the A slot first: once it is free, the code slot's previous unit was used,
                        // so the phase awaited next is not mistaken for an older one)
                        ok = mbar_wait(aempty + 8 * ab, aph ^ 1u) && ok;
                        ok = mbar_wait(pfull + 8 * pslot, pph) && ok;
                        if (!ok) break;
                        uint4 v[2][BITS / 2];
                        const uint32_t prow = (lds0 + (uint32_t)(pslot * Cfg::kUnitBytes)) ^ (uint32_t)(8 * BITS * (i % UB));
#pragma unroll
                        for (int c = 0; c < BITS / 2; ++c) {
                            v[0][c] = lds128_at<0>(prow ^ (uint32_t)(16 * c));
                            v[1][c] = lds128_at<Cfg::kUnitBytes / 2>(prow ^ (uint32_t)(16 * c));
                        }
                        const uint32_t arow = as + (uint32_t)(ab * kPairABytes) + sts0;
                        if constexpr (Cfg::kTmemA) tc_fence_after();          // behind the MMAs that read the slot
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint32_t o[32];                     // kTmemA: the row's 64 weights
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                uint32_t d[4];
                                if constexpr (BITS == 4) {
                                    const uint4 q = v[j][c >> 2];
                                    const uint32_t wd = (c & 3) == 0 ? q.x : ((c & 3) == 1 ? q.y : ((c & 3) == 2 ? q.z : q.w));
                                    pair_dequant8<4>(wd, 0u, a.flip, zc[j][c >> 2], sc[j][c >> 2], d);
                                } else {
                                    const uint4 q = v[j][c >> 1];
                                    pair_dequant8<8>((c & 1) ? q.z : q.x, (c & 1) ? q.w : q.y, a.flip, zc[j][c >> 2],
                                                     sc[j][c >> 2], d);
                                }
                                if constexpr (Cfg::kTmemA) {
#pragma unroll
                                    for (int e = 0; e < 4; ++e) o[4 * c + e] = d[e];
                                } else if (j == 0) {
                                    sts128_at<0>(arow ^ (uint32_t)(16 * c), d);
                                } else {
                                    sts128_at<kPairABytes / 2>(arow ^ (uint32_t)(16 * c), d);
                                }
                            }
                            if constexpr (Cfg::kTmemA)
                                tmem_st_32x32b_x32(tmem_a + (uint32_t)(64 * ab + 32 * j) + ((uint32_t)(wg * 32) << 16), o);
                        }
                        release();
                    }
                    if (phase == 0 && ok) epilogue();
                }
                if (more) {                                   // the segment's other slots
                    const int n = (pair_group(a, b0 + nb - 1, 1) >> 2) - quad0 + 1;
                    advance(quads + n - 1);
                    quads += n;
                }
            } else {
                // thread = weight row r of the block, 128 channels (one A tile) q: a warp's scale
                // loads touch sixteen rows.  The two threads of a row take their chunks in
                // orders that differ by 4, which keeps their shared-memory stores on
                // different banks.
                const int r = wg * 16 + (lane >> 1), q = lane & 1;
                const int c0 = r0 + rank * 2 * kPairRows + 128 * q;      // first input channel
                // (a row or channel behind the last reads the last one's pair: the tokens' values
                // there are zeros, or the results are dropped)
                const int pieces = a.gshift >= 7 ? 1 : (a.gshift == 6 ? 2 : 4);   // groups in 128 channels
                const int g0 = c0 >> a.gshift, glast = a.groups - 1, gfirst = min(g0, glast);
                auto fetch = [&](int blk, uint32_t (&sb)[4], uint32_t (&zb)[4]) {
                    int b = b0 + min(blk, nb - 1);
                    const bool second = b >= per_product;
                    if (second) b -= per_product;
                    const int64_t at = (int64_t)min(b * kPairBlock + r, a.N - 1) * a.groups;
                    const uint16_t* sp = (second ? a.scales[1] : a.scales[0]) + at;
                    const uint16_t* zp = (second ? a.zeros[1] : a.zeros[0]) + at;
                    sb[0] = ldg_u16(sp + gfirst);
                    if (!sym) zb[0] = ldg_u16(zp + gfirst);
                    if (pieces == 1) return;
#pragma unroll
                    for (int t = 1; t < 4; ++t)
                        if (t < pieces) {
                            sb[t] = ldg_u16(sp + min(g0 + t, glast));
                            if (!sym) zb[t] = ldg_u16(zp + min(g0 + t, glast));
                        }
                };
                // pairs of this group's next two blocks
                uint32_t sa[4], za[4], sn[4], zn[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) sa[t] = za[t] = sn[t] = zn[t] = 0u;
                if (more) {
                    fetch(i, sa, za);
                    fetch(i + NG, sn, zn);
                }
                const uint32_t row = ps + (uint32_t)(r * 128 + (BITS == 8 ? q * (kPairBlock * 128) : 0));
                const uint32_t line = as + (uint32_t)(q * (kPairABytes / 2) + r * 128 + (((4 * q) ^ (r & 7)) * 16));
                for (int phase = pending ? 0 : 1; phase < 2; ++phase) {
                    const int hi = phase == 0 ? min(nb, NA) : nb;
                    for (; i < hi && ok; i += NG) {
                        uint32_t sc[4], zc[4];                   // pairs of the four 32-channel pieces
                        sc[0] = pair_scale(dup16(sa[0]), worst);
                        zc[0] = pair_zero<BITS>(dup16(za[0]), sym);
                        if (pieces == 1) {
#pragma unroll
                            for (int t = 1; t < 4; ++t) {
                                sc[t] = sc[0];
                                zc[t] = zc[0];
                            }
                        } else {
#pragma unroll
                            for (int t = 1; t < 4; ++t) {
                                sc[t] = pair_scale(dup16(pieces == 4 ? sa[t] : sa[t >> 1]), worst);
                                zc[t] = pair_zero<BITS>(dup16(pieces == 4 ? za[t] : za[t >> 1]), sym);
                            }
                        }
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            sa[t] = sn[t];
                            za[t] = zn[t];
                        }
                        fetch(i + 2 * NG, sn, zn);
                        ok = mbar_wait(aempty + 8 * ab, aph ^ 1u) && ok;       // first, as above
                        ok = mbar_wait(pfull + 8 * pslot, pph) && ok;
                        if (!ok) break;
                        const uint32_t prow = row + (uint32_t)(pslot * Cfg::kUnitBytes);
                        uint4 v[BITS];                           // the thread's codes
#pragma unroll
                        for (int c = 0; c < BITS; ++c)
                            v[c] = lds128_addr(prow + (uint32_t)((((BITS == 4 ? 4 * q : 0) + c) ^ (r & 7)) * 16));
                        const uint32_t aline = line + (uint32_t)(ab * kPairABytes);
#pragma unroll
                        for (int b = 0; b < 2; ++b) {            // blocks of 64 channels
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                // step c: chunk c of thread 0, chunk c ^ 4 of thread 1
                                const uint32_t ss = q ? sc[2 * b + 1 - (c >> 2)] : sc[2 * b + (c >> 2)];
                                const uint32_t zz = q ? zc[2 * b + 1 - (c >> 2)] : zc[2 * b + (c >> 2)];
                                uint32_t d[4];
                                if constexpr (BITS == 4) {
                                    const uint4 lo = v[2 * b + (c >> 2)], hi4 = v[2 * b + 1 - (c >> 2)];
                                    const uint32_t wl = (c & 3) == 0 ? lo.x : ((c & 3) == 1 ? lo.y : ((c & 3) == 2 ? lo.z : lo.w));
                                    const uint32_t wh = (c & 3) == 0 ? hi4.x : ((c & 3) == 1 ? hi4.y : ((c & 3) == 2 ? hi4.z : hi4.w));
                                    pair_dequant8<4>(q ? wh : wl, 0u, a.flip, zz, ss, d);
                                } else {
                                    const uint4 x0 = v[4 * b + (c >> 1)], x1 = v[4 * b + ((c >> 1) ^ 2)];
                                    const uint32_t w0 = (c & 1) ? (q ? x1.z : x0.z) : (q ? x1.x : x0.x);
                                    const uint32_t w1 = (c & 1) ? (q ? x1.w : x0.w) : (q ? x1.y : x0.y);
                                    pair_dequant8<8>(w0, w1, a.flip, zz, ss, d);
                                }
                                if (b == 0) sts128_at<0>(aline ^ (uint32_t)(16 * c), d);
                                else sts128_at<8192>(aline ^ (uint32_t)(16 * c), d);
                            }
                        }
                        release();
                    }
                    if (phase == 0 && ok) epilogue();
                }
            }
            // this segment's epilogue waits for the next segment's first blocks
            pending = more;
            if (more) {
                e_r0 = r0;
                e_m0 = walk.tile % a.tiles_m * mma_n;
                e_publish = walk.u0 != 0;
                e_f1 = walk.followers_end(a, slot, slots);
            }
        }
        if (worst >= kPairNoScale) report_error(kErrWideScale);
        __syncwarp();
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();      // neither CTA leaves while the other may still use it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_g<PAIR>(tmem_d, tmem_cols);
    }
}

}  // namespace w4a16
