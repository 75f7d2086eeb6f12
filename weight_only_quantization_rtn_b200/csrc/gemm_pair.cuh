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
// PAIR: two CTAs of a cluster compute one tile together (cta_group::2): each holds its
// own 128 rows of both A tiles and half of the tokens, one thread of the even CTA issues
// the MMAs (M = 256) for both, and each SM reads half of the B operand.
//
// DGRAD needs Ŵ with the reduction along its rows.  The codes stay as they are stored:
// a block is 64 weight rows x 256 input channels, dequantized into the "MN-major" layout
// (64 channels contiguous per 128-byte swizzled line, lines along the rows), which the
// tensor core reads as the transposed A operand; nothing is transposed in memory.
//
// Warps: 0 loads (TMA: token tile with the 128-byte swizzle, codes), 1 issues the MMAs
// and owns the tensor memory, 2..9 dequantize and afterwards run the epilogue.  Scales
// and zero points go from global memory to registers, ahead of their block, so any
// number of groups per row and any alignment is read the same way.
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
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// mbar_wait for a barrier that the other CTA of the pair arrives on (bounded).
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if (global_timer_ns() - t0 > kWaitTimeoutNs) {
            report_error(kErrMbarTimeout);
            return false;
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
constexpr int kPairDequantWarps = 8;
constexpr int kPairThreads = (2 + kPairDequantWarps) * 32;
constexpr int kPairBlock = 64;          // reduction per stage
constexpr int kPairRows = 128;          // rows of one A tile per CTA
constexpr int kPairABytes = 2 * kPairRows * kPairBlock * 2;   // both A tiles of a stage

// BT: tokens of the CTA's B tile (PAIR: of each CTA; the MMA's N is 2·BT).
template <int BT, bool PAIR, int BITS>
struct PairConfig {
    static constexpr int kMmaN = PAIR ? 2 * BT : BT;
    static constexpr int kXBytes = BT * kPairBlock * 2;
    static constexpr int kPBytes = 2 * kPairRows * kPairBlock * BITS / 8;   // codes of a stage
    // Small token tiles: the loads of a stage are small beside the A tiles they turn into,
    // and they come from HBM, so they get a ring of their own, deep enough to cover the
    // memory latency; large tiles keep one ring (slot i holds X, codes and A tiles).
    static constexpr bool kSplitRing = !PAIR && BT < 128;
    static constexpr int kABufs0 = 3;
    static constexpr int kBudget = 232448 - 2048;
    static constexpr int kLoadBytes = kXBytes + kPBytes;
    static constexpr int kStagesRaw = kSplitRing ? (kBudget - kABufs0 * kPairABytes) / kLoadBytes
                                                 : kBudget / (kLoadBytes + kPairABytes);
    static constexpr int kStages = kStagesRaw > 8 ? 8 : kStagesRaw;
    static constexpr int kABufs = kSplitRing ? kABufs0 : kStages;
    static constexpr int kSmemBytes = kStages * kLoadBytes + kABufs * kPairABytes + 1024 + 1024;
    static constexpr int kTmemCols = 2 * kMmaN;
    static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "TMEM columns");
    static_assert(kStages >= 2 && kABufs >= 2 && kSmemBytes <= 232448, "shared memory");
};

struct PairArgs {
    const uint16_t* scales[2];   // GATED: gate, up; DGRAD: one per product
    const uint16_t* zeros[2];
    uint16_t* out;               // GATED: H [M, N]; DGRAD: dX [M, K]
    uint16_t* G;                 // GATED: kept outputs, or null
    uint16_t* U;
    float* partials;             // split reduction: fp32 parts, or null
    int M, N, K;
    int gshift;                  // log2 g; 31 for per-channel (one group per row)
    int groups;                  // groups per row
    uint32_t flip;               // symmetric codes: 0x88888888 or 0x80808080, else 0
    float zsym;                  // symmetric codes: 8 or 128 (the flipped code of 0), else 0
    int act;
    int products;                // DGRAD: 1 or 2
    int blocks;                  // reduction blocks in all
    int blocks_split;            // per split
};

// Zero point as the dequantization wants it: the bf16 pair of 128 + z (4-bit codes), or
// the binary32 2^23 + z (8-bit codes).
template <int BITS>
__device__ __forceinline__ uint32_t pair_zero(uint32_t z_bits, bool sym, float zsym) {
    const float z = sym ? zsym : bf16_bits_to_f32(z_bits);
    if (BITS == 4) return dup16(f32_to_bf16_bits_rn(128.0f + z));
    return __float_as_uint(8388608.0f + z);
}

// 32 codes (4-bit: one 16-byte chunk; 8-bit: two) of one scale group -> 16 bf16 pairs.
template <int BITS>
__device__ __forceinline__ void pair_dequant8(uint32_t w0, uint32_t w1, uint32_t flip, uint32_t zz,
                                              uint32_t s_bits, uint32_t out[4]) {
    if constexpr (BITS == 4) {
        const uint32_t ss = dup16(s_bits);
        const uint32_t lo = (w0 ^ flip) & 0x0F0F0F0Fu;
        const uint32_t hi = ((w0 ^ flip) >> 4) & 0x0F0F0F0Fu;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t sel = (uint32_t)j | 0x80u | ((uint32_t)(4 + j) << 8) | 0xC000u;
            out[j] = bf16x2_mul(bf16x2_sub(isolate_magic<false>(__byte_perm(lo, hi, sel), 0x000F000Fu), zz), ss);
        }
    } else {
        const float s = bf16_bits_to_f32(s_bits), zoff = __uint_as_float(zz);
        const uint32_t w[2] = {w0 ^ flip, w1 ^ flip};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i] = (__uint_as_float(__byte_perm(w[h], 0x4B000000u, 0x7540u + (uint32_t)i)) - zoff) * s;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out[2 * h]) : "f"(f[1]), "f"(f[0]));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out[2 * h + 1]) : "f"(f[3]), "f"(f[2]));
        }
    }
}

__device__ __forceinline__ void sts128_addr(uint32_t addr, const uint32_t v[4]) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3])
                 : "memory");
}

// Feature (GATED) or input channel (DGRAD) of row r of accumulator j of a CTA.
template <bool DGRAD>
__device__ __forceinline__ int pair_row(int r0, int rank, int j, int r) {
    return DGRAD ? r0 + rank * 2 * kPairRows + j * kPairRows + r : r0 + rank * kPairRows + r;
}

// One finished 32-token strip of a row: g (and u) hold the accumulators' values.
template <bool DGRAD>
__device__ __forceinline__ void pair_store(const PairArgs& a, int row0, int row1, int m, float v0, float v1) {
    if constexpr (DGRAD) {
        const int64_t at = (int64_t)m * a.K;
        if (row0 < a.K) a.out[at + row0] = (uint16_t)f32_to_bf16_bits_rn(v0);
        if (row1 < a.K) a.out[at + row1] = (uint16_t)f32_to_bf16_bits_rn(v1);
    } else {
        if (row0 >= a.N) return;
        const int64_t at = (int64_t)m * a.N + row0;
        a.out[at] = (uint16_t)f32_to_bf16_bits_rn(act_value(a.act, v0) * v1);
        if (a.G != nullptr) {
            a.G[at] = (uint16_t)f32_to_bf16_bits_rn(v0);
            a.U[at] = (uint16_t)f32_to_bf16_bits_rn(v1);
        }
    }
}

template <int BT, bool PAIR, int BITS, bool DGRAD>
__global__ void __launch_bounds__(kPairThreads, 1)
    gemm_pair_kernel(const __grid_constant__ CUtensorMap tmX0, const __grid_constant__ CUtensorMap tmX1,
                     const __grid_constant__ CUtensorMap tmP0, const __grid_constant__ CUtensorMap tmP1,
                     const PairArgs a) {
    using Cfg = PairConfig<BT, PAIR, BITS>;
    constexpr int S = Cfg::kStages, NA = Cfg::kABufs;
    constexpr bool kSplit = Cfg::kSplitRing;
    constexpr int kCtas = PAIR ? 2 : 1;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* as = smem;                              // NA x kPairABytes
    uint8_t* xs = as + NA * kPairABytes;             // S x kXBytes
    uint8_t* ps = xs + S * Cfg::kXBytes;             // S x kPBytes
    uint64_t* full = reinterpret_cast<uint64_t*>(ps + S * Cfg::kPBytes);
    uint64_t* empty = full + S;
    uint64_t* afull = empty + S;
    uint64_t* aempty = afull + NA;
    uint64_t* accf = aempty + NA;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(accf + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)cluster_ctarank() : 0;
    const int tile = (int)blockIdx.x / kCtas;
    const int tokens = kCtas * BT;
    const int tiles_m = (a.M + tokens - 1) / tokens;
    const int m0 = (tile % tiles_m) * tokens;
    const int r0 = (tile / tiles_m) * (DGRAD ? 2 : 1) * kCtas * kPairRows;
    const int b0 = (int)blockIdx.y * a.blocks_split;
    const int nb = min(a.blocks - b0, a.blocks_split);
    const int per_product = a.blocks / a.products;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), kSplit ? 1 + kPairDequantWarps : 1);
        }
        for (int s = 0; s < NA; ++s) {
            mbar_init(smem_u32(&afull[s]), kCtas * kPairDequantWarps);
            mbar_init(smem_u32(&aempty[s]), 1);
        }
        mbar_init(smem_u32(accf), 1);
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmX0);
        prefetch_tensormap(&tmP0);
        if (!DGRAD || a.products > 1) prefetch_tensormap(&tmP1);
        if (DGRAD && a.products > 1) prefetch_tensormap(&tmX1);
    }
    if (warp == 1) tmem_alloc_g<PAIR>(smem_u32(tmem_holder), Cfg::kTmemCols);
    tc_fence_before();
    __syncwarp();
    if constexpr (PAIR) cluster_sync_all();      // the pair's barriers are set up before either arrives
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem_d = *tmem_holder;

    if (warp == 0) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            int issued = 0;
            for (int i = 0; i < nb; ++i) {
                const int s = i % S;
                if (!mbar_wait(smem_u32(&empty[s]), ((uint32_t)(i / S) & 1u) ^ 1u)) break;
                const uint32_t bar = smem_u32(&full[s]);
                const uint32_t x = smem_u32(xs + s * Cfg::kXBytes), p = smem_u32(ps + s * Cfg::kPBytes);
                mbar_arrive_expect_tx(bar, Cfg::kXBytes + Cfg::kPBytes);
                if constexpr (DGRAD) {
                    const int b = b0 + i, prod = b / per_product, n = (b - prod * per_product) * kPairBlock;
                    const CUtensorMap* tx = prod ? &tmX1 : &tmX0;
                    const CUtensorMap* tp = prod ? &tmP1 : &tmP0;
                    tma_load_2d(x, tx, n, m0 + rank * BT, bar);
                    const int c0 = (r0 + rank * 2 * kPairRows) * BITS / 8;   // code bytes; boxes of 128
#pragma unroll
                    for (int h = 0; h < BITS / 4; ++h)
                        tma_load_2d(p + h * kPairBlock * 128, tp, c0 + 128 * h, n, bar);
                } else {
                    const int k = (b0 + i) * kPairBlock;
                    tma_load_2d(x, &tmX0, k, m0 + rank * BT, bar);
                    tma_load_2d(p, &tmP0, k * BITS / 8, r0 + rank * kPairRows, bar);
                    tma_load_2d(p + Cfg::kPBytes / 2, &tmP1, k * BITS / 8, r0 + rank * kPairRows, bar);
                }
                ++issued;
            }
            // Do not leave while copies into this CTA's shared memory are in flight.
            for (int i = (issued > S ? issued - S : 0); i < issued; ++i)
                if (!mbar_wait(smem_u32(&full[i % S]), (uint32_t)(i / S) & 1u)) break;
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issue (even CTA)
        if (lane == 0 && rank == 0) {
            constexpr uint32_t idesc = idesc_bf16_f32(kCtas * kPairRows, Cfg::kMmaN) |
                                       (DGRAD ? kIdescAMnMajor : 0u);
            for (int i = 0; i < nb; ++i) {
                const int s = i % S, ab = i % NA;
                // (the dequantizers arrive after the stage's loads landed, X among them)
                if (!mbar_wait_cluster(smem_u32(&afull[ab]), (uint32_t)(i / NA) & 1u)) break;
                tc_fence_after();
                const uint32_t at = smem_u32(as + ab * kPairABytes);
                const uint32_t xt = smem_u32(xs + s * Cfg::kXBytes);
#pragma unroll
                for (int kk = 0; kk < kPairBlock / 16; ++kk) {
                    const uint64_t bd = sw128_kmajor_desc(xt + kk * 32);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t aj = at + j * (kPairABytes / 2);
                        const uint64_t ad = DGRAD ? sw128_mnmajor_desc(aj + kk * 2048, 8192)
                                                  : sw128_kmajor_desc(aj + kk * 32);
                        tc_mma_bf16_g<PAIR>(tmem_d + (uint32_t)(j * Cfg::kMmaN), ad, bd, idesc,
                                            (i | kk) != 0 ? 1u : 0u);
                    }
                }
                tc_commit_g<PAIR>(smem_u32(&empty[s]));
                if (kSplit) tc_commit_g<PAIR>(smem_u32(&aempty[ab]));
            }
            tc_commit_g<PAIR>(smem_u32(accf));   // also on the error path: no MMA outlives the CTA
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ dequantize
        const int w = warp - 2;
        const bool sym = a.flip != 0u;
        bool ok = true;
        auto release = [&](int s, int ab) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) mbar_arrive_cluster(mapa_u32(smem_u32(&afull[ab]), 0));
                else mbar_arrive(smem_u32(&afull[ab]));
                if (kSplit) mbar_arrive(smem_u32(&empty[s]));
            }
        };
        if constexpr (!DGRAD) {
            // thread = row r of both tiles, 32-wide half h of the block
            const int r = (warp & 3) * 32 + lane, h = w >> 2;
            const int n = r0 + rank * kPairRows + r;
            const bool row_ok = n < a.N;
            const bool vec = (a.groups & 7) == 0;             // rows of scales are 16-byte aligned
            int have = -1;                                    // the group whose pair is in sg, zg
            uint32_t sg[2] = {0u, 0u}, zg[2] = {0u, 0u};
            uint4 sv[2], zv[2];
            for (int i = 0; i < nb; ++i) {
                const int s = i % S, ab = i % NA;
                const int k = (b0 + i) * kPairBlock + 32 * h;
                const int grp = min(k >> a.gshift, a.groups - 1);
                if (grp != have) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t sb = 0u, zb = 0u;
                        if (vec) {
                            if (have < 0 || (grp >> 3) != (have >> 3)) {
                                const int64_t at = (int64_t)n * a.groups + (grp & ~7);
                                sv[j] = row_ok ? ldg_cached(a.scales[j] + at) : make_uint4(0, 0, 0, 0);
                                zv[j] = row_ok && !sym ? ldg_cached(a.zeros[j] + at) : make_uint4(0, 0, 0, 0);
                            }
                            const int q = grp & 7;
                            const uint32_t sw = q < 4 ? (q < 2 ? sv[j].x : sv[j].y) : (q < 6 ? sv[j].z : sv[j].w);
                            const uint32_t zw = q < 4 ? (q < 2 ? zv[j].x : zv[j].y) : (q < 6 ? zv[j].z : zv[j].w);
                            sb = (sw >> (16 * (q & 1))) & 0xFFFFu;
                            zb = (zw >> (16 * (q & 1))) & 0xFFFFu;
                        } else if (row_ok) {
                            const int64_t at = (int64_t)n * a.groups + grp;
                            sb = ldg_u16(a.scales[j] + at);
                            if (!sym) zb = ldg_u16(a.zeros[j] + at);
                        }
                        sg[j] = sb;
                        zg[j] = pair_zero<BITS>(zb, sym, a.zsym);
                    }
                    have = grp;
                }
                if (!mbar_wait(smem_u32(&full[s]), (uint32_t)(i / S) & 1u)) {
                    ok = false;
                    break;
                }
                if (kSplit && !mbar_wait(smem_u32(&aempty[ab]), ((uint32_t)(i / NA) & 1u) ^ 1u)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint8_t* prow = ps + s * Cfg::kPBytes + j * (Cfg::kPBytes / 2) + r * (kPairBlock * BITS / 8);
                    uint4 v, v8 = make_uint4(0, 0, 0, 0);
                    if constexpr (BITS == 4) {
                        v = lds128(prow + 16 * (h ^ ((r >> 2) & 1)));           // 32-byte swizzle
                    } else {
                        v = lds128(prow + 16 * ((2 * h) ^ ((r >> 1) & 3)));     // 64-byte swizzle
                        v8 = lds128(prow + 16 * ((2 * h + 1) ^ ((r >> 1) & 3)));
                    }
                    const uint32_t wv[8] = {v.x, v.y, v.z, v.w, v8.x, v8.y, v8.z, v8.w};
                    const uint32_t arow = smem_u32(as + ab * kPairABytes + j * (kPairABytes / 2)) + r * 128;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t d[4];
                        if constexpr (BITS == 4) pair_dequant8<4>(wv[c], 0u, a.flip, zg[j], sg[j], d);
                        else pair_dequant8<8>(wv[2 * c], wv[2 * c + 1], a.flip, zg[j], sg[j], d);
                        sts128_addr(arow + (uint32_t)(((4 * h + c) ^ (r & 7)) * 16), d);
                    }
                }
                release(s, ab);
            }
        } else {
            // thread = weight row r of the block, 64-channel block q: the four threads of a row
            // are neighbours, so that a warp's scale loads touch eight rows.  Each starts
            // at another chunk (2q), which keeps its shared-memory stores off the
            // banks of the other three.
            const int r = w * 8 + (lane >> 2), q = lane & 3;
            const int c0 = r0 + rank * 2 * kPairRows + 64 * q;       // first input channel
            const bool chan_ok = c0 < a.K;
            const int g0 = min(c0 >> a.gshift, a.groups - 1), g1 = min((c0 + 32) >> a.gshift, a.groups - 1);
            // scales and zeros of the next blocks, two ahead (raw bf16 bits)
            uint32_t sn[2][2], zn[2][2];
            auto fetch = [&](int i, uint32_t* sb, uint32_t* zb) {
                const int b = b0 + i, prod = b / per_product, n = (b - prod * per_product) * kPairBlock + r;
                sb[0] = sb[1] = zb[0] = zb[1] = 0u;
                if (i < nb && n < a.N && chan_ok) {
                    const uint16_t* sp = prod ? a.scales[1] : a.scales[0];
                    const uint16_t* zp = prod ? a.zeros[1] : a.zeros[0];
                    const int64_t at = (int64_t)n * a.groups;
                    sb[0] = ldg_u16(sp + at + g0);
                    if (!sym) zb[0] = ldg_u16(zp + at + g0);
                    sb[1] = sb[0];
                    zb[1] = zb[0];
                    if (g1 != g0) {
                        sb[1] = ldg_u16(sp + at + g1);
                        if (!sym) zb[1] = ldg_u16(zp + at + g1);
                    }
                }
            };
            fetch(0, sn[0], zn[0]);
            fetch(1, sn[1], zn[1]);
            for (int i = 0; i < nb; ++i) {
                const int s = i % S, ab = i % NA;
                const uint32_t s0 = sn[0][0], s1 = sn[0][1];
                const uint32_t z0 = pair_zero<BITS>(zn[0][0], sym, a.zsym), z1 = pair_zero<BITS>(zn[0][1], sym, a.zsym);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    sn[0][t] = sn[1][t];
                    zn[0][t] = zn[1][t];
                }
                fetch(i + 2, sn[1], zn[1]);
                if (!mbar_wait(smem_u32(&full[s]), (uint32_t)(i / S) & 1u)) {
                    ok = false;
                    break;
                }
                if (kSplit && !mbar_wait(smem_u32(&aempty[ab]), ((uint32_t)(i / NA) & 1u) ^ 1u)) {
                    ok = false;
                    break;
                }
                const uint32_t line = smem_u32(as + ab * kPairABytes) + (uint32_t)(q * 8192 + r * 128);
                const uint8_t* pst = ps + s * Cfg::kPBytes;
                if constexpr (BITS == 4) {
                    // 32 code bytes: logical chunks 2q, 2q + 1 of the row's eight (128-byte swizzle)
                    const uint4 va = lds128(pst + r * 128 + (((2 * q) ^ (r & 7)) * 16));
                    const uint4 vb = lds128(pst + r * 128 + (((2 * q + 1) ^ (r & 7)) * 16));
                    uint32_t u[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w}, v[8];
                    // u rotated by 2q words: step c handles chunk (c + 2q) mod 8
#pragma unroll
                    for (int c = 0; c < 8; ++c) v[c] = (q & 2) ? u[(c + 4) & 7] : u[c];
#pragma unroll
                    for (int c = 0; c < 8; ++c) u[c] = (q & 1) ? v[(c + 2) & 7] : v[c];
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const int ch = (c + 2 * q) & 7;
                        uint32_t d[4];
                        pair_dequant8<4>(u[c], 0u, a.flip, ch < 4 ? z0 : z1, ch < 4 ? s0 : s1, d);
                        sts128_addr(line + (uint32_t)((ch ^ (r & 7)) * 16), d);
                    }
                } else {
                    // 64 code bytes: chunks 4(q & 1) .. + 3 of the row in box q / 2
                    const uint8_t* row = pst + (q >> 1) * (kPairBlock * 128) + r * 128;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int cc = (c + q) & 3;              // 16 channels 16·cc .. + 15
                        const uint4 vv = lds128(row + (((4 * (q & 1) + cc) ^ (r & 7)) * 16));
                        uint32_t d[4];
                        pair_dequant8<8>(vv.x, vv.y, a.flip, cc < 2 ? z0 : z1, cc < 2 ? s0 : s1, d);
                        sts128_addr(line + (uint32_t)(((2 * cc) ^ (r & 7)) * 16), d);
                        pair_dequant8<8>(vv.z, vv.w, a.flip, cc < 2 ? z0 : z1, cc < 2 ? s0 : s1, d);
                        sts128_addr(line + (uint32_t)(((2 * cc + 1) ^ (r & 7)) * 16), d);
                    }
                }
                release(s, ab);
            }
        }
        // ------------------------------------------------------------ epilogue
        if (ok && mbar_wait_cluster(smem_u32(accf), 0)) {
            tc_fence_after();
            const int r = (warp & 3) * 32 + lane, h = w >> 2;
            const int row0 = pair_row<DGRAD>(r0, rank, 0, r), row1 = pair_row<DGRAD>(r0, rank, 1, r);
            const uint32_t t_lane = tmem_d + ((uint32_t)((warp & 3) * 32) << 16);
            float* part = a.partials == nullptr ? nullptr
                          : a.partials + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (2 * Cfg::kMmaN * kPairRows);
#pragma unroll 1
            for (int cb = h; cb < Cfg::kMmaN / 32; cb += 2) {
                uint32_t v0[32], v1[32];
                tmem_ld_32x32b_x32(t_lane + cb * 32, v0);
                tmem_ld_32x32b_x32(t_lane + Cfg::kMmaN + cb * 32, v1);
                tmem_wait_ld();
                if (part != nullptr) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        part[(cb * 32 + j) * kPairRows + r] = __uint_as_float(v0[j]);
                        part[(Cfg::kMmaN + cb * 32 + j) * kPairRows + r] = __uint_as_float(v1[j]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const int m = m0 + cb * 32 + j;
                        if (m < a.M) pair_store<DGRAD>(a, row0, row1, m, __uint_as_float(v0[j]), __uint_as_float(v1[j]));
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncwarp();
    if constexpr (PAIR) cluster_sync_all();      // neither CTA leaves while the other may still use it
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_g<PAIR>(tmem_d, Cfg::kTmemCols);
    }
}

// Adds the parts of a split reduction in split order and runs the epilogue.  Parts are
// [split][CTA][accumulator][token of the tile][128 rows]; one thread per row and token.
template <bool DGRAD>
__global__ void __launch_bounds__(256) pair_reduce_kernel(const PairArgs a, int splits, int ctas, int mma_n,
                                                          int kctas) {
    grid_dependency_wait();
    const int64_t per_cta = 2ll * mma_n * kPairRows;
    const int64_t stride = (int64_t)ctas * per_cta;
    const int64_t items = (int64_t)ctas * mma_n * kPairRows;
    const int tiles_m = (a.M + mma_n - 1) / mma_n;
    for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < items;
         e += (int64_t)gridDim.x * blockDim.x) {
        const int cta = (int)(e / (mma_n * kPairRows));
        const int in = (int)(e - (int64_t)cta * mma_n * kPairRows);
        const int r = in % kPairRows, t = in / kPairRows;
        const int tile = cta / kctas, rank = cta % kctas;
        const int m = (tile % tiles_m) * mma_n + t;
        if (m >= a.M) continue;
        const int r0 = (tile / tiles_m) * (DGRAD ? 2 : 1) * kctas * kPairRows;
        const float* p = a.partials + cta * per_cta + in;
        float v0 = 0.0f, v1 = 0.0f;
        for (int z = 0; z < splits; ++z) {
            v0 += __ldcg(p + z * stride);
            v1 += __ldcg(p + z * stride + (int64_t)mma_n * kPairRows);
        }
        pair_store<DGRAD>(a, pair_row<DGRAD>(r0, rank, 0, r), pair_row<DGRAD>(r0, rank, 1, r), m, v0, v1);
    }
}

}  // namespace w4a16
