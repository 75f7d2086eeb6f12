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
// PAIR (more than 128 tokens): two CTAs of a cluster compute one tile together
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
// Warps: 0 loads tokens (TMA, 128-byte swizzle), 18 loads codes (TMA), 1 issues the MMAs
// and owns the tensor memory, 2..17 dequantize and run the epilogue.  Three rings of
// shared memory, because the three have different sizes and lead times: token blocks,
// code units (GATED with 4 bits: 128 input channels, so that a row is 64 bytes; loaded as
// 32-byte rows the TMA engine's row rate, not bandwidth, paced the kernel) and dequantized
// A tiles.  Each dequantizing thread holds the next block's codes in registers while it
// works on the current one.  Scales and zero points go from global memory to registers
// ahead of their block, so any number of groups per row and any alignment is read the
// same way.
//
// The kernel is persistent, one CTA (or pair) per SM (or two): whole tiles are dealt in
// turn, and what is left (or everything, when there are fewer tiles than CTAs) may be
// split evenly along the reduction; then each CTA leaves binary32 parts of at most two
// tiles, which pair_reduce_kernel adds in a fixed order.
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
constexpr int kPairDequantWarps = 16;
constexpr int kPairCodeWarp = 2 + kPairDequantWarps;
constexpr int kPairThreads = (kPairCodeWarp + 1) * 32;
constexpr int kPairBlock = 64;          // reduction per block
constexpr int kPairRows = 128;          // rows of one A tile per CTA
constexpr int kPairABytes = 2 * kPairRows * kPairBlock * 2;   // both A tiles of a block: 32 KB
constexpr int kPairABufs = 3;
constexpr int kPairStageBytes = kPairDequantWarps * 1024;     // epilogue staging, 1 KB per warp
constexpr int kPairXBytes = 64 * 1024;                        // token ring
constexpr int kPairPBytes = 48 * 1024;                        // code ring
constexpr int kPairMaxX = 8;
constexpr int kPairSmemBytes = kPairABufs * kPairABytes + kPairXBytes + kPairPBytes + kPairStageBytes + 1024 + 1024;
static_assert(kPairSmemBytes <= 232448, "shared memory");

// Blocks of 64 that one code unit covers, and its bytes.
template <int BITS, bool DGRAD>
struct PairUnit {
    static constexpr int kBlocks = (!DGRAD && BITS == 4) ? 2 : 1;
    static constexpr int kBytes = 2 * kPairRows * kPairBlock * BITS / 8 * kBlocks;
    static constexpr int kSlots = kPairPBytes / kBytes;
    static_assert(kSlots >= 3, "code ring");
};

struct PairArgs {
    const uint16_t* scales[2];   // GATED: gate, up; DGRAD: one per product
    const uint16_t* zeros[2];
    uint16_t* out;               // GATED: H [M, N]; DGRAD: dX [M, K]
    uint16_t* G;                 // GATED: kept outputs, or null
    uint16_t* U;
    float* partials;             // split reduction: binary32 parts
    int M, N, K;
    int gshift;                  // log2 g; 31 for per-channel (one group per row)
    int groups;                  // groups per row
    uint32_t flip;               // symmetric codes: 0x88888888 or 0x80808080, else 0
    float zsym;                  // symmetric codes: 8 or 128 (the flipped code of 0), else 0
    int act;
    int products;                // DGRAD: 1 or 2
    int bt;                      // tokens of a CTA's tile (PAIR: half of the tile's)
    int acc_cols;                // tensor-memory columns of one accumulator (power of two)
    int blocks;                  // reduction blocks of a tile
    int tiles_m;
    int whole;                   // tiles [0, whole) are computed whole, dealt in turn
    int tiles;                   // the others [whole, tiles) are split evenly ...
    int sharers;                 // ... over this many CTAs (pairs), in code units; 0: none
};

// A CTA's (pair's) share of the work: whole tiles first, then its range of the split
// tiles' units, as segments (tile, first unit, units).
template <int UB>
struct PairWalk {
    int slots, slot, upt;        // CTAs (pairs), this one, units per tile
    int tile, u0, units;
    int64_t at, end;             // split range still to do
    int part;                    // index of a split segment's part, -1 for a whole tile
    __device__ __forceinline__ void init(const PairArgs& a, int slots_, int slot_) {
        slots = slots_;
        slot = slot_;
        upt = (a.blocks + UB - 1) / UB;
        tile = slot - slots;
        at = end = 0;
        if (a.sharers > 0 && slot < a.sharers) {
            const int64_t total = (int64_t)(a.tiles - a.whole) * upt;
            at = total * slot / a.sharers;
            end = total * (slot + 1) / a.sharers;
        }
        part = -1;
    }
    __device__ __forceinline__ bool next(const PairArgs& a) {
        if (part < 0) {
            tile += slots;
            if (tile < a.whole) {
                u0 = 0;
                units = upt;
                return true;
            }
        }
        if (at >= end) return false;
        ++part;                              // 0, then 1
        tile = a.whole + (int)(at / upt);
        u0 = (int)(at % upt);
        units = (int)(end - at < upt - u0 ? end - at : upt - u0);
        at += units;
        return true;
    }
    __device__ __forceinline__ int first_block() const { return u0 * UB; }
    __device__ __forceinline__ int count(const PairArgs& a) const {
        const int last = (u0 + units) * UB;
        return (last < a.blocks ? last : a.blocks) - u0 * UB;
    }
};

// Zero point as the dequantization wants it, from the bf16 pair (z, z): the pair of
// 128 + z (4-bit codes), or the binary32 2^23 + z (8-bit codes).
template <int BITS>
__device__ __forceinline__ uint32_t pair_zero(uint32_t zz, bool sym, float zsym) {
    if (BITS == 4) return sym ? 0x43084308u : bf16x2_add(zz, 0x43004300u);
    return __float_as_uint(8388608.0f + (sym ? zsym : __uint_as_float(zz & 0xFFFF0000u)));
}

// Eight codes -> four bf16 pairs in natural order.  4 bits (w0): PRMT brings code 2j of
// the word and code 2j + 1 of the word shifted by 4 into the low bytes of the halves, one
// LOP3 masks the nibbles and sets the exponent of 128 (symmetric codes: bit 3 flipped in
// the same LOP3).  8 bits (w0, w1): as dequant4_bytes in gemm_tcgen05.cuh.
template <int BITS>
__device__ __forceinline__ void pair_dequant8(uint32_t w0, uint32_t w1, uint32_t flip, uint32_t zz,
                                              uint32_t ss, uint32_t out[4]) {
    if constexpr (BITS == 4) {
        const uint32_t magic = 0x43004300u | (flip & 0x00080008u), hi = w0 >> 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // bytes: [w.j, any, (w >> 4).j, any]
            const uint32_t sel = (uint32_t)j | ((uint32_t)j << 4) | ((uint32_t)(4 + j) << 8) | ((uint32_t)(4 + j) << 12);
            uint32_t q;
            asm("lop3.b32 %0, %1, 0x000F000F, %2, 0x6A;" : "=r"(q) : "r"(__byte_perm(w0, hi, sel)), "r"(magic));
            out[j] = bf16x2_mul(bf16x2_sub(q, zz), ss);
        }
    } else {
        const float s = __uint_as_float(ss & 0xFFFF0000u), zoff = __uint_as_float(zz);
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

__device__ __forceinline__ uint4 lds128_addr(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
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
        if (a.act == W4A16_ACT_SILU) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v0[i] = act_value(W4A16_ACT_SILU, v0[i]) * v1[i];
        } else if (a.act == W4A16_ACT_GELU) {
#pragma unroll 1
            for (int i = 0; i < 16; ++i) v0[i] = act_value(W4A16_ACT_GELU, v0[i]) * v1[i];
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) v0[i] = act_value(a.act, v0[i]) * v1[i];
        }
        strip_store(v0, stage, a.out, m, a.M, c, a.N, lane);
    }
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

template <bool PAIR, int BITS, bool DGRAD>
__global__ void __launch_bounds__(kPairThreads, 1)
    gemm_pair_kernel(const __grid_constant__ CUtensorMap tmX0, const __grid_constant__ CUtensorMap tmX1,
                     const __grid_constant__ CUtensorMap tmP0, const __grid_constant__ CUtensorMap tmP1,
                     const PairArgs a) {
    using Unit = PairUnit<BITS, DGRAD>;
    constexpr int UB = Unit::kBlocks, SP = Unit::kSlots, NA = kPairABufs;
    constexpr int kCtas = PAIR ? 2 : 1;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t as = smem_u32(smem);              // NA x kPairABytes
    const uint32_t xs = as + NA * kPairABytes;       // token ring: SX x bt x 128 bytes
    const uint32_t ps = xs + kPairXBytes;            // SP code units
    const uint32_t st = ps + kPairPBytes;            // epilogue staging
    const uint32_t bars = st + kPairStageBytes;
    const int x_bytes = a.bt * kPairBlock * 2;
    const int SX = min(kPairXBytes / x_bytes, kPairMaxX);
    const uint32_t xfull = bars, xempty = xfull + 8 * kPairMaxX;
    const uint32_t pfull = xempty + 8 * kPairMaxX, pempty = pfull + 8 * SP;
    const uint32_t afull = pempty + 8 * SP, aempty = afull + 8 * NA;
    const uint32_t accf = aempty + 8 * NA;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + (accf + 8 - as));

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)cluster_ctarank() : 0;
    const int slots = (int)gridDim.x / kCtas, slot = (int)blockIdx.x / kCtas;
    const int per_product = a.blocks / a.products;
    const int mma_n = kCtas * a.bt;

    if (threadIdx.x == 0) {
        for (int s = 0; s < SX; ++s) {
            mbar_init(xfull + 8 * s, 1);
            mbar_init(xempty + 8 * s, 1);
        }
        for (int s = 0; s < SP; ++s) {
            mbar_init(pfull + 8 * s, 1);
            mbar_init(pempty + 8 * s, UB * kPairDequantWarps / 2);
        }
        for (int s = 0; s < NA; ++s) {
            mbar_init(afull + 8 * s, kCtas * kPairDequantWarps / 2);
            mbar_init(aempty + 8 * s, 1);
        }
        mbar_init(accf, 1);
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
    if (warp == 1) tmem_alloc_g<PAIR>(smem_u32(tmem_holder), 2 * a.acc_cols);
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();      // the pair's barriers are set up before either arrives
    tc_fence_after();
    const uint32_t tmem_d = *tmem_holder;
    PairWalk<UB> walk;
    walk.init(a, slots, slot);

    if (warp == 0) {
        // ------------------------------------------------------------ token loads
        if (lane == 0) {
            int s = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            while (ok && walk.next(a)) {
                const int b0 = walk.first_block(), nb = walk.count(a);
                const int m0 = walk.tile % a.tiles_m * mma_n + rank * a.bt;
                for (int i = 0; i < nb; ++i) {
                    ok = mbar_wait(xempty + 8 * s, ph ^ 1u);
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
            while (ok && walk.next(a)) {
                const int r0 = pair_row0<DGRAD>(a, walk.tile, kCtas);
                for (int u = 0; u < walk.units; ++u) {
                    ok = mbar_wait(pempty + 8 * s, ph ^ 1u);
                    if (!ok) break;
                    const uint32_t bar = pfull + 8 * s, p = ps + s * Unit::kBytes;
                    mbar_arrive_expect_tx(bar, Unit::kBytes);
                    if constexpr (DGRAD) {
                        int b = walk.u0 + u;
                        const CUtensorMap* tp = &tmP0;
                        if (b >= per_product) {
                            b -= per_product;
                            tp = &tmP1;
                        }
                        const int c0 = (r0 + rank * 2 * kPairRows) * BITS / 8;   // code bytes; boxes of 128
#pragma unroll
                        for (int h = 0; h < BITS / 4; ++h)
                            tma_load_2d(p + h * kPairBlock * 128, tp, c0 + 128 * h, b * kPairBlock, bar);
                    } else {
                        const int k = (walk.u0 + u) * UB * kPairBlock, n = r0 + rank * kPairRows;
                        tma_load_2d(p, &tmP0, k * BITS / 8, n, bar);
                        tma_load_2d(p + Unit::kBytes / 2, &tmP1, k * BITS / 8, n, bar);
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
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = idesc_bf16_f32(kCtas * kPairRows, mma_n) | (DGRAD ? kIdescAMnMajor : 0u);
            int s = 0, ab = 0;
            uint32_t pa = 0;
            bool ok = true;
            while (ok && walk.next(a)) {
                const int nb = walk.count(a);
                for (int i = 0; i < nb; ++i) {
                    // (a dequantizing warp of each CTA arrives after the tokens landed there too)
                    ok = mbar_wait_cluster(afull + 8 * ab, pa);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t at = as + ab * kPairABytes, xt = xs + s * x_bytes;
#pragma unroll
                    for (int kk = 0; kk < kPairBlock / 16; ++kk) {
                        const uint64_t bd = sw128_kmajor_desc(xt + kk * 32);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t aj = at + j * (kPairABytes / 2);
                            const uint64_t ad = DGRAD ? sw128_mnmajor_desc(aj + kk * 2048, 8192)
                                                      : sw128_kmajor_desc(aj + kk * 32);
                            tc_mma_bf16_g<PAIR>(tmem_d + (uint32_t)(j * a.acc_cols), ad, bd, idesc,
                                                (i | kk) != 0 ? 1u : 0u);
                        }
                    }
                    tc_commit_g<PAIR>(xempty + 8 * s);
                    tc_commit_g<PAIR>(aempty + 8 * ab);
                    if (++s == SX) s = 0;
                    if (++ab == NA) { ab = 0; pa ^= 1u; }
                }
                tc_commit_g<PAIR>(accf);         // also on the error path: no MMA outlives the CTA
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ dequantize, epilogue
        // Two groups of eight warps take the blocks in turn, so that one group's waits, fences
        // and loads hide behind the other's arithmetic and each warp pays its per-block
        // overhead for eight chunks of codes.
        const int w = warp - 2, grp = w >> 3, wg = w & 7;
        const bool sym = a.flip != 0u;
        const uint32_t afull_r = PAIR ? mapa_u32(afull, 0) : afull;
        int cnt = 0, ucnt = 0, seg = 0;              // blocks and units of the segments before
        bool ok = true;
        while (ok && walk.next(a)) {
            const int r0 = pair_row0<DGRAD>(a, walk.tile, kCtas);
            const int b0 = walk.first_block(), nb = walk.count(a);
            // this group's first block in each ring: slot and phase
            int ab = (cnt + grp) % NA, xslot = (cnt + grp) % SX;
            uint32_t aph = (uint32_t)((cnt + grp) / NA) & 1u, xph = (uint32_t)((cnt + grp) / SX) & 1u;
            const int ufirst = ucnt + (UB == 2 ? 0 : grp);
            int pslot = ufirst % SP;
            uint32_t pph = (uint32_t)(ufirst / SP) & 1u;
            cnt += nb;
            ucnt += walk.units;
            // The A tiles of a block are written: visible to the tensor core, then counted; the
            // codes were used, so their slot is given back.  (Given back right behind the
            // loads, a slot was seen refilled before a load of it had been performed.)
            auto release = [&]() {
                fence_proxy_async_smem();
                __syncwarp();
                // one warp of the group also vouches for the block's tokens
                if (wg == 0) ok = mbar_wait(xfull + 8 * xslot, xph) && ok;
                if (lane == 0) {
                    if constexpr (PAIR) mbar_arrive_cluster(afull_r + 8 * ab);
                    else mbar_arrive(afull + 8 * ab);
                    mbar_arrive(pempty + 8 * pslot);
                }
                xslot += 2;
                if (xslot >= SX) { xslot -= SX; xph ^= 1u; }
                ab += 2;
                if (ab >= NA) { ab -= NA; aph ^= 1u; }
                pslot += UB == 2 ? 1 : 2;
                if (pslot >= SP) { pslot -= SP; pph ^= 1u; }
            };
            if constexpr (!DGRAD) {
                // thread = row r of both matrices, 32-wide half h of the block
                const int r = (wg & 3) * 32 + lane, h = wg >> 2;
                const int n = r0 + rank * kPairRows + r;
                const bool row_ok = n < a.N;
                const bool vec = (a.groups & 7) == 0;         // rows of scales are 16-byte aligned
                const int64_t srow = (int64_t)(row_ok ? n : 0) * a.groups;
                const uint32_t sts0 = (uint32_t)(r * 128 + (((4 * h) ^ (r & 7)) * 16));   // chunk c: ^ 16·c
                const uint32_t lds0 = ps + (uint32_t)(r * 64) +
                                      (uint32_t)(((BITS == 4 ? 2 * grp + h : 2 * h) ^ ((r >> 1) & 3)) * 16);
                uint32_t ss[2], zz[2];                        // the current group's pairs
                int have = -1;
                if (!vec) {
                    // the pair of the group ahead, loaded one change early
                    const int g0 = min(((b0 + grp) * kPairBlock + 32 * h) >> a.gshift, a.groups - 1);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        ss[j] = row_ok ? ldg_u16(a.scales[j] + srow + g0) : 0u;
                        zz[j] = row_ok && !sym ? ldg_u16(a.zeros[j] + srow + g0) : 0u;
                    }
                }
                uint4 s8[2], z8[2];                           // eight groups of the row
                uint32_t sc[2] = {0u, 0u}, zc[2] = {0u, 0u};
                for (int i = grp; i < nb && ok; i += 2) {
                    const int g = min(((b0 + i) * kPairBlock + 32 * h) >> a.gshift, a.groups - 1);
                    if (g != have) {
                        if (vec) {
                            if (have < 0 || (g >> 3) != (have >> 3)) {
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    s8[j] = row_ok ? ldg_cached(a.scales[j] + srow + (g & ~7)) : make_uint4(0, 0, 0, 0);
                                    z8[j] = row_ok && !sym ? ldg_cached(a.zeros[j] + srow + (g & ~7)) : make_uint4(0, 0, 0, 0);
                                }
                            }
                            const bool up = (g & 4) != 0, odd = (g & 2) != 0;
                            const uint32_t sel = (g & 1) ? 0x3232u : 0x1010u;
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const uint32_t s0 = up ? s8[j].z : s8[j].x, s1 = up ? s8[j].w : s8[j].y;
                                const uint32_t z0 = up ? z8[j].z : z8[j].x, z1 = up ? z8[j].w : z8[j].y;
                                sc[j] = __byte_perm(odd ? s1 : s0, 0u, sel);
                                zc[j] = pair_zero<BITS>(__byte_perm(odd ? z1 : z0, 0u, sel), sym, a.zsym);
                            }
                        } else {
                            const int gn = min(((b0 + i + 2) * kPairBlock + 32 * h) >> a.gshift, a.groups - 1);
                            const int ahead = gn != g ? gn : min(g + 1, a.groups - 1);
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                sc[j] = dup16(ss[j]);
                                zc[j] = pair_zero<BITS>(dup16(zz[j]), sym, a.zsym);
                                ss[j] = row_ok ? ldg_u16(a.scales[j] + srow + ahead) : 0u;
                                zz[j] = row_ok && !sym ? ldg_u16(a.zeros[j] + srow + ahead) : 0u;
                            }
                        }
                        have = g;
                    }
                    ok = mbar_wait(pfull + 8 * pslot, pph) && ok;
                    uint4 v[2], v8[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t at = lds0 + (uint32_t)(pslot * Unit::kBytes + j * (Unit::kBytes / 2));
                        v[j] = lds128_addr(at);
                        v8[j] = BITS == 8 ? lds128_addr(at ^ 16u) : make_uint4(0, 0, 0, 0);
                    }
                    ok = mbar_wait(aempty + 8 * ab, aph ^ 1u) && ok;
                    if (!ok) break;
                    const uint32_t arow = as + (uint32_t)(ab * kPairABytes) + sts0;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t wv[8] = {v[j].x, v[j].y, v[j].z, v[j].w, v8[j].x, v8[j].y, v8[j].z, v8[j].w};
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t d[4];
                            if constexpr (BITS == 4) pair_dequant8<4>(wv[c], 0u, a.flip, zc[j], sc[j], d);
                            else pair_dequant8<8>(wv[2 * c], wv[2 * c + 1], a.flip, zc[j], sc[j], d);
                            sts128_addr((arow ^ (uint32_t)(16 * c)) + (uint32_t)(j * (kPairABytes / 2)), d);
                        }
                    }
                    release();
                }
                if (UB == 2 && ok && grp == 1 && (nb & 1)) {
                    // the segment's last unit has no block for this group
                    ok = mbar_wait(pfull + 8 * pslot, pph) && ok;
                    if (lane == 0) mbar_arrive(pempty + 8 * pslot);
                }
            } else {
                // thread = weight row r of the block, 64-channel block q: the four threads of a row
                // are neighbours, so that a warp's scale loads touch eight rows.  Each starts
                // at another chunk (2q), which keeps its shared-memory stores off the banks
                // of the other three.
                const int r = wg * 8 + (lane >> 2), q = lane & 3;
                const int c0 = r0 + rank * 2 * kPairRows + 64 * q;       // first input channel
                const bool chan_ok = c0 < a.K;
                const int g0 = min(c0 >> a.gshift, a.groups - 1), g1 = min((c0 + 32) >> a.gshift, a.groups - 1);
                auto fetch = [&](int i, uint32_t* sb, uint32_t* zb) {
                    int b = b0 + i;
                    const bool second = b >= per_product;
                    if (second) b -= per_product;
                    const int n = b * kPairBlock + r;
                    sb[0] = sb[1] = zb[0] = zb[1] = 0u;
                    if (i < nb && n < a.N && chan_ok) {
                        const uint16_t* sp = (second ? a.scales[1] : a.scales[0]) + (int64_t)n * a.groups;
                        const uint16_t* zp = (second ? a.zeros[1] : a.zeros[0]) + (int64_t)n * a.groups;
                        sb[0] = ldg_u16(sp + g0);
                        if (!sym) zb[0] = ldg_u16(zp + g0);
                        if (g1 != g0) {
                            sb[1] = ldg_u16(sp + g1);
                            if (!sym) zb[1] = ldg_u16(zp + g1);
                        }
                    }
                };
                // pairs of this group's next two blocks
                uint32_t sn[2][2], zn[2][2];
                fetch(grp, sn[0], zn[0]);
                fetch(grp + 2, sn[1], zn[1]);
                const uint32_t row = ps + (uint32_t)(r * 128);
                const uint32_t line = as + (uint32_t)(q * 8192 + r * 128);
                for (int i = grp; i < nb && ok; i += 2) {
                    uint32_t sc[2], zc[2];
                    sc[0] = dup16(sn[0][0]);
                    zc[0] = pair_zero<BITS>(dup16(zn[0][0]), sym, a.zsym);
                    sc[1] = g1 != g0 ? dup16(sn[0][1]) : sc[0];
                    zc[1] = g1 != g0 ? pair_zero<BITS>(dup16(zn[0][1]), sym, a.zsym) : zc[0];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        sn[0][t] = sn[1][t];
                        zn[0][t] = zn[1][t];
                    }
                    fetch(i + 4, sn[1], zn[1]);
                    ok = mbar_wait(pfull + 8 * pslot, pph) && ok;
                    const uint32_t prow = row + (uint32_t)(pslot * Unit::kBytes);
                    const uint32_t aline = line + (uint32_t)(ab * kPairABytes);
                    if constexpr (BITS == 4) {
                        // 32 code bytes: logical chunks 2q, 2q + 1 of the row's eight (128-byte swizzle)
                        const uint32_t at = prow + (uint32_t)(((2 * q) ^ (r & 7)) * 16);
                        const uint4 va = lds128_addr(at), vb = lds128_addr(at ^ 16u);
                        uint32_t u[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w}, v[8];
                        // u rotated by 2q words: step c handles chunk (c + 2q) mod 8
#pragma unroll
                        for (int c = 0; c < 8; ++c) v[c] = (q & 2) ? u[(c + 4) & 7] : u[c];
#pragma unroll
                        for (int c = 0; c < 8; ++c) u[c] = (q & 1) ? v[(c + 2) & 7] : v[c];
                        ok = mbar_wait(aempty + 8 * ab, aph ^ 1u) && ok;
                        if (!ok) break;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const int ch = (c + 2 * q) & 7;
                            const bool hi = ch >= 4;
                            uint32_t d[4];
                            pair_dequant8<4>(u[c], 0u, a.flip, hi ? zc[1] : zc[0], hi ? sc[1] : sc[0], d);
                            sts128_addr(aline + (uint32_t)((ch ^ (r & 7)) * 16), d);
                        }
                    } else {
                        ok = mbar_wait(aempty + 8 * ab, aph ^ 1u) && ok;
                        if (!ok) break;
                        // 64 code bytes: chunks 4(q & 1) .. + 3 of the row in box q / 2
                        const uint32_t box = prow + (uint32_t)((q >> 1) * (kPairBlock * 128));
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int cc = (c + q) & 3;              // channels 16·cc .. + 15
                            const uint4 vv = lds128_addr(box + (uint32_t)(((4 * (q & 1) + cc) ^ (r & 7)) * 16));
                            const bool hi = cc >= 2;
                            uint32_t d[4];
                            pair_dequant8<8>(vv.x, vv.y, a.flip, hi ? zc[1] : zc[0], hi ? sc[1] : sc[0], d);
                            sts128_addr(aline + (uint32_t)(((2 * cc) ^ (r & 7)) * 16), d);
                            pair_dequant8<8>(vv.z, vv.w, a.flip, hi ? zc[1] : zc[0], hi ? sc[1] : sc[0], d);
                            sts128_addr(aline + (uint32_t)(((2 * cc + 1) ^ (r & 7)) * 16), d);
                        }
                    }
                    release();
                }
            }
            // -------------------------------------------------------- epilogue
            if (!ok || !mbar_wait_cluster(accf, (uint32_t)seg & 1u)) break;
            ++seg;
            tc_fence_after();
            const int quarter = warp & 3;                      // the lanes this warp may read
            const int m0 = walk.tile % a.tiles_m * mma_n;
            const int strips = (min(mma_n, a.M - m0) + 15) / 16;
            const uint32_t t_lane = tmem_d + ((uint32_t)(quarter * 32) << 16);
            // which of the quarter's four warps this one is
            for (int sidx = w >> 2; sidx < strips; sidx += kPairDequantWarps / 4) {
                uint32_t v0[16], v1[16];
                const uint32_t t0 = t_lane + 16 * sidx;
                tmem_ld_16x256b_x2(t0, v0);
                tmem_ld_16x256b_x2(t0 + (16u << 16), v0 + 8);
                tmem_ld_16x256b_x2(t0 + a.acc_cols, v1);
                tmem_ld_16x256b_x2(t0 + a.acc_cols + (16u << 16), v1 + 8);
                tmem_wait_ld();
                if (walk.part < 0) {
                    float f0[16], f1[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        f0[e] = __uint_as_float(v0[e]);
                        f1[e] = __uint_as_float(v1[e]);
                    }
                    pair_emit<DGRAD>(a, f0, f1, st + w * 1024, r0, rank, quarter, m0 + 16 * sidx, lane);
                } else {
                    float4* part = reinterpret_cast<float4*>(
                        a.partials + ((int64_t)(slot * 2 + walk.part) * kCtas + rank) * pair_part_floats(mma_n) +
                        (int64_t)(sidx * 4 + quarter) * (2 * 16 * 32));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        part[e * 32 + lane] = make_float4(__uint_as_float(v0[4 * e]), __uint_as_float(v0[4 * e + 1]),
                                                          __uint_as_float(v0[4 * e + 2]), __uint_as_float(v0[4 * e + 3]));
                        part[(4 + e) * 32 + lane] =
                            make_float4(__uint_as_float(v1[4 * e]), __uint_as_float(v1[4 * e + 1]),
                                        __uint_as_float(v1[4 * e + 2]), __uint_as_float(v1[4 * e + 3]));
                    }
                }
            }
            tc_fence_before();      // the reads above precede this warp's next arrival, hence the next MMA
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();      // neither CTA leaves while the other may still use it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_g<PAIR>(tmem_d, 2 * a.acc_cols);
    }
}

// Adds the parts of the split tiles in the order of the reduction and runs the epilogue:
// one warp per strip of a CTA's rows, in the layout the parts were left in.
constexpr int kPairReduceThreads = 128;
template <bool DGRAD>
__global__ void __launch_bounds__(kPairReduceThreads) pair_reduce_kernel(const PairArgs a, int ctas, int upt) {
    __shared__ __align__(16) uint8_t stage[kPairReduceThreads / 32 * 1024];
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mma_n = ctas * a.bt, strips = (mma_n + 15) / 16;
    const int64_t item = (int64_t)blockIdx.x * (kPairReduceThreads / 32) + warp;
    const int quarter = (int)(item % 4), sidx = (int)(item / 4 % strips);
    const int64_t rest = item / 4 / strips;
    const int rank = (int)(rest % ctas), split = (int)(rest / ctas);
    const int tile = a.whole + split;
    if (tile >= a.tiles) return;
    const int m = tile % a.tiles_m * mma_n + 16 * sidx;
    if (m >= a.M) return;
    const int64_t total = (int64_t)(a.tiles - a.whole) * upt, u0 = (int64_t)split * upt, u1 = u0 + upt;
    // sharer c holds units [total·c/S, total·(c + 1)/S)
    const int first = (int)(((u0 + 1) * a.sharers - 1) / total), last = (int)((u1 * a.sharers - 1) / total);
    float v0[16], v1[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) v0[e] = v1[e] = 0.0f;
    for (int c = first; c <= last; ++c) {
        const int seg = total * c / a.sharers >= u0 ? 0 : 1;       // the tile is the sharer's first or second
        const float4* part = reinterpret_cast<const float4*>(
            a.partials + ((int64_t)(c * 2 + seg) * ctas + rank) * pair_part_floats(mma_n) +
            (int64_t)(sidx * 4 + quarter) * (2 * 16 * 32));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 p = __ldcg(part + e * 32 + lane), q = __ldcg(part + (4 + e) * 32 + lane);
            v0[4 * e] += p.x; v0[4 * e + 1] += p.y; v0[4 * e + 2] += p.z; v0[4 * e + 3] += p.w;
            v1[4 * e] += q.x; v1[4 * e + 1] += q.y; v1[4 * e + 2] += q.z; v1[4 * e + 3] += q.w;
        }
    }
    pair_emit<DGRAD>(a, v0, v1, smem_u32(stage) + warp * 1024, pair_row0<DGRAD>(a, tile, ctas), rank, quarter, m, lane);
}

}  // namespace w4a16
