// Weight gradient of a linear layer, straight through the quantizer to the dense weight:
//
//   dW[n, k] = Σ_m dY[m, n]·X[m, k]      (bf16 in, binary32 accumulation, bf16 out)
//
// Both operands are read with the reduction along their rows, so both are MN-major
// operands of the tensor core: TMA brings boxes of 64 tokens x 64 features with the
// 128-byte swizzle and nothing is transposed.  Bound by the tensor cores for the token
// counts of a training step, by writing dW for short ones.  Two CTAs of a cluster share a
// 256 x 256 tile (cta_group::2: each SM holds 128 rows of dYᵀ and half of X's columns, and
// reads half of the B operand).  The kernel is persistent, one pair per two SMs, with two
// accumulators in tensor memory, so that one tile's epilogue overlaps the next one's
// MMAs: a tile of 2048 tokens is only about 9 us of MMAs.  A warp's 32 rows x 64 channels leave
// through shared memory as one TMA store of full 128-byte lines (a lane writing its own row
// in 16-byte pieces took 65 us for M = 77, N = K = 8192, where writing dW is all there is to do;
// so it takes 31).  M = 2048, N = 4096, K = 11008: 127 us, 1460 TFLOP/s, in a short run, 149 us in a
// long one (power limit).
#pragma once

#include "gemm_pair.cuh"

namespace w4a16 {

constexpr int kWgEpiWarps = 8;
constexpr int kWgThreads = (2 + kWgEpiWarps) * 32;
constexpr int kWgBlockM = 64;                    // tokens per stage
constexpr int kWgTile = 256;                     // features x channels per pair
constexpr int kWgStageBytes = 2 * 128 * kWgBlockM * 2;   // A and B halves of one CTA: 32 KB
constexpr int kWgStages = 6;
constexpr int kWgOutBytes = kWgEpiWarps * 4096;           // a warp's 32 rows x 64 channels
constexpr int kWgSmemBytes = kWgStages * kWgStageBytes + kWgOutBytes + 1024 + 1024;
static_assert(kWgSmemBytes <= 232448, "shared memory");

__global__ void __launch_bounds__(kWgThreads, 1)
    gemm_wgrad_kernel(const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmX,
                      const __grid_constant__ CUtensorMap tmW, int M, int N, int K) {
    constexpr int S = kWgStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* outs = smem + S * kWgStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(outs + kWgOutBytes);
    uint64_t* pfull = full + S;          // the odd CTA's stage has landed (at the even CTA)
    uint64_t* empty = pfull + S;
    uint64_t* accf = empty + S;          // [2] accumulator complete
    uint64_t* acce = accf + 2;           // [2] accumulator drained by both CTAs (at the even CTA)
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acce + 2);

    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);   // uniform
    const int lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const int pairs = (int)gridDim.x / 2, pair = (int)blockIdx.x / 2;
    const int tiles_n = (N + kWgTile - 1) / kWgTile, tiles_k = (K + kWgTile - 1) / kWgTile;
    const int tiles = tiles_n * tiles_k;
    const int nb = (M + kWgBlockM - 1) / kWgBlockM;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&pfull[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&accf[b]), 1);
            mbar_init(smem_u32(&acce[b]), 2 * kWgEpiWarps);
        }
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc_g<true>(smem_u32(tmem_holder), 512);
    tc_fence_before();
    __syncwarp();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_d = *tmem_holder;

    if (warp == 0) {
        if (lane == 0) {
            prefetch_tensormap(&tmY);
            prefetch_tensormap(&tmX);
            int i = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                const int n0 = (t % tiles_n) * kWgTile + rank * 128, k0 = (t / tiles_n) * kWgTile + rank * 128;
                for (int b = 0; b < nb; ++b, ++i) {
                    const int s = i % S;
                    ok = mbar_wait(smem_u32(&empty[s]), ((uint32_t)(i / S) & 1u) ^ 1u);
                    if (!ok) break;
                    const uint32_t st = smem_u32(smem + s * kWgStageBytes), bar = smem_u32(&full[s]);
                    mbar_arrive_expect_tx(bar, kWgStageBytes);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        tma_load_2d(st + h * 8192, &tmY, n0 + 64 * h, b * kWgBlockM, bar);
                        tma_load_2d(st + 16384 + h * 8192, &tmX, k0 + 64 * h, b * kWgBlockM, bar);
                    }
                }
            }
            for (int j = (i > S ? i - S : 0); j < i; ++j)     // no copy outlives the CTA
                if (!mbar_wait(smem_u32(&full[j % S]), (uint32_t)(j / S) & 1u)) break;
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && rank == 1) {
            // tell the even CTA when a stage of this one has landed
            int i = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs)
                for (int b = 0; b < nb && ok; ++b, ++i) {
                    ok = mbar_wait(smem_u32(&full[i % S]), (uint32_t)(i / S) & 1u);
                    if (ok) mbar_arrive_cluster(mapa_u32(smem_u32(&pfull[i % S]), 0));
                }
        } else if (rank == 0) {
            // the whole warp runs the loop (descriptors in uniform registers), one lane issues
            constexpr uint32_t idesc = idesc_bf16_f32(256, 256) | kIdescAMnMajor | kIdescBMnMajor;
            const uint64_t ad0 = sw128_mnmajor_desc(smem_u32(smem), 8192);
            const uint64_t bd0 = sw128_mnmajor_desc(smem_u32(smem) + 16384, 8192);
            int s = 0, it = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs, ++it) {
                const int buf = it & 1;
                ok = mbar_wait_cluster(smem_u32(&acce[buf]), ((uint32_t)(it >> 1) & 1u) ^ 1u);
                if (!ok) break;
                for (int b = 0; b < nb; ++b) {
                    ok = mbar_wait(smem_u32(&full[s]), ph) && mbar_wait_cluster(smem_u32(&pfull[s]), ph);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ad = ad0 + (uint32_t)(s * (kWgStageBytes / 16)), bd = bd0 + (uint32_t)(s * (kWgStageBytes / 16));
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < kWgBlockM / 16; ++kk)
                            tc_mma_bf16_g<true>(tmem_d + (uint32_t)(buf * 256), ad + kk * 128, bd + kk * 128, idesc,
                                                (b | kk) != 0 ? 1u : 0u);
                        tc_commit_g<true>(smem_u32(&empty[s]));
                        if (b == nb - 1) tc_commit_g<true>(smem_u32(&accf[buf]));
                    }
                    __syncwarp();
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
            }
            if (!ok && elect_one()) tc_commit_g<true>(smem_u32(&accf[it & 1]));   // error: no MMA outlives the CTA
        }
        __syncwarp();
    } else {
        // epilogue: lane = feature row, 64 channels at a time
        const int h = (warp - 2) >> 2, quarter = warp & 3;
        const uint32_t out = smem_u32(outs) + (uint32_t)((warp - 2) * 4096);
        int it = 0;
        if (lane == 0) prefetch_tensormap(&tmW);
        for (int t = pair; t < tiles; t += pairs, ++it) {
            const int buf = it & 1;
            const int n = (t % tiles_n) * kWgTile + rank * 128 + 32 * quarter, k0 = (t / tiles_n) * kWgTile;
            if (!mbar_wait_cluster(smem_u32(&accf[buf]), (uint32_t)(it >> 1) & 1u)) break;
            tc_fence_after();
#pragma unroll 1
            for (int cb = h; cb < kWgTile / 64; cb += 2) {
                uint32_t v[64];
                const uint32_t at = tmem_d + (uint32_t)(buf * 256 + cb * 64) + ((uint32_t)(quarter * 32) << 16);
                tmem_ld_32x32b_x32(at, v);
                tmem_ld_32x32b_x32(at + 32, v + 32);
                tmem_wait_ld();
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // staging is free
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint32_t p[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        p[j] = pack_bf16(__uint_as_float(v[8 * c + 2 * j]), __uint_as_float(v[8 * c + 2 * j + 1]));
                    sts128_addr(out + (uint32_t)(lane * 128 + ((c ^ (lane & 7)) * 16)), p);
                }
                fence_proxy_async_smem();
                __syncwarp();
                const int k = k0 + 64 * cb;
                if (lane == 0 && n < N && k < K)
                    asm volatile(
                        "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n\t"
                        "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(&tmW)),
                        "r"(k), "r"(n), "r"(out)
                        : "memory");
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_u32(smem_u32(&acce[buf]), 0));
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_g<true>(tmem_d, 512);
    }
}

}  // namespace w4a16
