// Quantized embedding: table lookup, and the gradient of the dense table behind it.
//
// Lookup:  out[t, :] = bf16_rn(scale·Ŵ[id_t, :]),  Ŵ = bf16_rn((q − z)·s)
// A row is gathered as codes (0.53 bytes per weight with 4 bits), dequantized in
// registers and written once: bound by writing the bf16 rows.  One thread per 8 codes, so
// a warp reads 128 (256) contiguous code bytes and writes 512 contiguous bytes.
//
// Gradient:  dW[v, :] = scale·Σ_{t: id_t = v} dY[t, :], summed in binary32 in ascending t
// within windows of kGradWindow sorted tokens, windows added in order: the same inputs
// give the same bits.  Four steps, no atomics on values:
//   1. chunks of kSortChunk ids are sorted by (id, t) in shared memory, one bit of the id
//      per pass (each pass a stable split), one CTA per chunk;
//   2. with more than one chunk, each element's place among the other chunks is found by
//      binary search: its rank in the whole sorted list;
//   3. windows of kGradWindow sorted tokens are summed, one thread per 8 columns; runs of one
//      id inside a window are written at once, runs that cross its border leave a
//      binary32 part; rows of the table that no token names are set to zero by the same
//      launch, which is what most of its time goes to;
//   4. parts of a run are added in window order and written.
// An id below 0 or not below V names no row: it sorts behind all others and is dropped.
#pragma once

#include "common.cuh"

namespace w4a16 {

constexpr int kErrBadId = 2;

__device__ __forceinline__ int64_t load_id(const void* ids, int wide, int64_t t) {
    return wide ? static_cast<const int64_t*>(ids)[t] : (int64_t)static_cast<const int32_t*>(ids)[t];
}

// ------------------------------------------------------------------ lookup
template <int BITS>
__global__ void __launch_bounds__(256) embedding_kernel(const void* __restrict__ ids, int wide,
                                                        const uint8_t* __restrict__ codes,
                                                        const uint16_t* __restrict__ scales,
                                                        const uint16_t* __restrict__ zeros, int64_t V,
                                                        int chunks, int gshift, int groups, int sym,
                                                        float scale, uint4* __restrict__ out) {
    constexpr int U = 4;                                   // 8-code chunks per thread, 256 apart
    const int64_t t = blockIdx.x;
    const int64_t id = load_id(ids, wide, t);
    const bool valid = id >= 0 && id < V;
    if (id >= V && threadIdx.x == 0 && blockIdx.y == 0) report_error(kErrBadId);
    const int c0 = (int)blockIdx.y * 256 * U + threadIdx.x;
    const int64_t row = valid ? id : 0;
    const uint32_t flip = sym ? (BITS == 4 ? 0x88888888u : 0x80808080u) : 0u;
    uint2 w[U];
    uint32_t sb[U], zb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = c0 + 256 * u;
        w[u] = make_uint2(0u, 0u);
        sb[u] = zb[u] = 0u;
        if (valid && c < chunks) {
            if constexpr (BITS == 4) w[u].x = __ldg(reinterpret_cast<const uint32_t*>(codes + (row * chunks + c) * 4));
            else w[u] = __ldg(reinterpret_cast<const uint2*>(codes + (row * chunks + c) * 8));
            const int64_t at = row * groups + min((8 * c) >> gshift, groups - 1);
            sb[u] = ldg_u16(scales + at);
            if (!sym) zb[u] = ldg_u16(zeros + at);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = c0 + 256 * u;
        if (c >= chunks) continue;
        uint32_t d[4];
        if constexpr (BITS == 4) {
            const float z = sym ? 8.0f : bf16_bits_to_f32(zb[u]);
            dequant8_natural<false>(w[u].x ^ flip, dup16(f32_to_bf16_bits_rn(128.0f + z)), dup16(sb[u]), d);
        } else {
            const float s = bf16_bits_to_f32(sb[u]);
            const float zoff = 8388608.0f + (sym ? 128.0f : bf16_bits_to_f32(zb[u]));
            const uint32_t ww[2] = {w[u].x ^ flip, w[u].y ^ flip};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float f[2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    f[j] = (__uint_as_float(__byte_perm(ww[i >> 1], 0x4B000000u,
                                                        0x7540u + (uint32_t)(2 * (i & 1) + j))) - zoff) * s;
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d[i]) : "f"(f[1]), "f"(f[0]));
            }
        }
        if (!valid) {
            d[0] = d[1] = d[2] = d[3] = 0u;
        } else if (scale != 1.0f) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float lo = __uint_as_float(d[i] << 16) * scale, hi = __uint_as_float(d[i] & 0xFFFF0000u) * scale;
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d[i]) : "f"(hi), "f"(lo));
            }
        }
        out[t * chunks + c] = make_uint4(d[0], d[1], d[2], d[3]);
    }
}

// ------------------------------------------------------------------ gradient
constexpr int kSortThreads = 1024;
constexpr int kSortPer = 4;
constexpr int kSortChunk = kSortThreads * kSortPer;
constexpr int kGradWindow = 32;                  // sorted tokens per window
constexpr int kGradThreads = 128;
constexpr int kGradCols = kGradThreads * 8;      // columns per CTA
constexpr int kZeroRows = 32;                    // table rows per zeroing CTA

// Step 1.  skey / sidx: [chunks][kSortChunk].
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const void* __restrict__ ids, int wide,
                                                                  int64_t T, int64_t V, int key_bits,
                                                                  uint32_t* __restrict__ skey,
                                                                  uint32_t* __restrict__ sidx) {
    __shared__ uint32_t key_s[kSortChunk];
    __shared__ uint16_t idx_s[kSortChunk];
    __shared__ int warp_zeros[32];
    grid_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t base = (int64_t)blockIdx.x * kSortChunk;
    uint32_t key[kSortPer];
    uint32_t idx[kSortPer];
    // element order: warp, then item, then lane
#pragma unroll
    for (int i = 0; i < kSortPer; ++i) {
        const int p = warp * 32 * kSortPer + i * 32 + lane;
        const int64_t t = base + p;
        key[i] = (uint32_t)V;
        idx[i] = (uint32_t)p;
        if (t < T) {
            const int64_t id = load_id(ids, wide, t);
            if (id >= 0 && id < V) key[i] = (uint32_t)id;
            else if (id >= V) report_error(kErrBadId);
        }
    }
    for (int b = 0; b < key_bits; ++b) {
        uint32_t ball[kSortPer];
        int zeros = 0;
#pragma unroll
        for (int i = 0; i < kSortPer; ++i) {
            ball[i] = __ballot_sync(0xffffffffu, ((key[i] >> b) & 1u) == 0u);
            zeros += __popc(ball[i]);
        }
        if (lane == 0) warp_zeros[warp] = zeros;
        __syncthreads();
        const int mine = warp_zeros[lane];
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const int total = __shfl_sync(0xffffffffu, incl, 31);
        int z = __shfl_sync(0xffffffffu, incl - mine, warp);       // zeros before this warp
        int ones = total + warp * 32 * kSortPer - z;               // ones go behind all zeros
        const uint32_t below = (1u << lane) - 1u;
#pragma unroll
        for (int i = 0; i < kSortPer; ++i) {
            const int zb = __popc(ball[i] & below);
            const int at = (ball[i] >> lane) & 1u ? z + zb : ones + lane - zb;
            key_s[at] = key[i];
            idx_s[at] = (uint16_t)idx[i];
            z += __popc(ball[i]);
            ones += 32 - __popc(ball[i]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSortPer; ++i) {
            const int p = warp * 32 * kSortPer + i * 32 + lane;
            key[i] = key_s[p];
            idx[i] = idx_s[p];
        }
    }
#pragma unroll
    for (int i = 0; i < kSortPer; ++i) {
        const int64_t p = base + warp * 32 * kSortPer + i * 32 + lane;
        skey[p] = key[i];
        sidx[p] = (uint32_t)(base + idx[i]);
    }
}

// A load of what the previous grid wrote (after the dependency wait): not through the
// read-only path.
__device__ __forceinline__ uint32_t ld_u32(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// First place in key[0, n) not below v.
__device__ __forceinline__ int64_t lower_bound_u32(const uint32_t* key, int64_t n, uint32_t v) {
    int64_t lo = 0;
    while (n > 0) {
        const int64_t half = n >> 1;
        if (ld_u32(key + lo + half) < v) {
            lo += half + 1;
            n -= half + 1;
        } else {
            n = half;
        }
    }
    return lo;
}

// Step 2.  `lanes` threads (a power of two up to 32) per element, each searching chunks
// lane, lane + lanes, ...: equal ids of earlier chunks come first.
__global__ void __launch_bounds__(256) embed_rank_kernel(const uint32_t* __restrict__ skey,
                                                         const uint32_t* __restrict__ sidx, int chunks,
                                                         int lanes, uint32_t* __restrict__ key,
                                                         uint32_t* __restrict__ idx) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t total = (int64_t)chunks * kSortChunk;
    const int64_t e = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / lanes;
    if (e >= total) return;                                  // whole groups of `lanes` leave together
    const int sub = threadIdx.x % lanes;
    const int own = (int)(e / kSortChunk);
    const uint32_t k = ld_u32(skey + e);
    int64_t rank = 0;
    for (int c = sub; c < chunks; c += lanes)
        if (c != own)
            rank += lower_bound_u32(skey + (int64_t)c * kSortChunk, kSortChunk, c < own ? k + 1u : k);
    const uint32_t group = lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1u) << ((threadIdx.x & 31) / lanes * lanes);
    for (int o = lanes >> 1; o > 0; o >>= 1) rank += __shfl_xor_sync(group, rank, o);
    if (sub == 0) {
        rank += e - (int64_t)own * kSortChunk;
        key[rank] = k;
        idx[rank] = ld_u32(sidx + e);
    }
}

template <bool F32>
__device__ __forceinline__ void grad_write(void* dW, int64_t at, const float v[8], float scale) {
    if constexpr (F32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(dW) + at);
        o[0] = make_float4(v[0] * scale, v[1] * scale, v[2] * scale, v[3] * scale);
        o[1] = make_float4(v[4] * scale, v[5] * scale, v[6] * scale, v[7] * scale);
    } else {
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p[i]) : "f"(v[2 * i + 1] * scale), "f"(v[2 * i] * scale));
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dW) + at) = make_uint4(p[0], p[1], p[2], p[3]);
    }
}

// Step 3.  CTAs [0, windows·slices) sum windows, the rest zero the rows that no token
// names.  part: [windows][2][K] binary32 (slot 0: a run that began before the window,
// slot 1: a run that goes on behind it).
template <bool F32>
__global__ void __launch_bounds__(kGradThreads) embed_grad_kernel(const uint16_t* __restrict__ dY,
                                                                  const uint32_t* __restrict__ key,
                                                                  const uint32_t* __restrict__ idx,
                                                                  int64_t padded, int windows, int slices,
                                                                  int64_t V, int K, float scale,
                                                                  void* __restrict__ dW,
                                                                  float* __restrict__ part) {
    __shared__ uint32_t ks[kGradWindow + 2];
    __shared__ uint32_t is[kGradWindow];
    __shared__ uint32_t present;
    grid_launch_dependents();
    grid_dependency_wait();
    const int tid = threadIdx.x;
    if ((int64_t)blockIdx.x < (int64_t)windows * slices) {
        const int w = (int)(blockIdx.x / slices), slice = (int)(blockIdx.x % slices);
        const int64_t p0 = (int64_t)w * kGradWindow;
        if (tid < kGradWindow + 2) {
            const int64_t p = p0 + tid - 1;
            ks[tid] = p >= 0 && p < padded ? ld_u32(key + p) : 0xffffffffu;
        }
        if (tid < kGradWindow) is[tid] = ld_u32(idx + p0 + tid);
        __syncthreads();
        const int col = slice * kGradCols + tid * 8;
        if (col >= K) return;
        float acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
        bool began = ks[0] == ks[1];                 // the first run began in an earlier window
#pragma unroll 1
        for (int j0 = 0; j0 < kGradWindow; j0 += 8) {
            uint4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = (int64_t)ks[1 + j0 + j] < V ? ldg_stream(dY + (int64_t)is[j0 + j] * K + col)
                                                   : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t k = ks[1 + j0 + j];
                if ((int64_t)k >= V) return;         // only dropped ids from here on
                const uint32_t q[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[2 * i] += __uint_as_float(q[i] << 16);
                    acc[2 * i + 1] += __uint_as_float(q[i] & 0xFFFF0000u);
                }
                const bool last = j0 + j == kGradWindow - 1;
                const bool on = ks[2 + j0 + j] == k;         // the run goes on behind this token
                if (on && !last) continue;
                if (began || on) {
                    float* o = part + ((int64_t)w * 2 + (began ? 0 : 1)) * K + col;
                    *reinterpret_cast<float4*>(o) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    *reinterpret_cast<float4*>(o + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
                } else {
                    grad_write<F32>(dW, (int64_t)k * K + col, acc, scale);
                }
                began = false;
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
            }
        }
        return;
    }
    // zeroing: a mask of the rows that tokens name, from the sorted list
    const int64_t v0 = ((int64_t)blockIdx.x - (int64_t)windows * slices) * kZeroRows;
    const int rows = (int)(V - v0 < kZeroRows ? V - v0 : kZeroRows);
    if (tid == 0) present = 0u;
    __syncthreads();
    if (tid < rows) {
        const int64_t p = lower_bound_u32(key, padded, (uint32_t)(v0 + tid));
        if (p < padded && ld_u32(key + p) == (uint32_t)(v0 + tid)) atomicOr(&present, 1u << tid);
    }
    __syncthreads();
    const uint32_t mask = present;
    const int row16 = K * (F32 ? 4 : 2) / 16;                   // K is a multiple of 8
    uint4* o = static_cast<uint4*>(dW) + v0 * row16;
    for (int r = 0; r < rows; ++r) {
        if ((mask >> r) & 1u) continue;
        for (int c = tid; c < row16; c += kGradThreads) o[(int64_t)r * row16 + c] = make_uint4(0, 0, 0, 0);
    }
}

// Step 4.  One CTA per window whose last run goes on behind it and begins in it.
template <bool F32>
__global__ void __launch_bounds__(kGradThreads) embed_grad_join_kernel(const uint32_t* __restrict__ key,
                                                                       int64_t padded, int windows, int64_t V,
                                                                       int K, float scale,
                                                                       void* __restrict__ dW,
                                                                       const float* __restrict__ part) {
    grid_dependency_wait();
    const int w = (int)blockIdx.x;
    const int64_t end = (int64_t)(w + 1) * kGradWindow;         // first place behind the window
    if (end >= padded) return;
    const uint32_t k = ld_u32(key + end - 1);
    if ((int64_t)k >= V || ld_u32(key + end) != k) return;               // no run crosses this border
    // the window holds the run's beginning, unless the run fills it and began before
    if (w > 0 && ld_u32(key + end - kGradWindow) == k && ld_u32(key + end - kGradWindow - 1) == k) return;
    const int col = (int)blockIdx.y * kGradCols + threadIdx.x * 8;
    if (col >= K) return;
    // windows w + 1 .. w1 begin inside the run
    const int64_t last = lower_bound_u32(key + end, padded - end, k + 1u) + end - 1;
    const int w1 = (int)(last / kGradWindow);
    float acc[8];
    const float* p = part + ((int64_t)w * 2 + 1) * K + col;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = __ldcg(p + i);
    for (int j = w + 1; j <= w1; ++j) {
        const float4 a = __ldcg(reinterpret_cast<const float4*>(part + (int64_t)j * 2 * K + col));
        const float4 b = __ldcg(reinterpret_cast<const float4*>(part + (int64_t)j * 2 * K + col + 4));
        acc[0] += a.x; acc[1] += a.y; acc[2] += a.z; acc[3] += a.w;
        acc[4] += b.x; acc[5] += b.y; acc[6] += b.z; acc[7] += b.w;
    }
    grad_write<F32>(dW, (int64_t)k * K + col, acc, scale);
}

}  // namespace w4a16
