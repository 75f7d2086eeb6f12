// Quantized embedding: table lookup, and the gradient of the dense table behind it.
//
// Lookup:  out[t, :] = bf16_rn(scale·Ŵ[id_t, :]),  Ŵ = bf16_rn((q − z)·s)
// A row is gathered as codes (0.53 bytes per weight with 4 bits), dequantized in
// registers and written once: bound by writing the bf16 rows.  One thread per 8 codes, so
// a warp reads 128 (256) contiguous code bytes and writes 512 contiguous bytes (8192 ids,
// K = 8192, 8 bits: 36 to 39 us, 5.2 to 5.7 TB/s).
//
// Gradient:  dW[v, :] = scale·Σ_{t: id_t = v} dY[t, :], summed in binary32 in ascending t
// within windows of 32 or 64 sorted tokens (by T alone), windows added in order: the same inputs
// give the same bits.  Four steps, no atomics on values:
//   1. chunks of ids are sorted by (id, t) in shared memory, one CTA per chunk: stable radix
//      passes of five bits (the 32 digits are a warp's lanes, so counts live in registers);
//   2. with more than one chunk, each element's place among the other chunks is found by
//      binary search: its rank in the whole sorted list;
//   3. windows of 32 or 64 sorted tokens are summed, one thread per 8 columns; runs of one
//      id inside a window are written at once, runs that cross its border leave a
//      binary32 part;
//   4. parts of a run are added in window order and written.
// Most of the time goes to writing zeros into the rows that no token names.  Step 3 writes
// most of them (it finds them in the sorted list); the first 30 MB are written beside the
// sort, which leaves the machine idle (by CTAs that look through the ids themselves), the
// last sixteenth beside step 4.  Table of 32000 rows, K = 4096: 2048 ids, bf16 56 us; 16384 ids,
// binary32 127 us: 5.0 and 5.2 TB/s.
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
constexpr int kGradWindow = 64;                  // sorted tokens per window, at most
constexpr int kGradThreads = 128;
constexpr int kGradCols = kGradThreads * 8;      // columns per CTA
constexpr int kZeroRows = 8;                     // table rows per zeroing CTA

// Step 1.  PER ids per thread; W holds id << IB | place in the chunk (IB bits), so one word
// moves per pass.  skey / sidx: [chunks][THREADS·PER].  CTAs behind the chunks' zero rows
// [0, zero_end), `zero_rows_per` each.
template <typename W, int THREADS, int PER>
struct SortConfig {
    static constexpr int kChunk = THREADS * PER;
    static constexpr int kWarps = THREADS / 32;
    static constexpr int kIndexBits = kChunk == 1024 ? 10 : 14;
    static_assert(kChunk <= 1 << kIndexBits && THREADS % 32 == 0 && THREADS <= 1024, "chunk");
    static constexpr int kSmem = kChunk * (int)sizeof(W) + 32 * 33 * 4 + 32 * 4;
};

template <bool F32, int THREADS>
__device__ __forceinline__ void zero_rows_by_ids(const void* ids, int wide, int64_t T, int64_t v0, int64_t v1, int K,
                                                 void* __restrict__ dW, uint32_t* mask, int mask_words) {
    for (int i = threadIdx.x; i < mask_words; i += THREADS) mask[i] = 0u;
    __syncthreads();
    for (int64_t t0 = threadIdx.x; t0 < T; t0 += 8 * THREADS) {
        int64_t id[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) id[j] = t0 + j * THREADS < T ? load_id(ids, wide, t0 + j * THREADS) : -1;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (id[j] >= v0 && id[j] < v1) atomicOr(&mask[(id[j] - v0) >> 5], 1u << ((id[j] - v0) & 31));
    }
    __syncthreads();
    const int row16 = K / (F32 ? 4 : 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t v = v0 + warp; v < v1; v += THREADS / 32) {
        if ((mask[(v - v0) >> 5] >> ((v - v0) & 31)) & 1u) continue;
        uint4* o = static_cast<uint4*>(dW) + v * row16;
        for (int c = lane; c < row16; c += 32) o[c] = make_uint4(0, 0, 0, 0);
    }
}

template <typename W, int THREADS, int PER, bool F32>
__global__ void __launch_bounds__(THREADS) embed_sort_kernel(const void* __restrict__ ids, int wide, int64_t T,
                                                             int64_t V, int key_bits, uint32_t* __restrict__ skey,
                                                             uint32_t* __restrict__ sidx, int chunks,
                                                             int64_t zero_end, int zero_rows_per, int K,
                                                             void* __restrict__ dW) {
    using Cfg = SortConfig<W, THREADS, PER>;
    constexpr int IB = Cfg::kIndexBits;
    extern __shared__ __align__(16) uint8_t sort_smem[];
    W* word_s = reinterpret_cast<W*>(sort_smem);
    int* hist = reinterpret_cast<int*>(sort_smem + Cfg::kChunk * sizeof(W));      // [digit][33] by warp
    int* total = hist + 32 * 33;
    if ((int)blockIdx.x >= chunks) {
        const int64_t v0 = (int64_t)((int)blockIdx.x - chunks) * zero_rows_per;
        const int64_t v1 = v0 + zero_rows_per < zero_end ? v0 + zero_rows_per : zero_end;
        zero_rows_by_ids<F32, THREADS>(ids, wide, T, v0, v1, K, dW, reinterpret_cast<uint32_t*>(sort_smem),
                                       (zero_rows_per + 31) / 32);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t base = (int64_t)blockIdx.x * Cfg::kChunk;
    const uint32_t below = (1u << lane) - 1u;
    W word[PER];
    // element order: warp, then item, then lane
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int p = warp * 32 * PER + i * 32 + lane;
        const int64_t t = base + p;
        W key = (W)V;
        if (t < T) {
            const int64_t id = load_id(ids, wide, t);
            if (id >= 0 && id < V) key = (W)id;
            else if (id >= V) report_error(kErrBadId);
        }
        word[i] = key << IB | (W)p;
    }
    for (int b = 0; b < key_bits; b += 5) {
        // this warp's elements of each digit (counted by the lane of that number), and each
        // element's rank among them
        int count = 0;
        uint32_t rank[PER / 2];                  // two 16-bit ranks a word
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t d = (uint32_t)(word[i] >> (IB + b)) & 31u;
            uint32_t mine = 0xffffffffu, counted = 0xffffffffu;
#pragma unroll
            for (int k = 0; k < 5; ++k) {
                const uint32_t v = __ballot_sync(0xffffffffu, (d >> k) & 1u);
                mine &= (d >> k) & 1u ? v : ~v;
                counted &= (lane >> k) & 1 ? v : ~v;
            }
            const uint32_t r = (uint32_t)(__shfl_sync(0xffffffffu, count, d) + __popc(mine & below));
            if (i & 1) rank[i >> 1] |= r << 16;
            else rank[i >> 1] = r;
            count += __popc(counted);
        }
        hist[lane * 33 + warp] = count;
        __syncthreads();
        // a warp per digit: its elements in the warps before each warp
        for (int d = warp; d < 32; d += Cfg::kWarps) {
            const int c = lane < Cfg::kWarps ? hist[d * 33 + lane] : 0;
            int incl = c;
#pragma unroll
            for (int o = 1; o < Cfg::kWarps; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (lane < Cfg::kWarps) hist[d * 33 + lane] = incl - c;
            if (lane == Cfg::kWarps - 1) total[d] = incl;
        }
        __syncthreads();
        const int tot = total[lane];
        int dincl = tot;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, dincl, o);
            if (lane >= o) dincl += v;
        }
        const int start = dincl - tot + hist[lane * 33 + warp];      // of digit `lane`, this warp
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t d = (uint32_t)(word[i] >> (IB + b)) & 31u;
            const int at = __shfl_sync(0xffffffffu, start, d) + (int)((rank[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
            word_s[at] = word[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; ++i) word[i] = word_s[warp * 32 * PER + i * 32 + lane];
        // (the next pass writes word_s only after its first barrier, behind these reads)
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int64_t p = base + warp * 32 * PER + i * 32 + lane;
        skey[p] = (uint32_t)(word[i] >> IB);
        sidx[p] = (uint32_t)(base + (int64_t)(word[i] & (W)((1 << IB) - 1)));
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

// Step 2.  An element's rank is its place in its chunk plus, for every other chunk, the number
// of smaller ids there (of ids not larger, in the chunks before its own: equal ids keep
// their order).  SHARED: all chunks' keys are brought into shared memory first, four threads per
// element; else `lanes` threads (a power of two up to 32) per element search in L2.
constexpr int kRankThreads = 512;
constexpr int kRankPer = 4;                     // threads per element of the shared form
constexpr int64_t kRankShared = 16384;          // ids, at most, for the shared form

template <bool SHARED>
__global__ void __launch_bounds__(kRankThreads) embed_rank_kernel(const uint32_t* __restrict__ skey,
                                                                  const uint32_t* __restrict__ sidx, int chunks,
                                                                  int chunk, int lanes, uint32_t* __restrict__ key,
                                                                  uint32_t* __restrict__ idx) {
    extern __shared__ __align__(16) uint32_t rank_smem[];
    grid_dependency_wait();
    const int64_t total = (int64_t)chunks * chunk;
    if constexpr (SHARED) {
#pragma unroll 8
        for (int i = threadIdx.x; i < (int)total / 4; i += kRankThreads)
            reinterpret_cast<uint4*>(rank_smem)[i] = __ldcg(reinterpret_cast<const uint4*>(skey) + i);
        __syncthreads();
        const int e = (int)blockIdx.x * (kRankThreads / kRankPer) + threadIdx.x / kRankPer;   // < total: see the launch
        const int sub = threadIdx.x % kRankPer;
        const uint32_t k = rank_smem[e];
        const int own = e / chunk;
        int rank = 0;
        for (int c = sub; c < chunks; c += kRankPer) {
            if (c == own) continue;
            const uint32_t v = c < own ? k + 1u : k;
            const uint32_t* p = rank_smem + c * chunk;
            int lo = 0;                              // chunk is a power of two
            for (int half = chunk >> 1; half > 0; half >>= 1)
                if (p[lo + half - 1] < v) lo += half;
            rank += lo + (p[lo] < v ? 1 : 0);
        }
#pragma unroll
        for (int o = kRankPer >> 1; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
        if (sub == 0) {
            rank += e - own * chunk;
            key[rank] = k;
            idx[rank] = ld_u32(sidx + e);
        }
    } else {
        const int64_t e = ((int64_t)blockIdx.x * kRankThreads + threadIdx.x) / lanes;
        if (e >= total) return;                                  // whole groups of `lanes` leave together
        const int sub = threadIdx.x % lanes;
        const int own = (int)(e / chunk);
        const uint32_t k = ld_u32(skey + e);
        int64_t rank = 0;
        for (int c = sub; c < chunks; c += lanes)
            if (c != own) rank += lower_bound_u32(skey + (int64_t)c * chunk, chunk, c < own ? k + 1u : k);
        const uint32_t group =
            lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1u) << ((threadIdx.x & 31) / lanes * lanes);
        for (int o = lanes >> 1; o > 0; o >>= 1) rank += __shfl_xor_sync(group, rank, o);
        if (sub == 0) {
            rank += e - (int64_t)own * chunk;
            key[rank] = k;
            idx[rank] = ld_u32(sidx + e);
        }
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

// lower_bound_u32 by a warp: 32 probes a step instead of one.
__device__ __forceinline__ int64_t lower_bound_warp(const uint32_t* key, int64_t n, uint32_t v) {
    const int lane = threadIdx.x & 31;
    int64_t lo = 0;
    while (n > 0) {
        // probes divide the range into 33 parts (into single elements when it is short)
        const int64_t step = n / 33 + 1;
        const int64_t p = (lane + 1) * step - 1;
        const int less = __popc(__ballot_sync(0xffffffffu, p < n && ld_u32(key + lo + p) < v));
        // the first `less` probes are below v: the bound lies behind probe less − 1 and not
        // behind probe `less`
        const int64_t from = less * step, to = (less + 1) * step - 1;
        lo += from;
        n = (to < n ? to : n) - from;
    }
    return lo;
}

// Sets the rows v0 .. v0 + kZeroRows - 1 of the table that no token names to zero.
template <bool F32>
__device__ __forceinline__ void zero_rows(const uint32_t* key, int64_t padded, int64_t v0, int64_t V, int K,
                                          void* __restrict__ dW, uint32_t* present) {
    const int tid = threadIdx.x;
    const int rows = (int)(V - v0 < kZeroRows ? V - v0 : kZeroRows);
    if (tid < 32) {
        const int64_t lo = lower_bound_warp(key, padded, (uint32_t)v0);
        uint32_t mask = 0u;
        // most often the next 32 keys reach behind the rows; a long run is searched past
        if (tid < rows) {
            const uint32_t v = (uint32_t)(v0 + tid);
            int64_t p = lo;
            for (int j = 0; j < 32 && p < padded && ld_u32(key + p) < v; ++j) ++p;
            if (p < padded && ld_u32(key + p) < v) p += lower_bound_u32(key + p, padded - p, v);
            if (p < padded && ld_u32(key + p) == v) mask = 1u << tid;
        }
        mask = __reduce_or_sync(0xffffffffu, mask);
        if (tid == 0) *present = mask;
    }
    __syncthreads();
    const uint32_t mask = *present;
    const int row16 = K / (F32 ? 4 : 8);                        // K is a multiple of 32
    uint4* o = static_cast<uint4*>(dW) + v0 * row16;
    for (int r = 0; r < rows; ++r) {
        if ((mask >> r) & 1u) continue;
        for (int c = tid; c < row16; c += kGradThreads) o[(int64_t)r * row16 + c] = make_uint4(0, 0, 0, 0);
    }
}

// Step 3.  CTAs [0, windows·slices) sum windows, the rest zero rows [zero_begin, zero_end).  part:
// [windows][2][K] binary32 (slot 0: a run that began before the window, slot 1: a run that
// goes on behind it).
template <bool F32>
__global__ void __launch_bounds__(kGradThreads) embed_grad_kernel(const uint16_t* __restrict__ dY,
                                                                  const uint32_t* __restrict__ key,
                                                                  const uint32_t* __restrict__ idx,
                                                                  int64_t padded, int window, int windows, int slices,
                                                                  int64_t V, int64_t zero_begin,
                                                                  int64_t zero_end, int K,
                                                                  float scale, void* __restrict__ dW,
                                                                  float* __restrict__ part) {
    __shared__ uint32_t ks[kGradWindow + 2];
    __shared__ uint32_t is[kGradWindow];
    __shared__ uint32_t present;
    grid_dependency_wait();
    const int tid = threadIdx.x;
    if ((int64_t)blockIdx.x < (int64_t)windows * slices) {
        const int w = (int)(blockIdx.x / slices), slice = (int)(blockIdx.x % slices);
        const int64_t p0 = (int64_t)w * window;
        if (tid < window + 2) {
            const int64_t p = p0 + tid - 1;
            ks[tid] = p >= 0 && p < padded ? ld_u32(key + p) : 0xffffffffu;
        }
        if (tid < window) is[tid] = ld_u32(idx + p0 + tid);
        __syncthreads();
        const int col = slice * kGradCols + tid * 8;
        if (col >= K) return;
        float acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
        bool began = ks[0] == ks[1];                 // the first run began in an earlier window
#pragma unroll 1
        for (int j0 = 0; j0 < window; j0 += 8) {
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
                const bool last = j0 + j == window - 1;
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
    zero_rows<F32>(key, padded, zero_begin + ((int64_t)blockIdx.x - (int64_t)windows * slices) * kZeroRows, zero_end, K, dW,
                   &present);
}

// Step 4.  One CTA per window and slice, at work when the window's last run begins in it and
// goes on behind it; the CTAs behind them zero rows [zero_begin, V).
template <bool F32>
__global__ void __launch_bounds__(kGradThreads) embed_grad_join_kernel(const uint32_t* __restrict__ key,
                                                                       int64_t padded, int window, int windows, int slices,
                                                                       int64_t V, int64_t zero_begin, int K,
                                                                       float scale, void* __restrict__ dW,
                                                                       const float* __restrict__ part) {
    __shared__ uint32_t present;
    grid_dependency_wait();
    if ((int64_t)blockIdx.x >= (int64_t)windows * slices) {
        zero_rows<F32>(key, padded, zero_begin + ((int64_t)blockIdx.x - (int64_t)windows * slices) * kZeroRows, V, K, dW,
                       &present);
        return;
    }
    const int w = (int)(blockIdx.x / slices);
    const int64_t end = (int64_t)(w + 1) * window;         // first place behind the window
    if (end >= padded) return;
    const uint32_t k = ld_u32(key + end - 1), behind = ld_u32(key + end), first = ld_u32(key + end - window);
    const uint32_t before = w > 0 ? ld_u32(key + end - window - 1) : 0xffffffffu;
    // no run crosses this border, or the run fills the window and began before it
    if ((int64_t)k >= V || behind != k || (first == k && before == k)) return;
    // windows w + 1 .. w1 begin inside the run: a warp looks at the first keys of 32 windows
    int w1 = w;
    for (int j0 = w + 1;; j0 += 32) {
        const int64_t p = (int64_t)(j0 + (threadIdx.x & 31)) * window;
        const uint32_t on = __ballot_sync(0xffffffffu, p < padded && ld_u32(key + p) == k);
        const int run = __ffs(~on) - 1;                       // -1: all 32
        w1 = j0 + (run < 0 ? 32 : run) - 1;
        if (run >= 0) break;
    }
    const int col = (int)(blockIdx.x % slices) * kGradCols + threadIdx.x * 8;
    if (col >= K) return;
    float acc[8];
    const float* p = part + ((int64_t)w * 2 + 1) * K + col;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = __ldcg(p + i);
    for (int j0 = w + 1; j0 <= w1; j0 += 8) {
        // eight windows' loads in flight, then their sums in order
        float4 a[8], b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float* q = part + (int64_t)min(j0 + j, w1) * 2 * K + col;
            a[j] = __ldcg(reinterpret_cast<const float4*>(q));
            b[j] = __ldcg(reinterpret_cast<const float4*>(q + 4));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j0 + j > w1) break;
            acc[0] += a[j].x; acc[1] += a[j].y; acc[2] += a[j].z; acc[3] += a[j].w;
            acc[4] += b[j].x; acc[5] += b[j].y; acc[6] += b[j].z; acc[7] += b[j].w;
        }
    }
    grad_write<F32>(dW, (int64_t)k * K + col, acc, scale);
}

}  // namespace w4a16
