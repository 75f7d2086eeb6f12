// Host-side helpers shared by the library's translation units: device queries,
// argument checks, tensor-map encoding and the decode kernel's launch geometry.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>
#include <mutex>

#include "../../include/w4a16.h"
#include "gemv_decode.cuh"

namespace w4a16 {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

struct DeviceInfo {
    bool ready = false;
    int sm_count = 0;
    int cc_major = 0;
    int cc_minor = 0;
};

inline std::mutex g_mutex;
inline DeviceInfo g_devices[kMaxDevices];
inline PFN_cuTensorMapEncodeTiled_v12000 g_encode_tiled = nullptr;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Group sizes along K with kernels of their own.
inline bool grouped(int32_t g) { return g == 32 || g == 64 || g == 128; }

// Per-channel granularity: one group spanning the whole row (g == K), one scale
// and zero point per output feature ("量化实战深入（GPTQ / AWQ / SmoothQuant / KV 量化）", 量化粒度 table;
// "推理优化中“用精度换性能“的核心技术：量化", §3.4).
// Kernels take it as group size 0.
inline bool per_channel(int32_t g, int64_t K) { return !grouped(g) && (int64_t)g == K; }

// g is one of the grouped sizes with K a multiple of it, or g == K with K a
// multiple of 32 (packed rows of whole 16-byte chunks, as TMA needs).
inline bool valid_group(int32_t g, int64_t K) {
    if (grouped(g)) return K % g == 0;
    return per_channel(g, K) && K % 32 == 0;
}

inline w4a16_status device_info(DeviceInfo* out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return W4A16_ECUDA;
    std::lock_guard<std::mutex> lock(g_mutex);
    DeviceInfo& d = g_devices[dev];
    if (!d.ready) {
        if (cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&d.cc_major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&d.cc_minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
            return W4A16_ECUDA;
        d.ready = true;
    }
    *out = d;
    if (d.cc_major != 10 || d.cc_minor != 0) return W4A16_EUNSUPPORTED;   // built for sm_100a only
    return W4A16_OK;
}

inline w4a16_status encoder(PFN_cuTensorMapEncodeTiled_v12000* fn) {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (g_encode_tiled == nullptr) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess || p == nullptr)
            return W4A16_ECUDA;
        g_encode_tiled = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
    *fn = g_encode_tiled;
    return W4A16_OK;
}

// Value of the ready flags of one launch: another one for every launch of the process (the
// multiplication by an odd number is one to one), never 0, and like no data.
inline uint64_t launch_flag() {
    static std::atomic<uint64_t> launches{1};
    const uint64_t v = launches.fetch_add(1, std::memory_order_relaxed) * 0x9E3779B97F4A7C15ull;
    return v != 0 ? v : 1;
}

inline w4a16_status launch_status() {
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? W4A16_OK : W4A16_ECUDA;
}

// ---------------------------------------------------------------- plans
constexpr int kSmemPerBlockMax = 232448;  // opt-in maximum per CTA (227 KB)
constexpr int kMaxCtas = 65535;

// Decode kernel geometry for (M, N, K, g): 256-row x 256-K units, one CTA per
// SM with a ring of shared-memory stages and scale slabs filling its shared
// memory.
struct DecodeGeometry {
    int bits;          // code width, 4 or 8
    int mb;            // n8 MMA column blocks (1: M ≤ 8, 2: M ≤ 16)
    int rb;            // row blocks of 256 rows
    int kbn;           // K blocks of 256
    int64_t units;     // rb · kbn
    int gu;            // scale groups per row per unit (1 for per-channel)
    int sw;            // groups per staged scale row without TMA slabs (0 with them)
    int sz_tma;        // scales staged by TMA in 8-group slabs (rows 16-byte aligned)
    int slabs;         // slab ring slots (0 without TMA slabs)
    int slab_off;      // slab ring inside the dynamic shared memory
    int xf_off;        // fragment-ordered X inside a stage
    int sz_off;        // scales and zeros inside a stage
    int stage_bytes;   // multiple of 1024
    int stages;
    int ctas_per_sm;
    int smem_bytes;    // dynamic shared memory per CTA
};

// Outside the stages: zero fragments, barriers and flags (< 1024 bytes), plus
// slack to align the dynamic shared memory base to 1024 bytes.
constexpr int kDecFixedSmem = 1024 + 1024;

// Scale (and zero) groups of one row inside a 256-wide K block.
inline int decode_block_k(int bits) { return bits == 8 ? dec_block_k<8>() : dec_block_k<4>(); }
inline int decode_unit_groups(int32_t g, int64_t K, int bits) {
    return per_channel(g, K) ? 1 : decode_block_k(bits) / g;
}

// Stage: codes tile (16 KB, TMA, 128-byte swizzle) | X slice, natural order
// (M x 512 B, TMA) | X in fragment order (rows 576 B apart, the last one 512 B;
// 128-byte aligned) | without TMA slabs, scales and zeros (2 x 256 rows x gu bf16).
inline DecodeGeometry decode_geometry(int64_t M, int64_t N, int64_t K, int g, int bits = 4) {
    DecodeGeometry d{};
    d.bits = bits;
    d.mb = M <= 8 ? 1 : 2;
    d.rb = (int)((N + kDecRows - 1) / kDecRows);
    const int bk = decode_block_k(bits);
    const int xrb = bk * 2, xfrb = bk * 2 + 64;   // X rows: natural, fragment order (padded)
    d.kbn = (int)((K + bk - 1) / bk);
    d.units = (int64_t)d.rb * d.kbn;
    d.gu = decode_unit_groups(g, K, bits);
    d.sz_tma = (!per_channel(g, K) && (K / g) % 8 == 0) ? 1 : 0;
    const int m = M < 1 ? 1 : (int)M;
    const int xnat_end = kDecPBytes + m * xrb;
    d.xf_off = (xnat_end + 127) / 128 * 128;
    const int xf_end = d.xf_off + (m - 1) * xfrb + xrb;
    d.sz_off = (xf_end + 127) / 128 * 128;      // TMA destinations are 128-byte aligned
    // Scales in the stage only without TMA slabs; with them, a ring of slab slots.
    // A unit with a single group whose rows hold an even number of groups stages
    // the 4-byte aligned pair around it (the copy mode decode_scale_copy picks).
    const bool pairs = !d.sz_tma && !per_channel(g, K) && d.gu == 1 && (K / g) % 2 == 0;
    d.sw = d.sz_tma ? 0 : (pairs ? 2 : d.gu);
    const int stage_raw = d.sz_off + 2 * kDecRows * d.sw * 2;
    d.stage_bytes = (stage_raw + 1023) / 1024 * 1024;
    // Slab slots: one the consumers read, plus enough for the units the producer
    // may run ahead (the ring depth) at 8/gu units per slab, plus one for a slab
    // boundary in between; at least 2, at most one per stage plus one.
    const int ups = d.sz_tma ? 8 / d.gu : 1;
    auto slabs_for = [&](int stages) {
        if (!d.sz_tma) return 0;
        int sl = (stages + 1 + ups - 1) / ups + 1;
        if (sl > stages + 1) sl = stages + 1;
        if (sl < 2) sl = 2;
        if (sl > kDecMaxSlabs) sl = kDecMaxSlabs;
        return sl;
    };
    auto fits = [&](int stages, int budget) {
        return stages * d.stage_bytes + slabs_for(stages) * kDecSlabBytes <= budget;
    };
    // One CTA per SM (16 consumer warps; two such CTAs would not fit the registers).
    int one = 0;
    while (one < kDecMaxStages && fits(one + 1, kSmemPerBlockMax - kDecFixedSmem)) ++one;
    d.ctas_per_sm = 1;
    d.stages = one;
    d.slabs = slabs_for(d.stages);
    d.slab_off = d.stages * d.stage_bytes;
    d.smem_bytes = d.slab_off + d.slabs * kDecSlabBytes + kDecFixedSmem;
    return d;
}

// The stage layout's invariants: every TMA destination (codes, X, scale and zero
// slabs) 128-byte aligned, the codes tile 1024-byte aligned (128-byte swizzle),
// the fragment-ordered X 128-byte aligned (bank spread of the consumers' loads),
// and the ring within the shared memory of one CTA.
inline bool decode_geometry_ok(const DecodeGeometry& d, int64_t M) {
    const int m = M < 1 ? 1 : (int)M;
    const int sw = d.sw;                       // scales in the stage only without slabs
    const int xrb = decode_block_k(d.bits) * 2, xfrb = xrb + 64;
    return (d.bits == 4 || d.bits == 8) && d.stage_bytes % 1024 == 0 && kDecPBytes % 128 == 0 &&
           d.xf_off % 128 == 0 && d.xf_off >= kDecPBytes + m * xrb && d.sz_off % 128 == 0 &&
           d.sz_off >= d.xf_off + (m - 1) * xfrb + xrb &&
           (kDecRows * sw * 2) % 128 == 0 && d.sz_off + 2 * kDecRows * sw * 2 <= d.stage_bytes &&
           d.stages >= 2 && d.stages <= kDecMaxStages && d.slab_off % 1024 == 0 &&
           (d.sz_tma ? d.slabs >= 2 && d.slabs <= kDecMaxSlabs : d.slabs == 0) &&
           kDecSlabBytes % 1024 == 0 && d.smem_bytes <= kSmemPerBlockMax;
}

// Workspace of a decode launch with `ctas` CTAs: (rb + ctas) slots, slot rb + c
// holding CTA c's part of a row block that the stream-K partition splits —
// per slot 16 ready flags (DecodeFlag), then 16 warps x 32 lanes x 4·mb fp32 partial sums.
// Scratch: no initialization is needed (a flag counts only when it holds the
// ready pattern, which the consuming CTA clears again).
template <typename Flag = uint32_t>
inline int64_t decode_flag_bytes(const DecodeGeometry& d, int64_t ctas) {
    return ((int64_t)(d.rb + ctas) * kDecConsumers * (int64_t)sizeof(Flag) + 255) / 256 * 256;
}

template <typename Flag = uint32_t>
inline int64_t decode_workspace_bytes(const DecodeGeometry& d, int64_t ctas) {
    return decode_flag_bytes<Flag>(d, ctas) + (int64_t)(d.rb + ctas) * kDecConsumers * 32 * 16 * d.mb;
}

// Row blocks the even unit split cuts between CTAs.
inline int64_t decode_split_blocks(const DecodeGeometry& d, int64_t ctas) {
    int64_t n = 0, last = -1;
    for (int64_t b = 1; b < ctas; ++b) {
        const int64_t u = b * d.units / ctas;
        if (u % d.kbn != 0 && u / d.kbn != last) {
            ++n;
            last = u / d.kbn;
        }
    }
    return n;
}

inline w4a16_status check_shape(int64_t M, int64_t N, int64_t K, int32_t g, int32_t sym) {
    if (sym != 0 && sym != 1) return W4A16_EINVAL;
    if (M < 0 || N < 0 || K <= 0) return W4A16_EINVAL;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return W4A16_EINVAL;
    if (!valid_group(g, K)) return W4A16_EINVAL;
    return W4A16_OK;
}

// SM count of the current device, queried once per device (148 when no device
// can be queried, e.g. for host-only planning on a machine without a GPU).
inline int current_sm_count() {
    static std::atomic<int> cached[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return 148;
    }
    int sms = cached[dev].load(std::memory_order_relaxed);
    if (sms > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
        cudaGetLastError();
        return 148;
    }
    cached[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

// Tensor maps are encoded on the host for every launch; a call repeated with
// the same buffers (the common case: fixed weights, reused activation and output
// buffers) finds its maps in this per-thread cache instead of re-encoding them.
struct TmKey {
    const void* base;
    uint64_t inner, outer, row_bytes;
    uint32_t box_inner, box_outer;
    int dtype, swizzle;
    bool operator==(const TmKey& o) const {
        return base == o.base && inner == o.inner && outer == o.outer && row_bytes == o.row_bytes &&
               box_inner == o.box_inner && box_outer == o.box_outer && dtype == o.dtype &&
               swizzle == o.swizzle;
    }
};

struct TmEntry {
    bool valid;
    TmKey key;
    CUtensorMap map;
};

constexpr int kTmCacheSize = 256;

inline size_t tm_hash(const TmKey& k) {
    uint64_t h = reinterpret_cast<uintptr_t>(k.base) * 0x9E3779B97F4A7C15ull;
    for (uint64_t v : {k.inner, k.outer, k.row_bytes, (uint64_t)k.box_inner, (uint64_t)k.box_outer,
                       (uint64_t)k.dtype, (uint64_t)k.swizzle})
        h = (h ^ v) * 0x100000001B3ull;
    return (size_t)(h >> 17) % kTmCacheSize;
}

inline w4a16_status encode_2d(CUtensorMap* map, CUtensorMapDataType dtype, const void* base,
                       uint64_t inner, uint64_t outer, uint64_t row_bytes, uint32_t box_inner,
                       uint32_t box_outer, CUtensorMapSwizzle swizzle) {
    thread_local TmEntry cache[kTmCacheSize];
    const TmKey key{base, inner, outer, row_bytes, box_inner, box_outer, (int)dtype, (int)swizzle};
    TmEntry& e = cache[tm_hash(key)];
    if (e.valid && e.key == key) {
        *map = e.map;
        return W4A16_OK;
    }
    PFN_cuTensorMapEncodeTiled_v12000 fn;
    w4a16_status st = encoder(&fn);
    if (st != W4A16_OK) return st;
    cuuint64_t dims[2] = {inner, outer};
    cuuint64_t strides[1] = {row_bytes};
    cuuint32_t box[2] = {box_inner, box_outer};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(map, dtype, 2, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return W4A16_ECUDA;
    e.valid = true;
    e.key = key;
    e.map = *map;
    return W4A16_OK;
}

// Bytes per scale copy for grouped scales: the largest of 16, 8, 4 that divides
// both a unit's scale bytes per row (gu·2) and the scale row stride (K/g·2), so
// that copies are aligned and never cross the end of a row; 2 = plain loads.
inline int decode_scale_copy(int gu, int64_t groups) {
    for (int cs = 16; cs >= 4; cs /= 2)
        if (cs <= gu * 2 && (gu * 2) % cs == 0 && (groups * 2) % cs == 0) return cs;
    // one group per unit (8-bit codes at g = 128): the aligned pair holding it
    if (gu == 1 && groups % 2 == 0) return 3;
    return 2;
}

inline int grid_for(int64_t work_items, int threads, int sm_count) {
    const int64_t blocks = (work_items + threads - 1) / threads;
    const int64_t cap = (int64_t)sm_count * 8;   // grid-stride loops beyond 8 CTAs per SM
    return (int)(blocks < cap ? (blocks < 1 ? 1 : blocks) : cap);
}

}  // namespace w4a16
