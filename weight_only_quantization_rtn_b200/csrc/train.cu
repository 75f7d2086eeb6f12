// C ABI of the operators around the quantized linear layer: the gated feed-forward block
// and its backward pass, the linear layer's gradients, the quantized embedding and its
// table's gradient.  The public contract is documented in include/w4a16.h.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "../../include/w4a16.h"
#include "embedding.cuh"
#include "gate_backward.cuh"
#include "gemm_pair.cuh"
#include "gemm_wgrad.cuh"
#include "gemv_decode.cuh"
#include "host.cuh"
#include "pair_plan.cuh"

using namespace w4a16;

namespace {

// Tensor map of a 2-D array of rows, encoded for this launch.
w4a16_status encode_rows(CUtensorMap* map, CUtensorMapDataType dtype, const void* base, uint64_t inner,
                         uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
                         CUtensorMapSwizzle swizzle) {
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
    return r == CUDA_SUCCESS ? W4A16_OK : W4A16_ECUDA;
}

// Ids are read one by one, so a list may begin at any of them.
bool aligned_to(const void* p, int32_t bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

bool valid_act(int32_t act) { return act >= W4A16_ACT_SILU && act <= W4A16_ACT_RELU; }

int64_t round8(int64_t n) { return (n + 7) / 8 * 8; }

int group_shift(int32_t g, int64_t K) {
    if (per_channel(g, K)) return 31;
    return g == 32 ? 5 : (g == 64 ? 6 : 7);
}

// Opt-in shared memory of a kernel, once per device.
template <typename F>
w4a16_status set_smem(F* kern, int bytes, bool (&done)[kMaxDevices]) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return W4A16_ECUDA;
    if (!done[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
            cudaGetLastError();
            return W4A16_ECUDA;
        }
        done[dev] = true;
    }
    return W4A16_OK;
}

// ---------------------------------------------------------------- gemm_pair launches
template <typename... A, typename... B>
w4a16_status launch_chained(void (*kern)(A...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                            B... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, static_cast<A>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return W4A16_ECUDA;
    }
    return W4A16_OK;
}

template <bool PAIR, int BITS, bool DGRAD>
w4a16_status launch_pair_t(const PairPlan& p, const CUtensorMap* tmX, const CUtensorMap* tmP, PairArgs args,
                           void* workspace, cudaStream_t stream) {
    auto kern = gemm_pair_kernel<PAIR, BITS, DGRAD>;
    static bool done[kMaxDevices] = {};
    w4a16_status st = set_smem(kern, PairConfig<PAIR, BITS, DGRAD>::kSmem, done);
    if (st != W4A16_OK) return st;
    pair_plan_args(p, &args);
    if (p.split) {
        args.flags = static_cast<uint64_t*>(workspace);
        args.ready = launch_flag();
        args.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + p.flag_bytes);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.grid * p.ctas), 1, 1);
    cfg.blockDim = dim3(PairConfig<PAIR, BITS, DGRAD>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = PairConfig<PAIR, BITS, DGRAD>::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kern, tmX[0], tmX[1], tmP[0], tmP[1], args) != cudaSuccess) {
        cudaGetLastError();
        return W4A16_ECUDA;
    }
    return W4A16_OK;
}

template <int BITS, bool DGRAD>
w4a16_status launch_pair(const PairPlan& p, const CUtensorMap* tmX, const CUtensorMap* tmP, const PairArgs& args,
                         void* workspace, cudaStream_t stream) {
    if (p.tiles > kMaxDim / (p.blocks + 1)) return W4A16_EINVAL;
    return p.ctas == 2 ? launch_pair_t<true, BITS, DGRAD>(p, tmX, tmP, args, workspace, stream)
                       : launch_pair_t<false, BITS, DGRAD>(p, tmX, tmP, args, workspace, stream);
}

struct Weights {
    const void* codes;
    const void* scales;
    const void* zeros;
};

bool weights_ok(const Weights& w, int32_t sym) {
    return w.codes && w.scales && (sym || w.zeros) && aligned16(w.codes) && aligned16(w.scales) &&
           (sym || aligned16(w.zeros));
}

void fill_weight_args(PairArgs* a, const Weights* w, int count, int64_t K, int32_t g, int32_t sym, int bits) {
    for (int i = 0; i < 2; ++i) {
        a->scales[i] = static_cast<const uint16_t*>(w[i < count ? i : 0].scales);
        a->zeros[i] = static_cast<const uint16_t*>(w[i < count ? i : 0].zeros);
    }
    a->gshift = group_shift(g, K);
    a->groups = per_channel(g, K) ? 1 : (int)(K / g);
    a->flip = sym ? (bits == 4 ? 0x88888888u : 0x80808080u) : 0u;
}

// dX [M, K] = Σ_p dY_p·Ŵ_p, dY_p rows of `ld` elements (a multiple of 8).
w4a16_status launch_dgrad(const PairPlan& p, const void* const* dY, const Weights* w, int products, int64_t M,
                          int64_t N, int64_t ld, int64_t K, int32_t g, int32_t sym, int bits, void* dX,
                          void* parts, cudaStream_t stream) {
    CUtensorMap tmX[2], tmP[2];
    w4a16_status st;
    const uint64_t row_bytes = (uint64_t)K * bits / 8;
    for (int i = 0; i < 2; ++i) {
        const int j = i < products ? i : 0;
        st = encode_rows(&tmX[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dY[j], (uint64_t)N, (uint64_t)M, (uint64_t)ld * 2,
                         kPairBlock, (uint32_t)p.bt, CU_TENSOR_MAP_SWIZZLE_128B);
        if (st != W4A16_OK) return st;
        st = encode_rows(&tmP[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, w[j].codes, row_bytes, (uint64_t)N, row_bytes, 128,
                         kPairBlock, CU_TENSOR_MAP_SWIZZLE_128B);
        if (st != W4A16_OK) return st;
    }
    PairArgs a{};
    fill_weight_args(&a, w, products, K, g, sym, bits);
    a.out = static_cast<uint16_t*>(dX);
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.products = products;
    return bits == 8 ? launch_pair<8, true>(p, tmX, tmP, a, parts, stream)
                     : launch_pair<4, true>(p, tmX, tmP, a, parts, stream);
}

PairPlan dgrad_plan(int64_t M, int64_t N, int64_t K, int products) {
    return pair_plan(M, K, 2 * kPairRows, (int64_t)products * ((N + kPairBlock - 1) / kPairBlock), 1,
                     current_sm_count());
}

// ---------------------------------------------------------------- gated, decode form
template <int MB, bool SYM, int G, int BITS>
w4a16_status launch_gated_decode_t(int64_t grid, int smem, const DecodeMaps<true, true>& maps, const DecodeArgs& args,
                                   cudaStream_t stream) {
    auto kern = gemv_decode_kernel<MB, SYM, G, BITS, true>;
    static bool done[kMaxDevices] = {};
    w4a16_status st = set_smem(kern, kSmemPerBlockMax, done);
    if (st != W4A16_OK) return st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kDecThreads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, maps, args) != cudaSuccess) {
        cudaGetLastError();
        return W4A16_ECUDA;
    }
    return W4A16_OK;
}

template <int MB, bool SYM, int BITS>
w4a16_status launch_gated_decode_g(int gsel, int64_t grid, int smem, const DecodeMaps<true, true>& maps,
                                   const DecodeArgs& args, cudaStream_t stream) {
    switch (gsel) {
        case 32: return launch_gated_decode_t<MB, SYM, 32, BITS>(grid, smem, maps, args, stream);
        case 64: return launch_gated_decode_t<MB, SYM, 64, BITS>(grid, smem, maps, args, stream);
        case 128: return launch_gated_decode_t<MB, SYM, 128, BITS>(grid, smem, maps, args, stream);
        default: return launch_gated_decode_t<MB, SYM, 0, BITS>(grid, smem, maps, args, stream);
    }
}

// 64-wide blocks per code unit of the tensor-core kernel (PairConfig::kUnitBlocks).
int gated_unit_blocks(int64_t M, int bits) {
    if (M > kPairMaxSingle)
        return bits == 8 ? PairConfig<true, 8, false>::kUnitBlocks : PairConfig<true, 4, false>::kUnitBlocks;
    return bits == 8 ? PairConfig<false, 8, false>::kUnitBlocks : PairConfig<false, 4, false>::kUnitBlocks;
}

// What a gated call of up to 16 tokens runs.  The decode kernel starts and ends sooner; the
// tensor-core kernel, whatever the tokens, dequantizes faster than 8-bit codes or two blocks of
// eight tokens do there.  They meet near 10^8 weights a matrix (4 bits, M = 16: 8192^2 33.3 us
// decode, 33.9 tensor cores; 8192 x 28672 113.9 and 82.5; 8 bits, M = 1: 29.8 and 35.5, 104.3
// and 88.8; 4 bits, M = 8: 81.3 and 82.7, so there it stays the decode kernel).
bool gated_decode(int64_t M, int64_t N, int64_t K, int bits) {
    return M <= 16 && ((bits == 4 && M <= 8) || N <= (int64_t(96) << 20) / K);
}

struct GatedPlan {
    bool decode;
    DecodeGeometry d;
    int64_t grid;
    PairPlan p;
    int64_t bytes;
};

w4a16_status gated_plan(int64_t M, int64_t N, int64_t K, int32_t g, int32_t path, int bits, GatedPlan* out) {
    if (path < W4A16_PATH_AUTO || path > W4A16_PATH_TENSORCORE) return W4A16_EINVAL;
    if (path == W4A16_PATH_DECODE && M > 16) return W4A16_EINVAL;
    GatedPlan q{};
    q.decode = path == W4A16_PATH_DECODE || (path == W4A16_PATH_AUTO && gated_decode(M, N, K, bits));
    if (N > kMaxDim / 2) return W4A16_EINVAL;
    if (q.decode) {
        q.d = decode_geometry(M, 2 * ((N + 127) / 128 * 128), K, g, bits);
        if (!decode_geometry_ok(q.d, M)) return W4A16_EUNSUPPORTED;
        q.grid = current_sm_count();
        if (q.grid > q.d.units) q.grid = q.d.units;
        if (q.grid < 1) q.grid = 1;
        q.bytes = decode_workspace_bytes<uint64_t>(q.d, q.grid);
    } else {
        q.p = pair_plan(M, N, kPairRows, (K + kPairBlock - 1) / kPairBlock, gated_unit_blocks(M, bits), current_sm_count());
        q.bytes = q.p.bytes;
    }
    *out = q;
    return W4A16_OK;
}

w4a16_status launch_gated_decode(const GatedPlan& q, const void* X, int64_t M, int64_t K, const Weights* w,
                                 int64_t N, int32_t g, int32_t sym, int32_t act, void* H, void* G, void* U,
                                 void* workspace, bool static_weights, int bits, cudaStream_t stream) {
    const DecodeGeometry& d = q.d;
    const uint64_t row_bytes = (uint64_t)K * bits / 8;
    const bool pc = per_channel(g, K);
    const uint64_t groups = pc ? 1 : (uint64_t)(K / g);
    DecodeMaps<true, true> maps;
    maps.codes = static_cast<const uint8_t*>(w[0].codes);
    maps.codes2 = static_cast<const uint8_t*>(w[1].codes);
    maps.x = static_cast<const uint16_t*>(X);
    w4a16_status st = encode_rows(&maps.P, CU_TENSOR_MAP_DATA_TYPE_UINT8, w[0].codes, row_bytes, (uint64_t)N, row_bytes,
                                  kDecUnitRowBytes, kDecRows / 2, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st == W4A16_OK)
        st = encode_rows(&maps.P2, CU_TENSOR_MAP_DATA_TYPE_UINT8, w[1].codes, row_bytes, (uint64_t)N, row_bytes,
                         kDecUnitRowBytes, kDecRows / 2, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st == W4A16_OK)
        st = encode_rows(&maps.X, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, X, (uint64_t)K, (uint64_t)M, (uint64_t)K * 2,
                         (uint32_t)decode_block_k(bits), (uint32_t)M, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (st != W4A16_OK) return st;
    maps.S = maps.Z = maps.P;
    maps.S2 = maps.Z2 = maps.P2;
    if (d.sz_tma) {
        CUtensorMap* to[4] = {&maps.S, &maps.S2, &maps.Z, &maps.Z2};
        const void* from[4] = {w[0].scales, w[1].scales, w[0].zeros, w[1].zeros};
        for (int i = 0; i < (sym ? 2 : 4); ++i) {
            st = encode_rows(to[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, from[i], groups, (uint64_t)N, groups * 2, 8,
                             kDecRows / 2, CU_TENSOR_MAP_SWIZZLE_NONE);
            if (st != W4A16_OK) return st;
        }
    }
    DecodeArgs a{};
    a.scales = static_cast<const uint16_t*>(w[0].scales);
    a.zeros = static_cast<const uint16_t*>(w[0].zeros);
    maps.scales2 = static_cast<const uint16_t*>(w[1].scales);
    maps.zeros2 = static_cast<const uint16_t*>(w[1].zeros);
    a.Y = static_cast<uint16_t*>(H);
    maps.G = static_cast<uint16_t*>(G);
    maps.U = static_cast<uint16_t*>(U);
    maps.act = act;
    maps.ready = launch_flag();
    a.ws_flag = workspace;
    a.ws_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + decode_flag_bytes<uint64_t>(d, q.grid));
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.RB = d.rb;
    a.KBn = d.kbn;
    a.Gtot = (int)groups;
    a.stages = d.stages;
    a.stage_bytes = d.stage_bytes;
    a.xf_off = d.xf_off;
    a.sz_off = d.sz_off;
    a.sz_tma = d.sz_tma;
    a.slab_off = d.slab_off;
    a.slabs = d.slabs;
    a.sz_copy = pc ? 16 : decode_scale_copy(d.gu, K / g);
    a.early = static_weights ? 1 : 0;
    a.units = d.units;
    const int gsel = pc ? 0 : g;
#define W4A16_GATED(MBV, SYMV)                                                                             \
    (bits == 8 ? launch_gated_decode_g<MBV, SYMV, 8>(gsel, q.grid, d.smem_bytes, maps, a, stream)          \
               : launch_gated_decode_g<MBV, SYMV, 4>(gsel, q.grid, d.smem_bytes, maps, a, stream))
    if (d.mb == 1) return sym ? W4A16_GATED(1, true) : W4A16_GATED(1, false);
    return sym ? W4A16_GATED(2, true) : W4A16_GATED(2, false);
#undef W4A16_GATED
}

w4a16_status gated_impl(const void* X, int64_t M, int64_t K, const Weights* w, int64_t N, int32_t g, int32_t sym,
                        int32_t act, void* H, void* G, void* U, void* workspace, size_t workspace_bytes,
                        int32_t path, void* stream, int bits) {
    const bool static_weights = (path & W4A16_STATIC_WEIGHTS) != 0;
    path &= ~W4A16_STATIC_WEIGHTS;
    w4a16_status st = check_shape(M, N, K, g, sym);
    if (st != W4A16_OK) return st;
    if (!valid_act(act)) return W4A16_EINVAL;
    GatedPlan q;
    st = gated_plan(M, N, K, g, path, bits, &q);
    if (st != W4A16_OK) return st;
    if (M == 0 || N == 0) return W4A16_OK;
    if (!X || !H || !weights_ok(w[0], sym) || !weights_ok(w[1], sym) || (G == nullptr) != (U == nullptr))
        return W4A16_EINVAL;
    if (!aligned16(X) || !aligned16(H) || (G && (!aligned16(G) || !aligned16(U)))) return W4A16_EINVAL;
    if (workspace_bytes < (size_t)q.bytes) return W4A16_EWORKSPACE;
    if (q.bytes > 0 && (workspace == nullptr || !aligned16(workspace))) return W4A16_EINVAL;
    DeviceInfo di;
    if ((st = device_info(&di)) != W4A16_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (q.decode)
        return launch_gated_decode(q, X, M, K, w, N, g, sym, act, H, G, U, workspace, static_weights, bits, s);
    CUtensorMap tmX[2], tmP[2];
    st = encode_rows(&tmX[0], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, X, (uint64_t)K, (uint64_t)M, (uint64_t)K * 2, kPairBlock,
                     (uint32_t)q.p.bt, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != W4A16_OK) return st;
    tmX[1] = tmX[0];
    const uint64_t row_bytes = (uint64_t)K * bits / 8;
    for (int i = 0; i < 2; ++i) {
        st = encode_rows(&tmP[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, w[i].codes, row_bytes, (uint64_t)N, row_bytes,
                         q.p.ctas == 2 ? 64 : 128, kPairRows,
                         q.p.ctas == 2 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
        if (st != W4A16_OK) return st;
    }
    PairArgs a{};
    fill_weight_args(&a, w, 2, K, g, sym, bits);
    a.out = static_cast<uint16_t*>(H);
    a.G = static_cast<uint16_t*>(G);
    a.U = static_cast<uint16_t*>(U);
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.act = act;
    a.products = 1;
    return bits == 8 ? launch_pair<8, false>(q.p, tmX, tmP, a, workspace, s)
                     : launch_pair<4, false>(q.p, tmX, tmP, a, workspace, s);
}

size_t gated_ws(int64_t M, int64_t N, int64_t K, int32_t g, int32_t path, int bits) {
    GatedPlan q;
    if (check_shape(M, N, K, g, 0) != W4A16_OK || M == 0 || N == 0) return 0;
    if (gated_plan(M, N, K, g, path & ~W4A16_STATIC_WEIGHTS, bits, &q) != W4A16_OK) return 0;
    return (size_t)q.bytes;
}

// Bytes of the padded copies of `products` gradients with rows of N elements.
int64_t pad_bytes(int64_t M, int64_t N, int products) {
    return N % 8 == 0 ? 0 : products * round256(M * round8(N) * 2);
}

w4a16_status dgrad_impl(const void* dY, int64_t M, int64_t N, const Weights& w, int64_t K, int32_t g, int32_t sym,
                        void* dX, void* workspace, size_t workspace_bytes, void* stream, int bits) {
    w4a16_status st = check_shape(M, N, K, g, sym);
    if (st != W4A16_OK) return st;
    if (M == 0) return W4A16_OK;
    if (!dX || !aligned16(dX)) return W4A16_EINVAL;
    if (N > 0 && (!dY || !aligned16(dY) || !weights_ok(w, sym))) return W4A16_EINVAL;
    const PairPlan p = dgrad_plan(M, N, K, 1);
    const int64_t pad = pad_bytes(M, N, 1), need = pad + p.bytes;
    if (workspace_bytes < (size_t)need) return W4A16_EWORKSPACE;
    if (need > 0 && (!workspace || !aligned16(workspace))) return W4A16_EINVAL;
    DeviceInfo di;
    if ((st = device_info(&di)) != W4A16_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (N == 0) return cudaMemsetAsync(dX, 0, (size_t)(M * K * 2), s) == cudaSuccess ? W4A16_OK : W4A16_ECUDA;
    int64_t ld = N;
    if (pad > 0) {
        ld = round8(N);
        pad_rows_kernel<<<grid_for(M * ld, 256, di.sm_count), 256, 0, s>>>(
            static_cast<const uint16_t*>(dY), M, (int)N, (int)ld, static_cast<uint16_t*>(workspace));
        if ((st = launch_status()) != W4A16_OK) return st;
        dY = workspace;
    }
    return launch_dgrad(p, &dY, &w, 1, M, N, ld, K, g, sym, bits, dX, static_cast<uint8_t*>(workspace) + pad, s);
}

size_t dgrad_ws(int64_t M, int64_t N, int64_t K, int32_t g, int products) {
    if (check_shape(M, N, K, g, 0) != W4A16_OK || M == 0 || N == 0) return 0;
    return (size_t)(pad_bytes(M, N, products) + dgrad_plan(M, N, K, products).bytes);
}

w4a16_status gated_backward_impl(const void* dH, const void* G, const void* U, int64_t M, int64_t N,
                                 const Weights* w, int64_t K, int32_t g, int32_t sym, int32_t act, void* dX,
                                 void* dG, void* dU, void* workspace, size_t workspace_bytes, void* stream,
                                 int bits) {
    w4a16_status st = check_shape(M, N, K, g, sym);
    if (st != W4A16_OK) return st;
    if (!valid_act(act)) return W4A16_EINVAL;
    if (M == 0) return W4A16_OK;
    if (!dX || !aligned16(dX)) return W4A16_EINVAL;
    if (N > 0) {
        const void* in[5] = {dH, G, U, dG, dU};
        for (const void* t : in)
            if (!t || !aligned16(t)) return W4A16_EINVAL;
        if (!weights_ok(w[0], sym) || !weights_ok(w[1], sym)) return W4A16_EINVAL;
    }
    const PairPlan p = dgrad_plan(M, N, K, 2);
    const int64_t pad = pad_bytes(M, N, 2), need = pad + p.bytes;
    if (workspace_bytes < (size_t)need) return W4A16_EWORKSPACE;
    if (need > 0 && (!workspace || !aligned16(workspace))) return W4A16_EINVAL;
    DeviceInfo di;
    if ((st = device_info(&di)) != W4A16_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (N == 0) return cudaMemsetAsync(dX, 0, (size_t)(M * K * 2), s) == cudaSuccess ? W4A16_OK : W4A16_ECUDA;
    const void* dY[2] = {dG, dU};
    int64_t ld = N;
    if (pad == 0) {
        const int64_t chunks = M * N / 8;
        gate_backward_kernel<<<grid_for(chunks, 256, di.sm_count), 256, 0, s>>>(
            static_cast<const uint4*>(dH), static_cast<const uint4*>(G), static_cast<const uint4*>(U), chunks, act,
            static_cast<uint4*>(dG), static_cast<uint4*>(dU));
    } else {
        ld = round8(N);
        uint16_t* p0 = static_cast<uint16_t*>(workspace);
        uint16_t* p1 = p0 + pad / 4;                       // half of the padded bytes further
        gate_backward_rows_kernel<<<grid_for(M * ld, 256, di.sm_count), 256, 0, s>>>(
            static_cast<const uint16_t*>(dH), static_cast<const uint16_t*>(G), static_cast<const uint16_t*>(U), M,
            (int)N, (int)ld, act, static_cast<uint16_t*>(dG), static_cast<uint16_t*>(dU), p0, p1);
        dY[0] = p0;
        dY[1] = p1;
    }
    if ((st = launch_status()) != W4A16_OK) return st;
    return launch_dgrad(p, dY, w, 2, M, N, ld, K, g, sym, bits, dX, static_cast<uint8_t*>(workspace) + pad, s);
}

// ---------------------------------------------------------------- embedding
w4a16_status embedding_impl(const void* ids, int32_t id_bytes, int64_t T, const Weights& w, int64_t V, int64_t K,
                            int32_t g, int32_t sym, float scale, void* out, void* stream, int bits) {
    w4a16_status st = check_shape(T, V, K, g, sym);
    if (st != W4A16_OK) return st;
    if (id_bytes != 4 && id_bytes != 8) return W4A16_EINVAL;
    if (T == 0) return W4A16_OK;
    if (!ids || !out || !aligned_to(ids, id_bytes) || !aligned16(out)) return W4A16_EINVAL;
    if (V > 0 && !weights_ok(w, sym)) return W4A16_EINVAL;
    DeviceInfo di;
    if ((st = device_info(&di)) != W4A16_OK) return st;
    const int chunks = (int)(K / 8);
    const int gy = (chunks + 1023) / 1024;
    if (gy > 65535) return W4A16_EINVAL;
    const dim3 grid((unsigned)T, (unsigned)gy, 1);
    const int groups = per_channel(g, K) ? 1 : (int)(K / g);
    auto kern = bits == 8 ? embedding_kernel<8> : embedding_kernel<4>;
    kern<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(
        ids, id_bytes == 8 ? 1 : 0, static_cast<const uint8_t*>(w.codes), static_cast<const uint16_t*>(w.scales),
        static_cast<const uint16_t*>(w.zeros), V, chunks, group_shift(g, K), groups, sym, scale,
        static_cast<uint4*>(out));
    return launch_status();
}

// Workspace of the embedding gradient: chunk-sorted keys and tokens, the same merged
// (more than one chunk), and the windows' binary32 parts.
struct EmbedGradPlan {
    int key_bits;            // of the ids 0 .. V (V: dropped)
    bool small;              // chunks of 1024 ids, else of 16384
    int64_t chunk, chunks, padded;
    int window;              // sorted tokens per window
    int64_t windows;
    int64_t list_bytes;      // one key or token list
    int64_t bytes;
};

// Chunks of 1024 ids spread the sort over many SMs (2048 ids in one CTA of 4096: 10 us, in two
// of 1024: 4 us); ranking costs ids x chunks, so from 65536 ids on a chunk holds 16384.
EmbedGradPlan embed_grad_plan(int64_t T, int64_t V, int64_t K) {
    EmbedGradPlan p{};
    while (p.key_bits < 31 && (int64_t(1) << p.key_bits) <= V) ++p.key_bits;
    p.small = T <= 65536;
    p.chunk = p.small ? 1024 : 16384;
    p.chunks = (T + p.chunk - 1) / p.chunk;
    p.padded = p.chunks * p.chunk;
    // (2048 ids: 37 us with 32, 42 with 64, which make half the CTAs; 16384 ids: joining the
    // parts takes 23 us with 32 and 14 with 64)
    p.window = T <= 4096 ? kGradWindow / 2 : kGradWindow;
    p.windows = (T + p.window - 1) / p.window;
    p.list_bytes = p.padded * 4;
    p.bytes = p.list_bytes * (p.chunks > 1 ? 4 : 2) + p.windows * 2 * K * 4;
    return p;
}

template <typename W, int THREADS, int PER, bool F32>
w4a16_status launch_sort(const EmbedGradPlan& p, const void* ids, int wide, int64_t T, int64_t V, uint32_t* skey,
                         uint32_t* sidx, int64_t zero_end, int zero_ctas, int64_t K, void* dW, cudaStream_t s) {
    using Cfg = SortConfig<W, THREADS, PER>;
    auto kern = embed_sort_kernel<W, THREADS, PER, F32>;
    static bool done[kMaxDevices] = {};
    w4a16_status st = set_smem(kern, Cfg::kSmem, done);
    if (st != W4A16_OK) return st;
    const int per = zero_ctas > 0 ? (int)((zero_end + zero_ctas - 1) / zero_ctas) : 0;
    kern<<<(unsigned)(p.chunks + zero_ctas), THREADS, Cfg::kSmem, s>>>(ids, wide, T, V, p.key_bits, skey, sidx,
                                                                       (int)p.chunks, zero_end, per, (int)K, dW);
    return launch_status();
}

bool embed_grad_ok(int64_t T, int64_t V, int64_t K) {
    return T >= 0 && V >= 0 && K > 0 && K % 32 == 0 && T <= kMaxDim / 2 && V < kMaxDim && K <= kMaxDim;
}

template <bool F32>
w4a16_status launch_embed_grad(const void* dY, const void* ids, int wide, int64_t T, int64_t V, int64_t K, float scale,
                               void* dW, void* workspace, cudaStream_t s) {
    const EmbedGradPlan p = embed_grad_plan(T, V, K);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    uint32_t* skey = reinterpret_cast<uint32_t*>(ws);
    uint32_t* sidx = reinterpret_cast<uint32_t*>(ws + p.list_bytes);
    uint32_t *key = skey, *idx = sidx;
    ws += 2 * p.list_bytes;
    if (p.chunks > 1) {
        key = reinterpret_cast<uint32_t*>(ws);
        idx = reinterpret_cast<uint32_t*>(ws + p.list_bytes);
        ws += 2 * p.list_bytes;
    }
    float* part = reinterpret_cast<float*>(ws);
    // Rows zeroed beside the sort: about 30 MB, what the machine writes in the sort's time.  Their
    // CTAs look through all ids and keep a bit per row in shared memory (4 KB at least).
    int64_t zero1 = T <= 16384 ? (int64_t)(30 << 20) / (K * (F32 ? 4 : 2)) : 0;
    if (zero1 > V / 4) zero1 = V / 4;
    const int zero_ctas = zero1 > 0 ? (int)(zero1 < 128 ? zero1 : 128) : 0;
    if (zero1 > 128ll * 8 * 4096) zero1 = 128ll * 8 * 4096;
    w4a16_status st;
    if (p.small && p.key_bits <= 22)
        st = launch_sort<uint32_t, 256, 4, F32>(p, ids, wide, T, V, skey, sidx, zero1, zero_ctas, K, dW, s);
    else if (p.small)
        st = launch_sort<uint64_t, 256, 4, F32>(p, ids, wide, T, V, skey, sidx, zero1, zero_ctas, K, dW, s);
    else
        st = launch_sort<uint64_t, 1024, 16, F32>(p, ids, wide, T, V, skey, sidx, zero1, zero_ctas, K, dW, s);
    if (st != W4A16_OK) return st;
    if (p.chunks > 1) {
        int lanes = 1;
        while (lanes < 32 && lanes < p.chunks) lanes *= 2;
        const bool shared = p.padded <= kRankShared;
        // (whole blocks: padded is a multiple of 1024)
        const int64_t blocks = shared ? p.padded * kRankPer / kRankThreads : p.padded * lanes / kRankThreads;
        static bool done[kMaxDevices] = {};
        if (shared && (st = set_smem(embed_rank_kernel<true>, (int)kRankShared * 4, done)) != W4A16_OK) return st;
        st = launch_chained(shared ? embed_rank_kernel<true> : embed_rank_kernel<false>, dim3((unsigned)blocks),
                            kRankThreads, shared ? (size_t)p.padded * 4 : 0, s, skey, sidx, (int)p.chunks,
                            (int)p.chunk, lanes, key, idx);
        if (st != W4A16_OK) return st;
    }
    const int slices = (int)((K + kGradCols - 1) / kGradCols);
    const int64_t zero2 = zero1 + (V - zero1) * 15 / 16;
    const int64_t blocks = p.windows * slices + (zero2 - zero1 + kZeroRows - 1) / kZeroRows;
    const int64_t blocks2 = p.windows * slices + (V - zero2 + kZeroRows - 1) / kZeroRows;
    if (blocks > kMaxDim || blocks2 > kMaxDim) return W4A16_EINVAL;
    st = launch_chained(embed_grad_kernel<F32>, dim3((unsigned)blocks), kGradThreads, 0, s,
                        static_cast<const uint16_t*>(dY), key, idx, p.padded, p.window, (int)p.windows, slices, V, zero1, zero2,
                        (int)K, scale, dW, part);
    if (st != W4A16_OK) return st;
    return launch_chained(embed_grad_join_kernel<F32>, dim3((unsigned)blocks2), kGradThreads, 0, s, key, p.padded,
                          p.window, (int)p.windows, slices, V, zero2, (int)K, scale, dW, part);
}

}  // namespace

// Reads and clears this translation unit's device error word.
int train_take_device_error(int* value) {
    int zero = 0;
    if (cudaMemcpyFromSymbol(value, g_device_error, sizeof(int)) != cudaSuccess) return 1;
    if (*value != 0 && cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int)) != cudaSuccess) return 1;
    return 0;
}

extern "C" {

size_t w4a16_gated_workspace_size(int64_t M, int64_t N, int64_t K, int32_t g, int32_t path) {
    return gated_ws(M, N, K, g, path, 4);
}

size_t w8a16_gated_workspace_size(int64_t M, int64_t N, int64_t K, int32_t g, int32_t path) {
    return gated_ws(M, N, K, g, path, 8);
}

w4a16_status w4a16_gated(const void* X, int64_t M, int64_t K, const void* gate_packed, const void* gate_scales,
                         const void* gate_zeros, const void* up_packed, const void* up_scales,
                         const void* up_zeros, int64_t N, int32_t g, int32_t sym, int32_t act, void* H, void* G,
                         void* U, void* workspace, size_t workspace_bytes, int32_t path, void* stream) {
    const Weights w[2] = {{gate_packed, gate_scales, gate_zeros}, {up_packed, up_scales, up_zeros}};
    return gated_impl(X, M, K, w, N, g, sym, act, H, G, U, workspace, workspace_bytes, path, stream, 4);
}

w4a16_status w8a16_gated(const void* X, int64_t M, int64_t K, const void* gate_codes, const void* gate_scales,
                         const void* gate_zeros, const void* up_codes, const void* up_scales, const void* up_zeros,
                         int64_t N, int32_t g, int32_t sym, int32_t act, void* H, void* G, void* U, void* workspace,
                         size_t workspace_bytes, int32_t path, void* stream) {
    const Weights w[2] = {{gate_codes, gate_scales, gate_zeros}, {up_codes, up_scales, up_zeros}};
    return gated_impl(X, M, K, w, N, g, sym, act, H, G, U, workspace, workspace_bytes, path, stream, 8);
}

size_t w4a16_gated_backward_workspace_size(int64_t M, int64_t N, int64_t K, int32_t g) {
    return dgrad_ws(M, N, K, g, 2);
}

w4a16_status w4a16_gated_backward(const void* dH, const void* G, const void* U, int64_t M, int64_t N,
                                  const void* gate_packed, const void* gate_scales, const void* gate_zeros,
                                  const void* up_packed, const void* up_scales, const void* up_zeros, int64_t K,
                                  int32_t g, int32_t sym, int32_t act, void* dX, void* dG, void* dU,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    const Weights w[2] = {{gate_packed, gate_scales, gate_zeros}, {up_packed, up_scales, up_zeros}};
    return gated_backward_impl(dH, G, U, M, N, w, K, g, sym, act, dX, dG, dU, workspace, workspace_bytes, stream, 4);
}

w4a16_status w8a16_gated_backward(const void* dH, const void* G, const void* U, int64_t M, int64_t N,
                                  const void* gate_codes, const void* gate_scales, const void* gate_zeros,
                                  const void* up_codes, const void* up_scales, const void* up_zeros, int64_t K,
                                  int32_t g, int32_t sym, int32_t act, void* dX, void* dG, void* dU,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    const Weights w[2] = {{gate_codes, gate_scales, gate_zeros}, {up_codes, up_scales, up_zeros}};
    return gated_backward_impl(dH, G, U, M, N, w, K, g, sym, act, dX, dG, dU, workspace, workspace_bytes, stream, 8);
}

size_t w4a16_gemm_dgrad_workspace_size(int64_t M, int64_t N, int64_t K, int32_t g) {
    return dgrad_ws(M, N, K, g, 1);
}

w4a16_status w4a16_gemm_dgrad(const void* dY, int64_t M, int64_t N, const void* packed, const void* scales,
                              const void* zeros, int64_t K, int32_t g, int32_t sym, void* dX, void* workspace,
                              size_t workspace_bytes, void* stream) {
    return dgrad_impl(dY, M, N, Weights{packed, scales, zeros}, K, g, sym, dX, workspace, workspace_bytes, stream, 4);
}

w4a16_status w8a16_gemm_dgrad(const void* dY, int64_t M, int64_t N, const void* codes, const void* scales,
                              const void* zeros, int64_t K, int32_t g, int32_t sym, void* dX, void* workspace,
                              size_t workspace_bytes, void* stream) {
    return dgrad_impl(dY, M, N, Weights{codes, scales, zeros}, K, g, sym, dX, workspace, workspace_bytes, stream, 8);
}

size_t w4a16_gemm_wgrad_workspace_size(int64_t M, int64_t N) {
    if (M <= 0 || N <= 0 || M > kMaxDim || N > kMaxDim) return 0;
    return (size_t)pad_bytes(M, N, 1);
}

w4a16_status w4a16_gemm_wgrad(const void* dY, const void* X, int64_t M, int64_t N, int64_t K, void* dW,
                              void* workspace, size_t workspace_bytes, void* stream) {
    if (M < 0 || N < 0 || K <= 0 || K % 32 != 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return W4A16_EINVAL;
    if (N == 0) return W4A16_OK;
    if (!dW || !aligned16(dW)) return W4A16_EINVAL;
    if (M > 0 && (!dY || !X || !aligned16(dY) || !aligned16(X))) return W4A16_EINVAL;
    const int64_t need = M > 0 ? pad_bytes(M, N, 1) : 0;
    if (workspace_bytes < (size_t)need) return W4A16_EWORKSPACE;
    if (need > 0 && (!workspace || !aligned16(workspace))) return W4A16_EINVAL;
    DeviceInfo di;
    w4a16_status st = device_info(&di);
    if (st != W4A16_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M == 0) return cudaMemsetAsync(dW, 0, (size_t)N * K * 2, s) == cudaSuccess ? W4A16_OK : W4A16_ECUDA;
    int64_t ld = N;
    if (need > 0) {
        ld = round8(N);
        pad_rows_kernel<<<grid_for(M * ld, 256, di.sm_count), 256, 0, s>>>(
            static_cast<const uint16_t*>(dY), M, (int)N, (int)ld, static_cast<uint16_t*>(workspace));
        if ((st = launch_status()) != W4A16_OK) return st;
        dY = workspace;
    }
    CUtensorMap tmY, tmX;
    st = encode_rows(&tmY, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dY, (uint64_t)N, (uint64_t)M, (uint64_t)ld * 2, 64, kWgBlockM,
                     CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != W4A16_OK) return st;
    st = encode_rows(&tmX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, X, (uint64_t)K, (uint64_t)M, (uint64_t)K * 2, 64, kWgBlockM,
                     CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != W4A16_OK) return st;
    CUtensorMap tmW;
    st = encode_rows(&tmW, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dW, (uint64_t)K, (uint64_t)N, (uint64_t)K * 2, 64, 32,
                     CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != W4A16_OK) return st;
    static bool done[kMaxDevices] = {};
    st = set_smem(gemm_wgrad_kernel, kWgSmemBytes, done);
    if (st != W4A16_OK) return st;
    const int64_t tiles = ((N + kWgTile - 1) / kWgTile) * ((K + kWgTile - 1) / kWgTile);
    const int64_t pairs = tiles < di.sm_count / 2 ? tiles : di.sm_count / 2;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
    cfg.blockDim = dim3(kWgThreads, 1, 1);
    cfg.dynamicSmemBytes = kWgSmemBytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, gemm_wgrad_kernel, tmY, tmX, tmW, (int)M, (int)N, (int)K) !=
        cudaSuccess) {
        cudaGetLastError();
        return W4A16_ECUDA;
    }
    return W4A16_OK;
}

w4a16_status w4a16_embedding(const void* ids, int32_t id_bytes, int64_t T, const void* packed, const void* scales,
                             const void* zeros, int64_t V, int64_t K, int32_t g, int32_t sym, float scale, void* out,
                             void* stream) {
    return embedding_impl(ids, id_bytes, T, Weights{packed, scales, zeros}, V, K, g, sym, scale, out, stream, 4);
}

w4a16_status w8a16_embedding(const void* ids, int32_t id_bytes, int64_t T, const void* codes, const void* scales,
                             const void* zeros, int64_t V, int64_t K, int32_t g, int32_t sym, float scale, void* out,
                             void* stream) {
    return embedding_impl(ids, id_bytes, T, Weights{codes, scales, zeros}, V, K, g, sym, scale, out, stream, 8);
}

size_t w4a16_embedding_grad_workspace_size(int64_t T, int64_t V, int64_t K) {
    if (!embed_grad_ok(T, V, K) || T == 0 || V == 0) return 0;
    return (size_t)embed_grad_plan(T, V, K).bytes;
}

w4a16_status w4a16_embedding_grad(const void* dY, const void* ids, int32_t id_bytes, int64_t T, int64_t V, int64_t K,
                                  float scale, int32_t f32, void* dW, void* workspace, size_t workspace_bytes,
                                  void* stream) {
    if (!embed_grad_ok(T, V, K) || (id_bytes != 4 && id_bytes != 8) || (f32 != 0 && f32 != 1)) return W4A16_EINVAL;
    if (V == 0) return W4A16_OK;
    if (!dW || !aligned16(dW)) return W4A16_EINVAL;
    if (T > 0 && (!dY || !ids || !aligned16(dY) || !aligned_to(ids, id_bytes))) return W4A16_EINVAL;
    const size_t need = w4a16_embedding_grad_workspace_size(T, V, K);
    if (workspace_bytes < need) return W4A16_EWORKSPACE;
    if (need > 0 && (!workspace || !aligned16(workspace))) return W4A16_EINVAL;
    DeviceInfo di;
    w4a16_status st = device_info(&di);
    if (st != W4A16_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0)
        return cudaMemsetAsync(dW, 0, (size_t)V * K * (f32 ? 4 : 2), s) == cudaSuccess ? W4A16_OK : W4A16_ECUDA;
    const int wide = id_bytes == 8 ? 1 : 0;
    return f32 ? launch_embed_grad<true>(dY, ids, wide, T, V, K, scale, dW, workspace, s)
               : launch_embed_grad<false>(dY, ids, wide, T, V, K, scale, dW, workspace, s);
}

}  // extern "C"
