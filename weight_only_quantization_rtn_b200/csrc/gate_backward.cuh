// Elementwise half of the gated block's backward pass, and the row padding that the
// tensor-core kernels' loads need.
//
//   dG = dH·U·act'(G),  dU = dH·act(G)
//
// in binary32 from the kept bf16 G and U, each rounded to bf16 once: they are results
// (the gradients at the two projections' outputs, which adapters and weight gradients
// start from) and the operands of the tensor-core product that gives dX, which takes
// bf16.  The rounding shows in dX: off by 0.0023 of its norm from the definition in
// binary64, where a product of unrounded operands is off by 0.0017, all of it dX's own
// rounding; a second bf16 part of each would double the product's time.  Bound by memory: 10
// bytes per element (2048 x 11008: 41 us, 5.4 TB/s, when nothing of it is in L2).  It is a pass of its own because
// the product reads each element once per block of 256 or 512 input channels: formed
// inside it, the exponentials and three reads would be repeated as often.
#pragma once

#include "activation.cuh"
#include "common.cuh"

namespace w4a16 {

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// dG and dU may be G's and U's own memory, so those four are not declared apart and G and U are
// not read through the read-only path; each element is read and then written by one thread.
//
// Eight elements per thread and step over the flat arrays (16-byte chunks).
__global__ void __launch_bounds__(256) gate_backward_kernel(const uint4* __restrict__ dH, const uint4* G,
                                                            const uint4* U, int64_t chunks, int act, uint4* dG,
                                                            uint4* dU) {
    for (int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; c < chunks;
         c += (int64_t)gridDim.x * blockDim.x) {
        const uint4 h = ldg_stream(dH + c), g = ld_stream(G + c), u = ld_stream(U + c);
        const uint32_t hv[4] = {h.x, h.y, h.z, h.w}, gv[4] = {g.x, g.y, g.z, g.w}, uv[4] = {u.x, u.y, u.z, u.w};
        uint32_t og[4], ou[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float dg[2], du[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float hx = __uint_as_float(j ? hv[i] & 0xFFFF0000u : hv[i] << 16);
                const float gx = __uint_as_float(j ? gv[i] & 0xFFFF0000u : gv[i] << 16);
                const float ux = __uint_as_float(j ? uv[i] & 0xFFFF0000u : uv[i] << 16);
                float av, dv;
                act_value_grad(act, gx, av, dv);
                dg[j] = hx * ux * dv;
                du[j] = hx * av;
            }
            og[i] = pack_bf16x2(dg[0], dg[1]);
            ou[i] = pack_bf16x2(du[0], du[1]);
        }
        dG[c] = make_uint4(og[0], og[1], og[2], og[3]);
        dU[c] = make_uint4(ou[0], ou[1], ou[2], ou[3]);
    }
}

// The same for rows of any length, element by element, with copies of dG and dU in rows
// padded with zeros to `ld` elements (a multiple of 8: TMA rows start on 16 bytes).
__global__ void __launch_bounds__(256) gate_backward_rows_kernel(const uint16_t* __restrict__ dH,
                                                                 const uint16_t* G, const uint16_t* U, int64_t M,
                                                                 int N, int ld, int act, uint16_t* dG, uint16_t* dU,
                                                                 uint16_t* __restrict__ pG,
                                                                 uint16_t* __restrict__ pU) {
    const int64_t total = M * ld;
    for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < total;
         e += (int64_t)gridDim.x * blockDim.x) {
        const int64_t m = e / ld;
        const int n = (int)(e - m * ld);
        uint16_t og = 0, ou = 0;
        if (n < N) {
            const int64_t at = m * N + n;
            const float hx = bf16_bits_to_f32(dH[at]), ux = bf16_bits_to_f32(U[at]);
            float av, dv;
            act_value_grad(act, bf16_bits_to_f32(G[at]), av, dv);
            og = (uint16_t)f32_to_bf16_bits_rn(hx * ux * dv);
            ou = (uint16_t)f32_to_bf16_bits_rn(hx * av);
            dG[at] = og;
            dU[at] = ou;
        }
        pG[e] = og;
        pU[e] = ou;
    }
}

// Rows of N elements copied into rows of `ld`, the rest zero.
__global__ void __launch_bounds__(256) pad_rows_kernel(const uint16_t* __restrict__ in, int64_t M, int N,
                                                       int ld, uint16_t* __restrict__ out) {
    const int64_t total = M * ld;
    for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < total;
         e += (int64_t)gridDim.x * blockDim.x) {
        const int64_t m = e / ld;
        const int n = (int)(e - m * ld);
        out[e] = n < N ? in[m * N + n] : (uint16_t)0;
    }
}

}  // namespace w4a16
