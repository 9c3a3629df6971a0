// linear_common.cuh -- the epilogue of the dense product, shared by its kernels:
//   y[t, n] = bf16_rn( act( sum + bias[n] ) + residual[t, n] ),  one rounding at the end.
#pragma once

#include "block_kernels.h"
#include "gemm_common.cuh"

namespace moe {

// cfg.activation: 0 none, 1 relu, 2 silu, 3 gelu (erf), 4 gelu (tanh form).  The two with a logistic
// take the hardware exponential and reciprocal (a few fp32 ulps, far below the bf16 rounding that
// follows); NaN stays NaN in every one.
__device__ __forceinline__ float linear_act(float v, int act) {
    switch (act) {
        case 1: return v < 0.0f ? 0.0f : v;
        case 2: return silu(v);
        case 3: return 0.5f * v * (1.0f + erff(v * 0.70710678f));
        case 4: {   // 0.5 (1 + tanh u) = 1 / (1 + e^-2u),  u = sqrt(2/pi) (v + 0.044715 v^3)
            const float u2 = 1.5957691f * fmaf(0.044715f * v * v, v, v);
            return __fdividef(v, 1.0f + __expf(-u2));
        }
        default: return v;
    }
}

__device__ __forceinline__ void add_bf16x8(float* v, uint4 w) { add_bias8(v, w); }

__device__ __forceinline__ uint4 pack_bf16x8(const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The lane's row t, columns c0 .. c0+31 from acc, when N is a multiple of 8 (16-byte rows).
__device__ __forceinline__ void linear_store32(const LinearArgs& p, float* acc, int t, int c0) {
    const size_t at = static_cast<size_t>(t) * p.N + c0;
#pragma unroll
    for (int c = 0; c < 32; c += 8) {
        if (c0 + c < p.N) {
            float* v = acc + c;
            if (p.bias) add_bias8(v, ld_nc_u4(reinterpret_cast<const uint4*>(p.bias + c0 + c)));
            if (p.act) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = linear_act(v[i], p.act);
            }
            // y may be the residual buffer itself: a plain load, by the thread that then stores
            if (p.res) add_bias8(v, *reinterpret_cast<const uint4*>(p.res + at + c));
            *reinterpret_cast<uint4*>(p.y + at + c) = pack_bf16x8(v);
        }
    }
}

// Any N: a warp's 32 rows x CW columns through shared memory (stage: 32 x (CW + 1) floats of the
// warp's own), stored by columns so that a warp writes runs of a row.  Every lane takes part.
template <int CW>
__device__ __forceinline__ void linear_store_any(const LinearArgs& p, float* stage, const float* acc, int t0, int c0) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < CW; ++j) stage[lane * (CW + 1) + j] = acc[j];
    __syncwarp();
    for (int i = lane; i < 32 * CW; i += 32) {
        const int t = t0 + i / CW, c = c0 + i % CW;
        if (t < p.T && c < p.N) {
            float v = stage[(i / CW) * (CW + 1) + i % CW];
            if (p.bias) v += __bfloat162float(p.bias[c]);
            v = linear_act(v, p.act);
            const size_t at = static_cast<size_t>(t) * p.N + c;
            if (p.res) v += __bfloat162float(p.res[at]);
            p.y[at] = __float2bfloat16_rn(v);
        }
    }
}

}  // namespace moe
