// norm.cu -- what stands in front of the layer and of a dense product: the residual addition with
// the RMS norm, and the 8-bit codes and scales of its result (moe_add_rms_norm); and the codes and
// scales of bf16 rows as they are (the first launch of moe_linear on bf16 input).
//
//   h = x + residual (fp32),  r = 1 / sqrt(mean_h h^2 + eps),  y = h * r * w
//   recipe 0:    s = amax * (1/448) per 128 columns, q = e4m3(y / s); s 0 -> 1
//   recipes 1, 2: s = 2^e per 32 columns, e the smallest with amax <= 448 * 2^e; q = e4m3(y * 2^-e)
// Scales are stored as every GEMM of the library reads them: [H/128][scale_rows] 4-byte words.
//
// Bound: HBM, each row read once and each output written once.  In a graph: 16384 x 4096 with a bf16 residual and
// fp32 scales (606 MB) 102 us, 5.9 TB/s; 4096 x 7168 with an fp32 residual and MXFP8 (383 MB) 71 us, 5.4 TB/s; a copy
// reaches 6.5.  64 x 2816 takes 3 us, the latency of a launch, a load, the sum over the block and a store.
#include "block_kernels.h"
#include "moe_common.cuh"

namespace moe {

namespace {

__device__ __forceinline__ void unpack8(uint4 raw, float* v) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight fp32 values in one 32-byte access (p 32-byte aligned): a whole sector a lane.
__device__ __forceinline__ void load8_f32(const float* p, float* v) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]) : "l"(p));
}
__device__ __forceinline__ void store8_f32(float* p, const float* v) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

__device__ __forceinline__ float absmax8(const float* v) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
    return m;
}

__device__ __forceinline__ uint2 codes8(const float* v) {
    return make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
}

// Sixteen lanes hold the 128 columns of one scale block, eight columns each; their maximum.
__device__ __forceinline__ float group16_max(float m) {
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// fp32 scale of a block with maximum amax, and its codes.  The scale is amax times the rounded 1/448,
// as a torch program on the GPU computes amax / 448.0, so that its codes are these; the layer's own
// quantizer divides, which can differ by one ulp of the scale.
// v / s is v times the reciprocal of s and the reciprocal's own remainder, v ih + v il: within 2^-46 of the
// quotient before its one rounding (16384 x 4096: 108 us in calls, 117 with a division).
__device__ __forceinline__ uint2 quant_fp32(const float* v, float amax, float& s) {
    s = __fmul_rn(amax, 1.0f / 448.0f);
    if (!(s > 0.0f)) s = 1.0f;                         // nothing, or less than the smallest scale: codes of zero
    float q[8];
    if (s > 1e-30f && s < 1e30f) {                     // the reciprocal and its remainder are normal numbers
        const float ih = __frcp_rn(s), il = fmaf(-ih, s, 1.0f) * ih;
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = fmaf(v[i], ih, v[i] * il);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(v[i], s);
    }
    return codes8(q);
}

// UE8M0 scales: four lanes hold a 32-column group.  Returns the codes; word = the four scale bytes
// of the lane's 128-column block, lowest group in the lowest byte (equal in its sixteen lanes).
// An infinity, which the conversion would make 448, is multiplied by zero: its code is NaN, as with an
// fp32 scale, and the finite columns of its group are zero.
__device__ __forceinline__ uint2 quant_mx(const float* v, uint32_t& word) {
    float m = absmax8(v);
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int e = mx_exponent(m);
    const float inv = m < INFINITY ? exp2_int(-e) : 0.0f;
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = v[i] * inv;
    const int lane = threadIdx.x & 31;
    word = static_cast<uint32_t>(e + 127) << (8 * ((lane >> 2) & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    return codes8(q);
}

}  // namespace

// ------------------------------------------------------------------------------------------
// TPR threads a row (a multiple of 32), CH chunks of eight columns a thread, so that the row stays
// in registers between the sum and the scaling and is read once.  Rows of a block are independent.
// The thread count and the chunks follow from H alone, and the sum is taken in a fixed order: a
// row's bits do not depend on the batch.  RES: 0 no residual, 1 bf16, 2 fp32.
template <int CH, int RES, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 6 : MAXT == 512 ? 3 : 1) k_add_rms_norm(NormArgs a) {
    __shared__ float s_sum[32];
    pdl_wait_then_release();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int wpr = a.tpr >> 5;                        // warps per row
    const int sub = warp / wpr;                        // row of the block
    const long long t = static_cast<long long>(blockIdx.x) * (blockDim.x / a.tpr) + sub;
    const int rt = tid - sub * a.tpr;                  // thread of the row
    const bool row_ok = t < a.T;
    const size_t base = static_cast<size_t>(row_ok ? t : 0) * a.H;

    float h[CH][8];
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = (c * a.tpr + rt) * 8;
        if (row_ok && col < a.H) {
            unpack8(*reinterpret_cast<const uint4*>(a.x + base + col), h[c]);
            if (RES == 1) {
                float r[8];
                unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.res) + base + col), r);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[c][i] += r[i];
            } else if (RES == 2) {
                float r[8];
                load8_f32(static_cast<const float*>(a.res) + base + col, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[c][i] += r[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) h[c][i] = 0.0f;
        }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(h[c][i], h[c][i], ss);
    ss = warp_sum(ss);
    if (lane == 0) s_sum[warp] = ss;
    __syncthreads();
    float tot = 0.0f;
    for (int w = 0; w < wpr; ++w) tot += s_sum[sub * wpr + w];
    const float r = 1.0f / sqrtf(tot / static_cast<float>(a.H) + a.eps);

#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = (c * a.tpr + rt) * 8;
        const bool ok = row_ok && col < a.H;
        if (RES == 1 && ok && a.res_out)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.res_out) + base + col) = pack8(h[c]);
        if (RES == 2 && ok && a.res_out) store8_f32(static_cast<float*>(a.res_out) + base + col, h[c]);
        float y[8];
        float4 w0 = make_float4(0.f, 0.f, 0.f, 0.f), w1 = w0;
        if (ok) {
            w0 = __ldg(reinterpret_cast<const float4*>(a.w + col));
            w1 = __ldg(reinterpret_cast<const float4*>(a.w + col) + 1);
        }
        const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = h[c][i] * r * w[i];
        if (ok && a.y) *reinterpret_cast<uint4*>(a.y + base + col) = pack8(y);
        if (!a.xq) continue;
        uint2 q;
        uint32_t word;
        if (a.recipe == 0) {
            float s;
            q = quant_fp32(y, group16_max(absmax8(y)), s);
            word = __float_as_uint(s);
        } else {
            q = quant_mx(y, word);
        }
        if (ok) {
            *reinterpret_cast<uint2*>(a.xq + base + col) = q;
            if ((lane & 15) == 0) a.xs[static_cast<size_t>(col >> 7) * a.a_pad + t] = word;
        }
    }
}

// The codes and scales of bf16 rows: a thread takes eight columns at two places, both loads first (4096 x 7168 in
// 18.7 us, 4.7 TB/s).
// Clears the status word of the call (its first kernel).
__global__ void __launch_bounds__(256) k_quant_rows(QuantRowsArgs a) {
    pdl_wait_then_release();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = MOE_OK;
    const int per_row = a.K >> 3;                      // a multiple of 16: a scale block stays in a half warp
    const long long n = static_cast<long long>(a.T) * per_row;
    const long long i0 = static_cast<long long>(blockIdx.x) * 512 + threadIdx.x;
    uint4 raw[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const long long i = i0 + 256 * h;
        raw[h] = i < n ? __ldg(reinterpret_cast<const uint4*>(a.x) + i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const long long i = i0 + 256 * h;
        float v[8];
        unpack8(raw[h], v);
        uint2 q;
        uint32_t word;
        if (a.recipe == 0) {
            float s;
            q = quant_fp32(v, group16_max(absmax8(v)), s);
            word = __float_as_uint(s);
        } else {
            q = quant_mx(v, word);
        }
        if (i >= n) continue;
        reinterpret_cast<uint2*>(a.xq)[i] = q;
        if ((threadIdx.x & 15) == 0) {
            const int t = static_cast<int>(i / per_row), blk = static_cast<int>(i - static_cast<long long>(t) * per_row) >> 4;
            a.xs[static_cast<size_t>(blk) * a.a_pad + t] = word;
        }
    }
}

template <int CH, int MAXT>
static cudaError_t launch_norm_ch(const NormArgs& a, int rows, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((a.T + rows - 1) / rows)), block(a.tpr * rows);
    if (!a.res) return launch_pdl(k_add_rms_norm<CH, 0, MAXT>, grid, block, 0, s, a);
    return a.res_fp32 ? launch_pdl(k_add_rms_norm<CH, 2, MAXT>, grid, block, 0, s, a)
                      : launch_pdl(k_add_rms_norm<CH, 1, MAXT>, grid, block, 0, s, a);
}

cudaError_t launch_add_rms_norm(NormArgs a, cudaStream_t s) {
    // Two chunks of eight columns a thread up to 512 threads a row (one where 256 do, four for the longest rows);
    // short rows share a block of 256.  Measured at 4096 x 7168: 54 us, with four chunks in 224 threads 58; at
    // 16384 x 4096: 101 us, with one chunk in 512 threads 126 (a thread's loads in flight halve; at 64 rows that
    // takes 2.7 us against 3.2, but the choice follows from H alone, so that a row's bits are the same in any batch).
    const int chunks = a.H / 8;
    const int ch = chunks <= 256 ? 1 : chunks <= 1024 ? 2 : 4;
    a.tpr = ((chunks + ch - 1) / ch + 31) / 32 * 32;
    const int rows = a.tpr >= 256 ? 1 : 256 / a.tpr;
    if (ch == 4) return launch_norm_ch<4, 1024>(a, rows, s);
    if (a.tpr > 256) return launch_norm_ch<2, 512>(a, rows, s);
    return ch == 1 ? launch_norm_ch<1, 256>(a, rows, s) : launch_norm_ch<2, 256>(a, rows, s);
}

cudaError_t launch_quant_rows(const QuantRowsArgs& a, cudaStream_t s) {
    const long long n = static_cast<long long>(a.T) * (a.K >> 3);
    return launch_pdl(k_quant_rows, dim3(static_cast<unsigned>((n + 511) / 512)), dim3(256), 0, s, a);
}

}  // namespace moe
