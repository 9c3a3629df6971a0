// balance.cu -- what a router is trained with: the balance loss with its per-expert counts
// (moe_balance_loss), and the gradient of the router logits from the routing weights and from that
// loss (moe_route_backward).
//
//   p[t, e]  = softmax(logits[t])  or  sigmoid(logits[t, e]) / sum_j sigmoid(logits[t, j])
//   f[s, e]  = E / (k n_s) * counts[s, e],   P[s, e] = mean of p[t, e] over the n_s counted tokens
//   loss     = coef / S' * sum over the S' sequences with n_s > 0 of  sum_e f[s, e] P[s, e]
// f does not depend on the logits, so d loss / d p[t, e] = coef * dloss / S' * f[s, e] / n_s, the same
// for every token of a sequence.
//
// Bound: one read of the logits (and one write of their gradient).  Sums are fp32 in registers, then
// per block and chunk in a fixed order without atomics on floats, so a result is the same on every
// run.
#include <math.h>

#include "block_kernels.h"
#include "moe_common.cuh"

namespace moe {

namespace {

constexpr int kWarps = 32;

// Sequence s's first token (s <= S), kept inside [0, T].
__device__ __forceinline__ int seq_at(const int32_t* off, int S, int T, int s) {
    if (!off) return s == 0 ? 0 : T;
    return min(max(__ldg(off + s), 0), T);
}

// The first sequence that ends behind token t (S if none does).
__device__ __forceinline__ int seq_after(const int32_t* off, int S, int T, int t) {
    int lo = 0, hi = S;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (seq_at(off, S, T, mid + 1) > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// A token's probabilities, NE experts a lane (expert lane + 32 i; past E: 0).
template <int NE>
__device__ __forceinline__ void probs(const float* row, int E, int routing, int lane, float (&p)[NE]) {
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) p[i] = lane + 32 * i < E ? __ldg(row + lane + 32 * i) : -INFINITY;
    if (routing == 0) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NE; ++i) m = fmaxf(m, p[i]);
        m = warp_max(m);
#pragma unroll
        for (int i = 0; i < NE; ++i) z += (p[i] = expf(p[i] - m));
    } else {
#pragma unroll
        for (int i = 0; i < NE; ++i) z += (p[i] = 1.0f / (1.0f + expf(-p[i])));
    }
    z = 1.0f / warp_sum(z);
#pragma unroll
    for (int i = 0; i < NE; ++i) p[i] *= z;
}

}  // namespace

// Block c takes the tokens of chunk c, sequence by sequence: a warp a token, the sums of p in
// registers, then over the warps in order.
template <int NE>
__global__ void __launch_bounds__(kWarps * 32) k_balance(BalanceArgs a) {
    __shared__ float s_p[kWarps][32 * NE];
    __shared__ int s_n[32 * NE + 2];                   // counts, counted tokens, ids out of range
    pdl_wait_then_release();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *a.status = MOE_OK;
        *a.ticket = 0;
    }
    const int c0 = blockIdx.x * a.chunk, c1 = min(a.T, c0 + a.chunk);
    for (int s = seq_after(a.off, a.S, a.T, c0); s < a.S; ++s) {
        const int b0 = max(c0, seq_at(a.off, a.S, a.T, s)), b1 = min(c1, seq_at(a.off, a.S, a.T, s + 1));
        if (seq_at(a.off, a.S, a.T, s) >= c1) break;
        if (b0 >= b1) continue;
        for (int e = threadIdx.x; e < a.E + 2; e += blockDim.x) s_n[e] = 0;
        __syncthreads();
        float acc[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) acc[i] = 0.0f;
        int counted = 0;
        for (int t = b0 + warp; t < b1; t += kWarps) {
            if (a.mask && !__ldg(a.mask + t)) continue;
            ++counted;
            float p[NE];
            probs<NE>(a.logits + static_cast<size_t>(t) * a.E, a.E, a.routing, lane, p);
#pragma unroll
            for (int i = 0; i < NE; ++i) acc[i] += p[i];
            for (int j = lane; j < a.K; j += 32) {
                const int e = __ldg(a.idx + static_cast<size_t>(t) * a.K + j);
                atomicAdd(&s_n[e >= 0 && e < a.E ? e : a.E + 1], 1);
            }
        }
        if (lane == 0 && counted) atomicAdd(&s_n[a.E], counted);
#pragma unroll
        for (int i = 0; i < NE; ++i) s_p[warp][lane + 32 * i] = acc[i];
        __syncthreads();
        const size_t slot = static_cast<size_t>(blockIdx.x) + s;
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
            float v = 0.0f;
            for (int w = 0; w < kWarps; ++w) v += s_p[w][e];
            a.part_p[slot * a.E + e] = v;
        }
        for (int e = threadIdx.x; e < a.E + 2; e += blockDim.x) a.part_n[slot * (a.E + 2) + e] = s_n[e];
        __syncthreads();
    }
}

// Block s joins sequence s's chunks in order; the last block to finish adds the sequences' losses.
__global__ void __launch_bounds__(1024) k_balance_join(BalanceArgs a) {
    __shared__ float s_p[1024];
    __shared__ int s_n[1024], s_tok, s_bad, s_last;
    __shared__ float s_red[32];
    pdl_wait_then_release();
    const int s = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E2 = (a.E + 31) & ~31, groups = 1024 / E2;
    const int g = threadIdx.x / E2, e = threadIdx.x % E2;
    const int b0 = seq_at(a.off, a.S, a.T, s), b1 = seq_at(a.off, a.S, a.T, s + 1);
    if (threadIdx.x == 0) {
        s_tok = 0, s_bad = 0;
        if (a.off) {
            const int o0 = a.off[s], o1 = a.off[s + 1];
            if (o0 < 0 || o1 > a.T || o0 > o1) s_bad = 1;
        }
    }
    __syncthreads();
    const int lo = b0 / a.chunk, hi = b0 < b1 ? (b1 - 1) / a.chunk : lo - 1;
    float v = 0.0f;
    int n = 0;
    if (g < groups && e < a.E)
        for (int c = lo + g; c <= hi; c += groups) {
            const size_t slot = static_cast<size_t>(c) + s;
            v += __ldcg(a.part_p + slot * a.E + e);
            n += __ldcg(a.part_n + slot * (a.E + 2) + e);
        }
    s_p[threadIdx.x] = v;
    s_n[threadIdx.x] = n;
    if (warp == 0) {
        int tok = 0, bad = 0;
        for (int c = lo + lane; c <= hi; c += 32) {
            const int32_t* q = a.part_n + (static_cast<size_t>(c) + s) * (a.E + 2) + a.E;
            tok += __ldcg(q);
            bad |= __ldcg(q + 1);
        }
        tok = __reduce_add_sync(0xffffffffu, tok);
        bad = __reduce_or_sync(0xffffffffu, bad);
        if (lane == 0) {
            s_tok = tok;
            s_bad |= bad;
        }
    }
    __syncthreads();
    const int tok = s_tok;
    float term = 0.0f;
    if (g == 0 && e < a.E) {
        for (int q = 1; q < groups; ++q) {
            v += s_p[q * E2 + e];
            n += s_n[q * E2 + e];
        }
        const float mean = tok ? v / static_cast<float>(tok) : 0.0f;
        a.mean[static_cast<size_t>(s) * a.E + e] = mean;
        a.counts[static_cast<size_t>(s) * a.E + e] = n;
        if (tok) term = static_cast<float>(n) * (static_cast<float>(a.E) / (static_cast<float>(a.K) * tok)) * mean;
    }
    term = warp_sum(term);
    if (lane == 0) s_red[warp] = term;
    __syncthreads();
    if (threadIdx.x == 0) {
        float l = 0.0f;
        for (int w = 0; w < 32; ++w) l += s_red[w];
        a.seq_loss[s] = l;
        a.tokens[s] = tok;
        if (s_bad) set_status(a.status, MOE_ERR_BOUNDS);
        __threadfence();
        s_last = atomicAdd(a.ticket, 1) == a.S - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    float l = 0.0f;
    int full = 0;
    for (int i = threadIdx.x; i < a.S; i += 1024) {
        l += __ldcg(a.seq_loss + i);
        full += __ldcg(a.tokens + i) > 0;
    }
    l = warp_sum(l);
    full = __reduce_add_sync(0xffffffffu, full);
    if (lane == 0) {
        s_red[warp] = l;
        s_n[warp] = full;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        l = 0.0f;
        full = 0;
        for (int w = 0; w < 32; ++w) {
            l += s_red[w];
            full += s_n[w];
        }
        a.tokens[a.S] = full;
        a.loss[0] = full ? a.coef * (l / static_cast<float>(full)) : 0.0f;
    }
}

// ------------------------------------------------------------------------------------------
// A warp a token.  With s = the probabilities' sum Z, u_j the routing weight before its scales and
// du_j = dw_j * rsf * per_expert_scale[e_j]:
//   softmax:              dl = p (dp - sum p dp)   with dp[e_j] += du_j
//   softmax, renormalized: dl = p (dp - sum p dp),  dl[e_j] += u_j (du_j - sum u du)
//   sigmoid s:            dl = s (1 - s) ds,  ds = (dp - sum p dp) / Z,  ds[e_j] += (du_j - sum u du) / sum s[e_j]
template <int NE>
__global__ void __launch_bounds__(kWarps * 32) k_route_backward(RouteBackwardArgs a) {
    extern __shared__ float s_mem[];                   // [kWarps][E] additions, then [kWarps][E] sums of dpes
    pdl_wait_then_release();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* add = s_mem + warp * a.E;
    float* dpes = s_mem + (kWarps + warp) * a.E;
    for (int e = lane; e < a.E; e += 32) {
        add[e] = 0.0f;
        if (a.dpes) dpes[e] = 0.0f;
    }
    __syncwarp();
    const int c0 = blockIdx.x * a.chunk, c1 = min(a.T, c0 + a.chunk);
    const float gl = a.dloss ? __ldg(a.dloss) * a.coef : 0.0f;
    int s = -1, s_lo = 0, s_hi = 0;                    // the sequence whose gradient is in g
    float g[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) g[i] = 0.0f;
    for (int t = c0 + warp; t < c1; t += kWarps) {
        bool bal = a.dloss && !(a.mask && !__ldg(a.mask + t));
        if (bal && !(s >= 0 && t >= s_lo && t < s_hi)) {
            const int q = seq_after(a.off, a.S, a.T, t);
            if (q < a.S && seq_at(a.off, a.S, a.T, q) <= t) {
                s = q;
                s_lo = seq_at(a.off, a.S, a.T, q);
                s_hi = seq_at(a.off, a.S, a.T, q + 1);
                const float n = static_cast<float>(__ldg(a.tokens + q)), full = static_cast<float>(__ldg(a.tokens + a.S));
                const float f = n > 0.0f ? gl / full * static_cast<float>(a.E) / (static_cast<float>(a.K) * n * n) : 0.0f;
#pragma unroll
                for (int i = 0; i < NE; ++i)
                    g[i] = lane + 32 * i < a.E
                               ? f * static_cast<float>(__ldg(a.counts + static_cast<size_t>(q) * a.E + lane + 32 * i))
                               : 0.0f;
            } else {
                bal = false;
            }
        }
        const float* row = a.logits + static_cast<size_t>(t) * a.E;
        const int32_t* idx = a.idx + static_cast<size_t>(t) * a.K;
        const float* dw = a.dw ? a.dw + static_cast<size_t>(t) * a.K : nullptr;
        // ---- the routing weights (a row without any gradient stays out: its logits may be anything)
        bool wts = false;
        if (dw) {
            bool nz = false;
            for (int j = lane; j < a.K; j += 32) nz |= __ldg(dw + j) != 0.0f;
            wts = __any_sync(0xffffffffu, nz);
        }
        float m = -INFINITY, z = 1.0f;                 // softmax of the whole row
        if (a.routing == 0 && (bal || (wts && !a.renorm))) {
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (lane + 32 * i < a.E) m = fmaxf(m, __ldg(row + lane + 32 * i));
            m = warp_max(m);
            z = 0.0f;
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (lane + 32 * i < a.E) z += expf(__ldg(row + lane + 32 * i) - m);
            z = warp_sum(z);
        }
        const bool norm = a.routing == 1 || a.renorm;
        if (wts) {
            float sm = -INFINITY, sz = 0.0f, sd = 0.0f;
            if (a.routing == 0 && norm) {
                for (int j = lane; j < a.K; j += 32) {
                    const int e = __ldg(idx + j);
                    if (e >= 0 && e < a.E) sm = fmaxf(sm, __ldg(row + e));
                }
                sm = warp_max(sm);
            }
            auto raw = [&](int e) {                    // the weight before the normalization
                const float l = __ldg(row + e);
                return a.routing == 1 ? 1.0f / (1.0f + expf(-l)) : norm ? expf(l - sm) : expf(l - m) / z;
            };
            if (norm) {
                for (int j = lane; j < a.K; j += 32) {
                    const int e = __ldg(idx + j);
                    if (e < 0 || e >= a.E) continue;
                    const float v = raw(e);
                    sz += v;
                    sd += v * (__ldg(dw + j) * a.rsf * (a.pes ? __ldg(a.pes + e) : 1.0f));
                }
                sz = warp_sum(sz);
                sd = warp_sum(sd) / sz;
            } else {
                sz = 1.0f;
            }
            for (int j = lane; j < a.K; j += 32) {
                const int e = __ldg(idx + j);
                if (e < 0 || e >= a.E) continue;
                const float d = __ldg(dw + j) * a.rsf, du = d * (a.pes ? __ldg(a.pes + e) : 1.0f);
                const float u = raw(e) / sz;
                atomicAdd(&add[e], !norm ? du : a.routing == 1 ? (du - sd) / sz : u * (du - sd));
                if (a.dpes) atomicAdd(&dpes[e], d * u);
            }
            __syncwarp();
        }
        // ---- the row's gradient
        float* out = a.dl + static_cast<size_t>(t) * a.E;
        if (!bal && !wts) {
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (lane + 32 * i < a.E) out[lane + 32 * i] = 0.0f;
            continue;
        }
        const bool direct = a.routing == 0 && !norm;   // the weights' gradient goes through the softmax
        float p[NE], d[NE], zs = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = lane + 32 * i;
            p[i] = 0.0f, d[i] = 0.0f;
            if (e >= a.E) continue;
            const float l = __ldg(row + e);
            p[i] = a.routing == 1 ? 1.0f / (1.0f + expf(-l)) : (bal || direct) ? expf(l - m) / z : 0.0f;
            d[i] = (bal ? g[i] : 0.0f) + (direct && wts ? add[e] : 0.0f);
            zs += p[i];
            dot = fmaf(p[i], d[i], dot);
        }
        dot = warp_sum(dot);
        if (a.routing == 1) {
            zs = warp_sum(zs);
            dot /= zs;
        }
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = lane + 32 * i;
            if (e >= a.E) continue;
            const float x = wts && !direct ? add[e] : 0.0f;
            float v;
            if (a.routing == 1) {
                const float l = __ldg(row + e);
                v = p[i] * (1.0f / (1.0f + expf(l))) * ((bal ? (d[i] - dot) / zs : 0.0f) + x);
            } else {
                v = fmaf(p[i], d[i] - dot, x);
            }
            out[e] = v;
        }
        __syncwarp();
        if (wts) {                                     // back to zero for the next token
            for (int j = lane; j < a.K; j += 32) {
                const int e = __ldg(idx + j);
                if (e >= 0 && e < a.E) add[e] = 0.0f;
            }
            __syncwarp();
        }
    }
    if (!a.dpes) return;
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        float v = 0.0f;
        for (int w = 0; w < kWarps; ++w) v += s_mem[(kWarps + w) * a.E + e];
        a.part[static_cast<size_t>(blockIdx.x) * a.E + e] = v;
    }
}

__global__ void __launch_bounds__(256) k_join_scale_grad(RouteBackwardArgs a) {
    pdl_wait_then_release();
    const int e = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (e >= a.E) return;
    float v = 0.0f;
    for (int c = lane; c < a.chunks; c += 32) v += __ldcg(a.part + static_cast<size_t>(c) * a.E + e);
    v = warp_sum(v);
    if (lane == 0) a.dpes[e] = v;
}

template <int NE>
static cudaError_t launch_backward_t(const RouteBackwardArgs& a, cudaStream_t s) {
    const size_t smem = static_cast<size_t>(kWarps) * a.E * 4 * (a.dpes ? 2 : 1);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k_route_backward<NE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(k_route_backward<NE>, dim3(a.chunks), dim3(kWarps * 32), smem, s, a);
}

cudaError_t launch_balance(const BalanceArgs& a, cudaStream_t s) {
    const int ne = (a.E + 31) / 32;
    const dim3 grid(a.chunks), block(kWarps * 32);
    const cudaError_t e = ne <= 1   ? launch_pdl(k_balance<1>, grid, block, 0, s, a)
                          : ne <= 2 ? launch_pdl(k_balance<2>, grid, block, 0, s, a)
                          : ne <= 4 ? launch_pdl(k_balance<4>, grid, block, 0, s, a)
                                    : launch_pdl(k_balance<8>, grid, block, 0, s, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_balance_join, dim3(a.S), dim3(1024), 0, s, a);
}

cudaError_t launch_route_backward(const RouteBackwardArgs& a, cudaStream_t s) {
    const int ne = (a.E + 31) / 32;
    const cudaError_t e = ne <= 1   ? launch_backward_t<1>(a, s)
                          : ne <= 2 ? launch_backward_t<2>(a, s)
                          : ne <= 4 ? launch_backward_t<4>(a, s)
                                    : launch_backward_t<8>(a, s);
    if (e != cudaSuccess || !a.dpes) return e;
    return launch_pdl(k_join_scale_grad, dim3((a.E + 7) / 8), dim3(256), 0, s, a);
}

}  // namespace moe
