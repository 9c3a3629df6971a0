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
// Bound: one read of the logits (and one write of their gradient).  A token is taken by G = 8 lanes
// (16 above 128 experts) with up to 16 experts each, so that a warp works on four tokens (two) at
// once and a sum over a row takes three shuffles (four) for all of them.  Sums are fp32 in
// registers, then per block and chunk in a fixed order without atomics on floats, so a result is the
// same on every run.
#include <math.h>

#include "block_kernels.h"
#include "moe_common.cuh"

namespace moe {

namespace {

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

// A row of E values over G lanes, NE a lane: four neighbours at a time (VEC: E a multiple of 4 and
// 16-byte rows), or every G-th.
template <int NE, int G, bool VEC>
struct Row {
    static __device__ __forceinline__ int expert(int i, int gl) {
        return VEC ? (i >> 2) * (4 * G) + gl * 4 + (i & 3) : i * G + gl;
    }
    template <typename T4, typename T>
    static __device__ __forceinline__ void load(const T* row, int E, int gl, bool ok, T (&v)[NE], T fill) {
        if (VEC) {
#pragma unroll
            for (int i = 0; i < NE; i += 4) {
                const int e = expert(i, gl);
                if (ok && e < E) {
                    const T4 x = __ldg(reinterpret_cast<const T4*>(row + e));
                    v[i] = x.x, v[i + 1] = x.y, v[i + 2] = x.z, v[i + 3] = x.w;
                } else {
                    v[i] = v[i + 1] = v[i + 2] = v[i + 3] = fill;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i) v[i] = ok && expert(i, gl) < E ? __ldg(row + expert(i, gl)) : fill;
        }
    }
    static __device__ __forceinline__ void store(float* row, int E, int gl, const float (&v)[NE]) {
        if (VEC) {
#pragma unroll
            for (int i = 0; i < NE; i += 4)
                if (expert(i, gl) < E)
                    *reinterpret_cast<float4*>(row + expert(i, gl)) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (expert(i, gl) < E) row[expert(i, gl)] = v[i];
        }
    }
};

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = 1; o < G; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = 1; o < G; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// e^x for x <= 0 as 2^(x log2 e): the product's rounding makes its relative error up to |x| 2^-24, under
// 2e-6 wherever e^x is above 1e-12, in two instructions against expf's eight.
__device__ __forceinline__ float exp_neg(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504f));
    return y;
}

// sigmoid(l) and sigmoid(l) (1 - sigmoid(l)) from t = e^-|l| in (0, 1]: neither overflows, and the
// second does not lose its digits where the first is near 1.
__device__ __forceinline__ float sigmoid(float l, float& slope) {
    const float t = exp_neg(-fabsf(l)), r = __frcp_rn(1.0f + t);
    slope = t * r * r;
    return l >= 0.0f ? r : t * r;                      // NaN: t is NaN
}

// v[i]: the logits (-inf past E) in, the probabilities out.  Every lane of the warp calls it.
template <int NE, int G, bool SIG>
__device__ __forceinline__ void row_probs(float (&v)[NE]) {
    float z = 0.0f;
    if (SIG) {
        float slope;
#pragma unroll
        for (int i = 0; i < NE; ++i) z += (v[i] = sigmoid(v[i], slope));   // -inf past E: 0
    } else {
        float m = v[0];
#pragma unroll
        for (int i = 1; i < NE; ++i) m = fmaxf(m, v[i]);
        m = group_max<G>(m);
#pragma unroll
        for (int i = 0; i < NE; ++i) z += (v[i] = exp_neg(v[i] - m));
    }
    z = 1.0f / group_sum<G>(z);
#pragma unroll
    for (int i = 0; i < NE; ++i) v[i] *= z;
}

constexpr int kBWarps = 32;                            // k_balance
constexpr int kRWarps = 8;                             // k_route_backward

}  // namespace

// Block c takes the tokens of chunk c, sequence by sequence; the sums of p stay in registers and are
// joined over the lanes and warps in order at a sequence's end.
template <int NE, int G, bool VEC, bool SIG>
__global__ void __launch_bounds__(kBWarps * 32) k_balance(BalanceArgs a) {
    using R = Row<NE, G, VEC>;
    constexpr int TPW = 32 / G, W = NE * G;
    __shared__ float s_p[kBWarps][W];
    __shared__ int s_n[W + 2];                         // counts, counted tokens, ids out of range
    pdl_wait_then_release();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gl = lane % G;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *a.status = MOE_OK;
        *a.ticket = 0;
    }
    const int c0 = blockIdx.x * a.chunk, c1 = min(a.T, c0 + a.chunk);
    for (int s = seq_after(a.off, a.S, a.T, c0); s < a.S; ++s) {
        const int s0 = seq_at(a.off, a.S, a.T, s);
        if (s0 >= c1) break;
        const int b0 = max(c0, s0), b1 = min(c1, seq_at(a.off, a.S, a.T, s + 1));
        if (b0 >= b1) continue;
        const int warps = min(kBWarps, (b1 - b0 + TPW - 1) / TPW);   // warps with a token
        for (int e = threadIdx.x; e < a.E + 2; e += blockDim.x) s_n[e] = 0;
        __syncthreads();
        if (warp < warps) {
            float acc[NE];
#pragma unroll
            for (int i = 0; i < NE; ++i) acc[i] = 0.0f;
            for (int tb = b0 + warp * TPW; tb < b1; tb += kBWarps * TPW) {
                const int t = tb + lane / G;
                const bool ok = t < b1 && !(a.mask && !__ldg(a.mask + t));
                float p[NE];
                R::template load<float4>(a.logits + static_cast<size_t>(ok ? t : 0) * a.E, a.E, gl, ok, p, -INFINITY);
                if (ok) {
                    for (int j = gl; j < a.K; j += G) {
                        const int e = __ldg(a.idx + static_cast<size_t>(t) * a.K + j);
                        atomicAdd(&s_n[e >= 0 && e < a.E ? e : a.E + 1], 1);
                    }
                    if (gl == 0) atomicAdd(&s_n[a.E], 1);
                }
                row_probs<NE, G, SIG>(p);
#pragma unroll
                for (int i = 0; i < NE; ++i) acc[i] += ok ? p[i] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < NE; ++i) {
#pragma unroll
                for (int o = G; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
                if (lane < G) s_p[warp][R::expert(i, gl)] = acc[i];
            }
        }
        __syncthreads();
        const size_t slot = static_cast<size_t>(blockIdx.x) + s;
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
            float v = 0.0f;
            for (int w = 0; w < warps; ++w) v += s_p[w][e];
            a.part_p[slot * a.E + e] = v;
        }
        for (int e = threadIdx.x; e < a.E + 2; e += blockDim.x) a.part_n[slot * (a.E + 2) + e] = s_n[e];
        __syncthreads();
    }
}

// Block (s, b) joins sequence s's chunks for experts 32 b .. 32 b + 31: a lane an expert, a warp every
// 32nd chunk, then the warps in order.  The last block to finish adds the losses.
__global__ void __launch_bounds__(1024) k_balance_join(BalanceArgs a) {
    __shared__ float s_p[32][33];
    __shared__ int s_n[32][33], s_tok[32], s_bad, s_last;
    __shared__ float s_red[32];
    pdl_wait_then_release();
    const int s = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = blockIdx.y * 32 + lane;
    const int b0 = seq_at(a.off, a.S, a.T, s), b1 = seq_at(a.off, a.S, a.T, s + 1);
    if (threadIdx.x == 0) s_bad = a.off && (a.off[s] < 0 || a.off[s + 1] > a.T || a.off[s] > a.off[s + 1]);
    __syncthreads();
    const int lo = b0 / a.chunk, hi = b0 < b1 ? (b1 - 1) / a.chunk : lo - 1;
    float v = 0.0f;
    int n = 0, tok = 0, bad = 0;
#pragma unroll 4
    for (int c = lo + warp; c <= hi; c += 32) {
        const size_t slot = static_cast<size_t>(c) + s;
        const int32_t* cnt = a.part_n + slot * (a.E + 2);
        if (e < a.E) {
            v += __ldcg(a.part_p + slot * a.E + e);
            n += __ldcg(cnt + e);
        }
        tok += __ldcg(cnt + a.E);                      // one address for the warp
        bad |= __ldcg(cnt + a.E + 1);
    }
    s_p[warp][lane] = v;
    s_n[warp][lane] = n;
    if (lane == 0) {
        s_tok[warp] = tok;
        if (bad) s_bad = 1;
    }
    __syncthreads();
    if (warp == 0) {
        tok = __reduce_add_sync(0xffffffffu, s_tok[lane]);
        v = 0.0f;
        n = 0;
        for (int w = 0; w < 32; ++w) {
            v += s_p[w][lane];
            n += s_n[w][lane];
        }
        float term = 0.0f;
        if (e < a.E) {
            const float mean = tok ? v / static_cast<float>(tok) : 0.0f;
            a.mean[static_cast<size_t>(s) * a.E + e] = mean;
            a.counts[static_cast<size_t>(s) * a.E + e] = n;
            if (tok)
                term = static_cast<float>(n) * (static_cast<float>(a.E) / (static_cast<float>(a.K) * static_cast<float>(tok))) * mean;
        }
        term = warp_sum(term);
        if (lane == 0) {
            a.seq_loss[static_cast<size_t>(s) * gridDim.y + blockIdx.y] = term;
            if (blockIdx.y == 0) a.tokens[s] = tok;
            if (s_bad) set_status(a.status, MOE_ERR_BOUNDS);
            __threadfence();
            s_last = atomicAdd(a.ticket, 1) == static_cast<int>(gridDim.x * gridDim.y) - 1;
        }
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    float l = 0.0f;
    int full = 0;
    for (int i = threadIdx.x; i < a.S * static_cast<int>(gridDim.y); i += 1024) l += __ldcg(a.seq_loss + i);
    for (int i = threadIdx.x; i < a.S; i += 1024) full += __ldcg(a.tokens + i) > 0;
    l = warp_sum(l);
    full = __reduce_add_sync(0xffffffffu, full);
    if (lane == 0) {
        s_red[warp] = l;
        s_tok[warp] = full;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        l = 0.0f;
        full = 0;
        for (int w = 0; w < 32; ++w) {
            l += s_red[w];
            full += s_tok[w];
        }
        a.tokens[a.S] = full;
        a.loss[0] = full ? a.coef * (l / static_cast<float>(full)) : 0.0f;
    }
}

// ------------------------------------------------------------------------------------------
// With Z the sum of the scores, u_j the routing weight before its scales, x_j = rsf * dw_j and
// du_j = x_j * per_expert_scale[e_j]:
//   softmax:               dl = p (dp - sum p dp)   with dp[e_j] += du_j
//   softmax, renormalized: dl = p (dp - sum p dp),  dl[e_j] += u_j (du_j - sum u du)
//   sigmoid s:             dl = s (1 - s) ds,  ds = (dp - sum p dp) / Z,  ds[e_j] += (du_j - sum u du) / sum_j s[e_j]
//   dscale[e] = sum over the tokens of x_j u_j
// The slots' terms reach the lanes that hold their experts through a row of shared memory.
enum { kDirect = 0, kRenorm = 1, kSigmoid = 2 };      // softmax, softmax renormalized, sigmoid

template <int NE, int G, bool VEC, int MODE>
__global__ void __launch_bounds__(kRWarps * 32) k_route_backward(RouteBackwardArgs a) {
    using R = Row<NE, G, VEC>;
    constexpr int TPW = 32 / G, W = NE * G;
    __shared__ __align__(16) float s_add[kRWarps * TPW][W];
    __shared__ float s_scale[kRWarps * TPW][W];        // a group's sums of dscale
    pdl_wait_then_release();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gl = lane % G, grp = lane / G;
    const unsigned group_mask = (G == 32 ? 0xffffffffu : (1u << G) - 1u) << (grp * G);
    float* add = s_add[warp * TPW + grp];
    float* dscale = s_scale[warp * TPW + grp];
    for (int e = gl; e < W; e += G) add[e] = dscale[e] = 0.0f;
    __syncwarp();
    const int c0 = blockIdx.x * a.chunk, c1 = min(a.T, c0 + a.chunk);
    const float gloss = a.dloss ? __ldg(a.dloss) * a.coef : 0.0f;
    int q = -1, q0 = 0, q1 = 0;                        // the sequence whose gradient is in g, its tokens
    float g[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) g[i] = 0.0f;
    for (int tb = c0 + warp * TPW; tb < c1; tb += kRWarps * TPW) {
        const int t = tb + grp;
        const bool in = t < c1;
        const size_t tr = static_cast<size_t>(in ? t : c0);
        const int32_t* idx = a.idx + tr * a.K;
        const float* dw = a.dw + tr * a.K;
        const float* row = a.logits + tr * a.E;
        // Every load first: the row and the lane's own slot (all there is when k <= G) do not wait for
        // what decides whether they are used.
        float p[NE], slope[NE];
        R::template load<float4>(row, a.E, gl, in, p, -INFINITY);
        int e0 = in && gl < a.K ? __ldg(idx + gl) : -1;
        float x0 = in && a.dw && gl < a.K ? __ldg(dw + gl) : 0.0f;
        bool bal = in && a.dloss && !(a.mask && !__ldg(a.mask + t));
        if (bal && !(t >= q0 && t < q1)) {             // another sequence than the last token's
            q = seq_after(a.off, a.S, a.T, t);
            q0 = seq_at(a.off, a.S, a.T, q);           // q = S: no sequence ends behind t
            q1 = q < a.S ? seq_at(a.off, a.S, a.T, q + 1) : 0;
            if (t >= q0 && t < q1) {
                const float n = static_cast<float>(__ldg(a.tokens + q)), full = static_cast<float>(__ldg(a.tokens + a.S));
                const float f = n > 0.0f ? gloss / full * static_cast<float>(a.E) / (static_cast<float>(a.K) * n * n) : 0.0f;
                int n_e[NE];
                R::template load<int4>(a.counts + static_cast<size_t>(q) * a.E, a.E, gl, true, n_e, 0);
#pragma unroll
                for (int i = 0; i < NE; ++i) g[i] = f * static_cast<float>(n_e[i]);
            } else {
                q1 = 0;                                // in no sequence: g is not this range's
            }
        }
        bal = bal && t >= q0 && t < q1;
        if (e0 >= a.E) e0 = -1;
        const float l0 = e0 >= 0 ? __ldg(row + e0) : -INFINITY;
        const float scale0 = e0 >= 0 && a.pes ? __ldg(a.pes + e0) : 1.0f;
        bool nz = x0 != 0.0f;                          // NaN counts
        if (in && a.dw)
            for (int j = gl + G; j < a.K; j += G) nz |= __ldg(dw + j) != 0.0f;
        const bool wts = __ballot_sync(0xffffffffu, nz) & group_mask;
        float z = 0.0f, m = -INFINITY;
        if (MODE == kSigmoid) {
#pragma unroll
            for (int i = 0; i < NE; ++i) z += (p[i] = sigmoid(p[i], slope[i]));
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i) m = fmaxf(m, p[i]);
            m = group_max<G>(m);
#pragma unroll
            for (int i = 0; i < NE; ++i) z += (p[i] = exp_neg(p[i] - m));
        }
        const float rz = 1.0f / group_sum<G>(z);       // p[i] stays unscaled: the probability is p[i] * rz

        // ---- the routing weights' terms (a token without them adds zeros)
        float sm = m;
        const bool more = wts && a.K > G;              // slots behind the lanes' first
        if (MODE == kRenorm) {
            float v = l0;
            if (more)
                for (int j = gl + G; j < a.K; j += G) {
                    const int e = __ldg(idx + j);
                    if (e >= 0 && e < a.E) v = fmaxf(v, __ldg(row + e));
                }
            sm = group_max<G>(v);
        }
        auto raw = [&](float l) {                      // the weight before the normalization
            float s;
            return MODE == kSigmoid ? sigmoid(l, s) : MODE == kRenorm ? exp_neg(l - sm) : exp_neg(l - m) * rz;
        };
        x0 *= a.rsf;
        const float v0 = e0 >= 0 ? raw(l0) : 0.0f, du0 = x0 * scale0;
        float sz = v0;
        if (more)
            for (int j = gl + G; j < a.K; j += G) {
                const int e = __ldg(idx + j);
                if (e >= 0 && e < a.E) sz += raw(__ldg(row + e));
            }
        // u = v / sz by division: a single slot has exactly u = 1 and no gradient through its weight
        sz = MODE == kDirect ? 1.0f : group_sum<G>(sz);
        auto weight = [&](float v) { return MODE == kDirect ? v : __fdiv_rn(v, sz); };
        const float u0 = weight(v0);
        float sd = 0.0f;
        if (MODE != kDirect) {
            sd = e0 >= 0 ? u0 * du0 : 0.0f;
            if (more)
                for (int j = gl + G; j < a.K; j += G) {
                    const int e = __ldg(idx + j);
                    if (e >= 0 && e < a.E)
                        sd += weight(raw(__ldg(row + e))) * (__ldg(dw + j) * a.rsf * (a.pes ? __ldg(a.pes + e) : 1.0f));
                }
            sd = group_sum<G>(sd);
        }
        auto term = [&](float u, float du) {           // what a slot adds to its expert
            return MODE == kDirect ? du : MODE == kSigmoid ? (du - sd) / sz : u * (du - sd);
        };
        if (wts && e0 >= 0) add[e0] = term(u0, du0);   // ids of a token are distinct: plain stores
        if (more)
            for (int j = gl + G; j < a.K; j += G) {
                const int e = __ldg(idx + j);
                if (e >= 0 && e < a.E)
                    add[e] = term(weight(raw(__ldg(row + e))), __ldg(dw + j) * a.rsf * (a.pes ? __ldg(a.pes + e) : 1.0f));
            }
        __syncwarp();

        // ---- the row
        float x[NE], dot = 0.0f;
        if (VEC) {
#pragma unroll
            for (int i = 0; i < NE; i += 4) {
                const float4 v = *reinterpret_cast<const float4*>(add + R::expert(i, gl));
                x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i) x[i] = add[R::expert(i, gl)];
        }
        // dp: the balance loss's, and for kDirect the slots' too
        const bool through = bal || (MODE == kDirect && wts);
        const float on = bal ? 1.0f : 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const float d = MODE == kDirect ? fmaf(on, g[i], x[i]) : on * g[i];
            dot = fmaf(p[i], d, dot);
        }
        dot = group_sum<G>(dot) * rz;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const float d = MODE == kDirect ? fmaf(on, g[i], x[i]) : on * g[i];
            // a token takes no part of a gradient that it does not have (its row may hold NaN)
            if (MODE == kSigmoid) p[i] = slope[i] * ((through ? (d - dot) * rz : 0.0f) + x[i]);
            else p[i] = (MODE == kDirect ? 0.0f : x[i]) + (through ? p[i] * rz * (d - dot) : 0.0f);
            if (MODE == kSigmoid && !bal && !wts) p[i] = 0.0f;
        }
        if (in) R::store(a.dl + tr * a.E, a.E, gl, p);
        __syncwarp();
        // ---- back to zero, and the scale's gradient
        if (wts && e0 >= 0) {
            add[e0] = 0.0f;
            if (a.dpes) dscale[e0] += x0 * u0;
        }
        if (more) {
            for (int j = gl + G; j < a.K; j += G) {
                const int e = __ldg(idx + j);
                if (e < 0 || e >= a.E) continue;
                add[e] = 0.0f;
                if (a.dpes) dscale[e] += __ldg(dw + j) * a.rsf * weight(raw(__ldg(row + e)));
            }
        }
        __syncwarp();
    }
    if (!a.dpes) return;
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        float v = 0.0f;
        for (int w = 0; w < kRWarps * TPW; ++w) v += s_scale[w][e];
        a.part[static_cast<size_t>(blockIdx.x) * a.E + e] = v;
    }
}

// A block joins 32 experts: a lane an expert, a warp every 32nd chunk, then the warps in order.
__global__ void __launch_bounds__(1024) k_join_scale_grad(RouteBackwardArgs a) {
    __shared__ float s_p[32][33];
    pdl_wait_then_release();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (e < a.E) {
#pragma unroll 4
        for (int c = warp; c < a.chunks; c += 32) v += __ldcg(a.part + static_cast<size_t>(c) * a.E + e);
    }
    s_p[warp][lane] = v;
    __syncthreads();
    if (warp || e >= a.E) return;
    v = 0.0f;
    for (int w = 0; w < 32; ++w) v += s_p[w][lane];
    a.dpes[e] = v;
}

namespace {

template <int NE, int G>
cudaError_t balance_t(const BalanceArgs& a, bool vec, cudaStream_t s) {
    const dim3 grid(a.chunks), block(kBWarps * 32);
    if (a.routing)
        return vec ? launch_pdl(k_balance<NE, G, true, true>, grid, block, 0, s, a)
                   : launch_pdl(k_balance<NE, G, false, true>, grid, block, 0, s, a);
    return vec ? launch_pdl(k_balance<NE, G, true, false>, grid, block, 0, s, a)
               : launch_pdl(k_balance<NE, G, false, false>, grid, block, 0, s, a);
}

template <int NE, int G, int MODE>
cudaError_t backward_m(const RouteBackwardArgs& a, bool vec, cudaStream_t s) {
    const dim3 grid(a.chunks), block(kRWarps * 32);
    return vec ? launch_pdl(k_route_backward<NE, G, true, MODE>, grid, block, 0, s, a)
               : launch_pdl(k_route_backward<NE, G, false, MODE>, grid, block, 0, s, a);
}

template <int NE, int G>
cudaError_t backward_t(const RouteBackwardArgs& a, bool vec, cudaStream_t s) {
    return a.routing  ? backward_m<NE, G, kSigmoid>(a, vec, s)
           : a.renorm ? backward_m<NE, G, kRenorm>(a, vec, s)
                      : backward_m<NE, G, kDirect>(a, vec, s);
}

bool rows16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

cudaError_t launch_balance(const BalanceArgs& a, cudaStream_t s) {
    const bool vec = a.E % 4 == 0 && rows16(a.logits);
    const cudaError_t e = a.E <= 32    ? balance_t<4, 8>(a, vec, s)
                          : a.E <= 64  ? balance_t<8, 8>(a, vec, s)
                          : a.E <= 128 ? balance_t<16, 8>(a, vec, s)
                                       : balance_t<16, 16>(a, vec, s);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_balance_join, dim3(a.S, (a.E + 31) / 32), dim3(1024), 0, s, a);
}

cudaError_t launch_route_backward(const RouteBackwardArgs& a, cudaStream_t s) {
    const bool vec = a.E % 4 == 0 && rows16(a.logits) && rows16(a.dl) && rows16(a.counts);
    const cudaError_t e = a.E <= 32    ? backward_t<4, 8>(a, vec, s)
                          : a.E <= 64  ? backward_t<8, 8>(a, vec, s)
                          : a.E <= 128 ? backward_t<16, 8>(a, vec, s)
                                       : backward_t<16, 16>(a, vec, s);
    if (e != cudaSuccess || !a.dpes) return e;
    return launch_pdl(k_join_scale_grad, dim3((a.E + 31) / 32), dim3(1024), 0, s, a);
}

}  // namespace moe
