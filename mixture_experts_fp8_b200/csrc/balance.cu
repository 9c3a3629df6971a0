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
// once and a sum over a row takes three shuffles (four) for all of them.  (65536 x 128 gradients with 16
// lanes of 8 experts: 24 us of kernel against 18.7, the instructions of a row's sums and slots are for half as
// many tokens.)  Sums are fp32 in registers, then per block and chunk in a fixed order without atomics on
// floats, so a result is the same on every run.
//
// In a stream of calls: the loss of 65536 x 128 (36 MB) 13.4 us, of 4096 x 256 in nine sequences 10.6 us
// (in a graph, from run to run, 13.8 to 15.4 and 9.8 to 11.3), of one token in a graph 4.6 us; the gradients
// of 65536 x 128 with the scales' (73 MB) 21.6 us, 3.4 TB/s, of 4096 x 256 6.3 us.  Small calls are the latency
// of two launches (one) with a read, a reduction and a write each; large gradients the chain of sums from row to
// row (38% of the issue slots, 16 warps an SM at 112 registers).
#include <math.h>

#include "block_kernels.h"
#include "moe_common.cuh"

namespace moe {

namespace {

// Offset i of the sequences, kept inside [0, T].
__device__ __forceinline__ int offset_at(const int32_t* off, int T, int i) { return min(max(__ldg(off + i), 0), T); }

// How many i of 0 .. S - 1 have pred(i), true up to some i and false behind it: all at once with a thread for
// each, where a search makes log2 S loads that wait for one another, or by that search above THREADS.
template <int THREADS, typename F>
__device__ __forceinline__ int block_count(int S, F pred) {
    if (S <= THREADS) return __syncthreads_count(static_cast<int>(threadIdx.x) < S && pred(threadIdx.x));
    int lo = 0, hi = S;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (pred(mid)) lo = mid + 1;
        else hi = mid;
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

// 16 bytes into shared memory, and the wait for all that the thread has asked for.
__device__ __forceinline__ void cp_async16(float* dst, const float* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// e^x for x <= 0 as 2^(x log2 e): the product's rounding makes its relative error up to |x| 2^-24, under
// 2e-6 wherever e^x is above 1e-12 (as much as the rounding of the logits' difference does), and e^x is zero
// below 2^-126.  In calls, against expf: the loss of 65536 x 128 13.1 us against 14.4, its gradients 21.7 against
// 22.4; the loss and the means are off 64 bits by 6e-8 relative there, a form with 64-bit sums by 3e-8.
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
constexpr int kJThreads = 512;                         // k_balance_join
constexpr int kRWarps = 8;                             // k_route_backward

}  // namespace

// Block c + s takes the tokens of chunk c that are in sequence s.  The sums of p stay in registers and are joined
// over the lanes and warps in order at the end.
template <int NE, int G, bool VEC, bool SIG>
__global__ void __launch_bounds__(kBWarps * 32) k_balance(BalanceArgs a) {
    using R = Row<NE, G, VEC>;
    constexpr int TPW = 32 / G, W = NE * G;
    __shared__ float s_p[kBWarps][W];
    __shared__ int s_n[W + 2];                         // counts, counted tokens, ids out of range
    const int slot = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gl = lane % G;
    for (int e = threadIdx.x; e < W + 2; e += blockDim.x) s_n[e] = 0;
    pdl_wait_then_release();
    if (slot == 0 && threadIdx.x == 0) {
        *a.status = MOE_OK;
        *a.ticket = 0;
    }
    int s = 0, b0 = 0, b1 = a.T;
    if (a.off) {                                       // the first sequence whose last slot is not before this one
        s = block_count<kBWarps * 32>(a.S, [&](int i) {
            return (offset_at(a.off, a.T, i + 1) + a.chunk - 1) / a.chunk - 1 + i < slot;
        });
        if (s == a.S) return;
        b0 = offset_at(a.off, a.T, s);
        b1 = offset_at(a.off, a.T, s + 1);
    } else {
        __syncthreads();
    }
    if (s > slot || slot - s > (a.T - 1) / a.chunk) return;
    const int c0 = (slot - s) * a.chunk;
    b0 = max(b0, c0);
    b1 = min(b1, min(a.T - c0, a.chunk) + c0);
    if (b0 >= b1) return;
    if (a.off && a.S > kBWarps * 32) __syncthreads();  // s_n
    const int warps = min(kBWarps, (b1 - b0 + TPW - 1) / TPW);   // warps with a token
    if (warp < warps) {
        float acc[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) acc[i] = 0.0f;
        for (int tb = b0 + warp * TPW; tb < b1; tb += kBWarps * TPW) {
            const int t = tb + lane / G;
            const bool in = t < b1;
            const int32_t* idx = a.idx + static_cast<size_t>(in ? t : b0) * a.K;
            float p[NE];                               // the loads do not wait for the mask's
            R::template load<float4>(a.logits + static_cast<size_t>(in ? t : b0) * a.E, a.E, gl, in, p, -INFINITY);
            const int e0 = gl < a.K ? __ldg(idx + gl) : 0;
            const bool ok = in && !(a.mask && !__ldg(a.mask + t));
            if (ok) {
                if (gl < a.K) atomicAdd(&s_n[e0 >= 0 && e0 < a.E ? e0 : W + 1], 1);
                for (int j = gl + G; j < a.K; j += G) {
                    const int e = __ldg(idx + j);
                    atomicAdd(&s_n[e >= 0 && e < a.E ? e : W + 1], 1);
                }
                if (gl == 0) atomicAdd(&s_n[W], 1);
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
    const int row = balance_row(a.E);                  // <= W; the sums past E are zero
    for (int e = threadIdx.x; e < row; e += blockDim.x) {
        float v = 0.0f;
        for (int w = 0; w < warps; ++w) v += s_p[w][e];
        a.part_p[static_cast<size_t>(slot) * row + e] = v;
        a.part_n[static_cast<size_t>(slot) * row + e] = s_n[e];
    }
    if (threadIdx.x == 0) a.part_t[slot] = make_int2(s_n[W], s_n[W + 1]);
}

// The `split` blocks of a cluster join sequence s's slots, an equal share of the experts each: Q threads (a power of
// two) take a share of a slot's row, four experts each, the block kJThreads / Q slots at a time and several times that
// in flight, then the threads of an expert in order.  The shares of the loss meet in the first block; the last first
// block to finish adds the losses of the sequences.
// (It asks for as much shared memory as k_balance: with another amount an SM would have to be divided anew before it
// starts, 65536 x 32 in 11.9 us instead of 8.8.)
template <bool SPLIT>
__global__ void __launch_bounds__(kJThreads) k_balance_join(BalanceArgs a, int lq) {
    constexpr int kWarps = kJThreads / 32, BATCH = 5;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int s_tok[kWarps];
    __shared__ float s_red[kWarps], s_term[8];
    __shared__ int s_last;
    const int split = SPLIT ? gridDim.y : 1, share = SPLIT ? blockIdx.y : 0, Q = 1 << lq, W = 4 * Q, rows = kJThreads >> lq;
    const int parts = Q < 32 ? kWarps : rows;
    float* const s_p = reinterpret_cast<float*>(smem); // [part][4 Q]: a warp is a part, or (Q = 64) two are
    int* const s_n = reinterpret_cast<int*>(s_p + parts * W);
    if (SPLIT) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // this block has started
    pdl_wait_then_release();
    const int s = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = threadIdx.x & (Q - 1);
    const int row = balance_row(a.E), e0 = share * W;
    int b0 = 0, b1 = a.T;
    bool bad = false;
    if (a.off) {
        const int r0 = __ldg(a.off + s), r1 = __ldg(a.off + s + 1);
        bad = r0 < 0 || r1 > a.T || r0 > r1;
        b0 = min(max(r0, 0), a.T);
        b1 = min(max(r1, 0), a.T);
    }
    const int lo = s + b0 / a.chunk, hi = b0 < b1 ? s + (b1 - 1) / a.chunk : lo - 1;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    int4 n = make_int4(0, 0, 0, 0);
    int tok = 0;
    for (int c = lo + threadIdx.x; c <= hi; c += kJThreads) {
        const int2 t = __ldcg(a.part_t + c);
        tok += t.x;
        bad |= t.y != 0;
    }
    if (e0 + 4 * col < row) {
        for (int c = lo + (static_cast<int>(threadIdx.x) >> lq); c <= hi; c += BATCH * rows) {
            float4 x[BATCH];
            int4 y[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                x[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                y[u] = make_int4(0, 0, 0, 0);
                if (c + u * rows <= hi) {
                    const size_t at = static_cast<size_t>(c + u * rows) * row + e0 + 4 * col;
                    x[u] = __ldcg(reinterpret_cast<const float4*>(a.part_p + at));
                    y[u] = __ldcg(reinterpret_cast<const int4*>(a.part_n + at));
                }
            }
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                v.x += x[u].x, v.y += x[u].y, v.z += x[u].z, v.w += x[u].w;
                n.x += y[u].x, n.y += y[u].y, n.z += y[u].z, n.w += y[u].w;
            }
        }
    }
    for (int o = Q; o < 32; o <<= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o), v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        v.z += __shfl_xor_sync(0xffffffffu, v.z, o), v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
        n.x += __shfl_xor_sync(0xffffffffu, n.x, o), n.y += __shfl_xor_sync(0xffffffffu, n.y, o);
        n.z += __shfl_xor_sync(0xffffffffu, n.z, o), n.w += __shfl_xor_sync(0xffffffffu, n.w, o);
    }
    if (Q >= 32 || lane < Q) {
        const int at = (Q < 32 ? warp : static_cast<int>(threadIdx.x) >> lq) * W + 4 * col;
        *reinterpret_cast<float4*>(s_p + at) = v;
        *reinterpret_cast<int4*>(s_n + at) = n;
    }
    tok = __reduce_add_sync(0xffffffffu, tok);
    if (lane == 0) s_tok[warp] = tok;
    if (__syncthreads_or(bad) && threadIdx.x == 0) set_status(a.status, MOE_ERR_BOUNDS);
    tok = 0;
    for (int w = 0; w < kWarps; ++w) tok += s_tok[w];
    float term = 0.0f;
    if (threadIdx.x < W && e0 + static_cast<int>(threadIdx.x) < a.E) {
        const int e = e0 + threadIdx.x;
        float p = 0.0f;
        int k = 0;
#pragma unroll 8
        for (int w = 0; w < parts; ++w) {
            p += s_p[w * W + threadIdx.x];
            k += s_n[w * W + threadIdx.x];
        }
        const float mean = tok ? p / static_cast<float>(tok) : 0.0f;
        a.mean[static_cast<size_t>(s) * a.E + e] = mean;
        a.counts[static_cast<size_t>(s) * a.E + e] = k;
        if (tok) term = static_cast<float>(k) * (static_cast<float>(a.E) / (static_cast<float>(a.K) * static_cast<float>(tok))) * mean;
    }
    term = warp_sum(term);
    if (lane == 0) s_red[warp] = term;
    __syncthreads();
    if (threadIdx.x == 0) {
        term = 0.0f;
        for (int w = 0; w < kWarps; ++w) term += s_red[w];
    }
    __syncwarp();
    if (SPLIT) {                                   // the shares go to the first block
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (threadIdx.x == 0) {
            uint32_t to;
            asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to)
                         : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(s_term + share))));
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(term) : "memory");
        }
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        if (share) return;
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    if (threadIdx.x == 0) {
        if (SPLIT) {
            term = 0.0f;
            for (int r = 0; r < split; ++r) term += s_term[r];
        }
        a.tokens[s] = tok;
        if (a.S == 1) {
            a.tokens[1] = tok > 0;
            a.loss[0] = tok ? a.coef * term : 0.0f;
            s_last = 0;
        } else {
            a.seq_loss[s] = term;
            __threadfence();
            s_last = atomicAdd(a.ticket, 1) == a.S - 1;
        }
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    float l = 0.0f;
    int full = 0;
    for (int i = threadIdx.x; i < a.S; i += kJThreads) {
        l += __ldcg(a.seq_loss + i);
        full += __ldcg(a.tokens + i) > 0;
    }
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
        for (int w = 0; w < kWarps; ++w) {
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
__global__ void __launch_bounds__(kRWarps * 32, NE <= 8 ? 4 : 2) k_route_backward(RouteBackwardArgs a) {
    using R = Row<NE, G, VEC>;
    constexpr int TPW = 32 / G, W = NE * G;
    __shared__ __align__(16) float s_add[kRWarps * TPW][W];
    __shared__ float s_scale[kRWarps * TPW][W];        // a group's sums of dscale
    __shared__ __align__(16) float s_row[VEC ? kRWarps * TPW : 1][W];   // VEC: a group's next logits, on their way
    pdl_wait_then_release();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gl = lane % G, grp = lane / G;
    const unsigned group_mask = (G == 32 ? 0xffffffffu : (1u << G) - 1u) << (grp * G);
    const int c0 = blockIdx.x * a.chunk, c1 = min(a.T, c0 + a.chunk), first = c0 + warp * TPW;
    // A token's row (VEC), its mask and the lane's own slot (all there is when k <= G) are asked for while the token
    // before it is worked on (65536 x 128: 20.5 -> 18.7 us; 4096 x 256, a token a group: 6.2 -> 6.5).
    float* const next_row = s_row[VEC ? warp * TPW + grp : 0];
    int next_e;
    float next_x;
    bool next_bal;
    auto fetch = [&](int t) {
        const bool in = t < c1;
        const size_t tr = static_cast<size_t>(in ? t : c0);
        if (VEC && in) {
#pragma unroll
            for (int i = 0; i < NE; i += 4)
                if (R::expert(i, gl) < a.E) cp_async16(next_row + R::expert(i, gl), a.logits + tr * a.E + R::expert(i, gl));
        }
        next_e = in && gl < a.K ? __ldg(a.idx + tr * a.K + gl) : -1;
        next_x = in && a.dw && gl < a.K ? __ldg(a.dw + tr * a.K + gl) : 0.0f;
        next_bal = in && a.dloss && !(a.mask && !__ldg(a.mask + t));
    };
    fetch(first + grp);
    float* add = s_add[warp * TPW + grp];
    float* dscale = s_scale[warp * TPW + grp];
    for (int e = gl; e < W; e += G) add[e] = dscale[e] = 0.0f;
    __syncwarp();
    const float gloss = a.dloss ? __ldg(a.dloss) * a.coef : 0.0f;
    int s_lo = 0, s_hi = 0;                            // the first sequences to end behind the block's first and last token
    if (a.dloss && a.off) {
        s_lo = block_count<kRWarps * 32>(a.S, [&](int i) { return offset_at(a.off, a.T, i + 1) <= c0; });
        s_hi = block_count<kRWarps * 32>(a.S, [&](int i) { return offset_at(a.off, a.T, i + 1) < c1; });
    }
    int q = -1, q0 = 0, q1 = 0;                        // the sequence whose gradient is in g, its tokens
    float g[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) g[i] = 0.0f;
    for (int tb = first; tb < c1; tb += kRWarps * TPW) {
        const int t = tb + grp;
        const bool in = t < c1;
        const size_t tr = static_cast<size_t>(in ? t : c0);
        const int32_t* idx = a.idx + tr * a.K;
        const float* dw = a.dw + tr * a.K;
        const float* row = a.logits + tr * a.E;
        float p[NE], slope[NE];
        const int e0 = next_e < a.E ? next_e : -1;
        float x0 = next_x;
        bool bal = next_bal;
        if (VEC) {
            cp_async_wait();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < NE; i += 4) {
                const int e = R::expert(i, gl);
                const bool has = in && e < a.E;
                const float4 v = *reinterpret_cast<const float4*>(next_row + e);
                p[i] = has ? v.x : -INFINITY, p[i + 1] = has ? v.y : -INFINITY;
                p[i + 2] = has ? v.z : -INFINITY, p[i + 3] = has ? v.w : -INFINITY;
            }
        } else {
            R::template load<float4>(row, a.E, gl, in, p, -INFINITY);
        }
        const float l0 = e0 < 0 ? -INFINITY : VEC ? next_row[e0] : __ldg(row + e0);
        __syncwarp();
        if (tb + kRWarps * TPW < c1) fetch(t + kRWarps * TPW);
        if (bal && !(t >= q0 && t < q1)) {             // another sequence than the last token's
            q = s_lo;
            for (int hi = s_hi; q < hi;) {
                const int mid = (q + hi) >> 1;
                if (offset_at(a.off, a.T, mid + 1) <= t) q = mid + 1;
                else hi = mid;
            }
            q0 = a.off ? offset_at(a.off, a.T, q) : 0;   // q = S: no sequence ends behind t
            q1 = !a.off ? a.T : q < a.S ? offset_at(a.off, a.T, q + 1) : 0;
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
        const float scale0 = e0 >= 0 && a.pes ? __ldg(a.pes + e0) : 1.0f;
        bool nz = e0 >= 0 && x0 != 0.0f;               // NaN counts; a slot without an expert does not
        if (in && a.dw)
            for (int j = gl + G; j < a.K; j += G) {
                const int e = __ldg(idx + j);
                nz |= e >= 0 && e < a.E && __ldg(dw + j) != 0.0f;
            }
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
        auto dp = [&](int i) { return MODE == kDirect ? (bal ? g[i] + x[i] : x[i]) : g[i]; };
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const float d = dp(i);
            dot = fmaf(p[i], d, dot);
        }
        dot = group_sum<G>(dot) * rz;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const float d = dp(i);
            // a token takes no part of a gradient that it does not have (its row or that gradient may hold NaN)
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
    for (int c = warp; c < a.chunks && e < a.E; c += 320) {
        float x[10];                                   // in flight
#pragma unroll
        for (int u = 0; u < 10; ++u) x[u] = c + 32 * u < a.chunks ? __ldcg(a.part + static_cast<size_t>(c + 32 * u) * a.E + e) : 0.0f;
#pragma unroll
        for (int u = 0; u < 10; ++u) v += x[u];
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
    const dim3 grid(a.slots), block(kBWarps * 32);
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
    // A sequence's experts over blocks of 32 where one block would read more than 96 KB of sums: one sequence of
    // 4096 x 256 (264 KB) takes 11.8 us with one block and 7.8 with eight (8.6 with four), one of 65536 x 64 (76 KB)
    // 11.1 with one and 15.4 with two, whose cluster does not start before the blocks of k_balance have left.
    int lq = a.E <= 32 ? 3 : a.E <= 64 ? 4 : a.E <= 128 ? 5 : 6, split = 1;
    if (8ll * balance_row(a.E) * a.slots / a.S > 96 * 1024) {
        split = 1 << (lq - 3);
        lq = 3;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.S, split);
    cfg.blockDim = dim3(kJThreads);
    cfg.dynamicSmemBytes = kBWarps * 4 * (a.E <= 32 ? 32 : a.E <= 64 ? 64 : a.E <= 128 ? 128 : 256);   // >= 32 Q parts
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = split;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    return split > 1 ? cudaLaunchKernelEx(&cfg, k_balance_join<true>, a, lq)
                     : cudaLaunchKernelEx(&cfg, k_balance_join<false>, a, lq);
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
