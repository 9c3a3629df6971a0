// linear_narrow.cu -- the dense FP8 product for few tokens (moe_linear), every recipe: swap-AB, so
// that a tile is 128 weight rows (output columns) by 32 or 64 tokens and computes little padding,
// with K split over a cluster so that a product of few tiles still uses every SM.
//
// A CTA of the cluster takes a contiguous share of the K groups: TMA loads of 128 weight rows and the
// token rows per 128-deep stage, then
//   recipe 0:    tcgen05.mma.kind::f8f6f4 per group into one of four TMEM buffers, promoted by the
//                epilogue warps, acc[token] += P * (a_s[token] * w_s[row]);
//   recipes 1, 2: the block-scaled MMA over the whole share in one TMEM accumulator, the weights'
//                scale atoms as SFA, the tokens' built per stage by one warp as SFB.
// The shares meet in shared memory: each CTA sends its partial sums of a token to the CTA that owns
// the token, one bulk copy per owner, which adds them in rank order and runs the epilogue.  (Plain
// distributed-shared-memory stores of the same sums took 14000 cycles at 64 tokens.)
// What bounds it: the weight bytes, and at one token the latency of one load, one MMA chain and the
// exchange.  In a graph: 1 x 7168 x 2048 MXFP8 5.8 us (15 MB, 2.6 TB/s), 64 x 2816 x 2816 with fp32
// scales and a residual 8.0 us.  Every wait is bounded.
#include "linear_common.cuh"

namespace moe {

namespace {

constexpr int kSThreads = 256;
constexpr int kSEpiWarps = 4;
constexpr int kSBuf = 4;                               // TMEM buffers of recipe 0
constexpr uint32_t kSA = kTileM * kTileK;              // 16 KB of weights
constexpr uint32_t kSSf = 512;

// Two CTAs an SM.  (One CTA with a ring as deep as its share was slower at one token, 18 against 14
// us: its shared memory keeps it off an SM until the kernel before it has left.)
template <int NT>
struct SL {
    static constexpr int stages = NT == 32 ? 4 : 3;
    static constexpr uint32_t bytes_b = NT * kTileK;
    static constexpr uint32_t b = kSA;
    static constexpr uint32_t ws = kSA + bytes_b;      // fp32 weight scales, or the weights' atom
    static constexpr uint32_t ts = ws + kSSf;          // fp32 token scales, or the tokens' atom
    static constexpr uint32_t stage = ts + kSSf;
    static constexpr uint32_t part = stages * stage;   // [source rank][token of mine][128]
    static constexpr uint32_t bars = part + NT * 128 * 4;
    static constexpr uint32_t nbars = 3 * stages + 2 * kSBuf + 2;   // full, sfready, empty, tfull, tempty, drain, xbar
    static constexpr uint32_t misc = bars + nbars * 8;
    static constexpr uint32_t end = misc + 16;
    static constexpr uint32_t smem = end + 1024;
    static constexpr uint32_t tmem_cols = NT == 32 ? 128 : 256;
    static constexpr uint32_t sf_col0 = NT;            // scale factors behind the one accumulator
    static_assert(stage % 1024 == 0, "stage alignment");
    static_assert(kSBuf * NT <= tmem_cols && sf_col0 + stages * 8 <= tmem_cols, "TMEM");
    static_assert(NT * 128 * 4 <= part, "the share's own sums fit in the stages");
    static_assert(smem <= 113 * 1024, "two CTAs an SM");
};

__device__ __forceinline__ uint32_t cluster_addr(uint32_t smem_addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr), "r"(rank));
    return r;
}

// One bulk copy from this CTA's shared memory into another's of the cluster, counted on the barrier there.
__device__ __forceinline__ void bulk_send(uint32_t dst_cluster, uint32_t src, uint32_t bytes, uint32_t bar_cluster) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     dst_cluster),
                 "r"(src), "r"(bytes), "r"(bar_cluster)
                 : "memory");
}

// The cluster barrier in its two halves (every thread of every CTA, once each).
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ void finish_one(const LinearArgs& p, float v, int t, int n) {
    if (p.bias) v += __bfloat162float(p.bias[n]);
    v = linear_act(v, p.act);
    const size_t at = static_cast<size_t>(t) * p.N + n;
    if (p.res) v += __bfloat162float(p.res[at]);
    p.y[at] = __float2bfloat16_rn(v);
}

}  // namespace

// Grid (split, weight blocks, token blocks), clusters of `split` CTAs.
template <int NT, bool MX>
__global__ void __launch_bounds__(kSThreads, 2)
    k_linear_narrow(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmT, const LinearArgs p) {
    using S = SL<NT>;
    constexpr int ST = S::stages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::bars);
    uint64_t* sfready = full + ST;
    uint64_t* empty = sfready + ST;
    uint64_t* tfull = empty + ST;
    uint64_t* tempty = tfull + kSBuf;
    uint64_t* drain = tempty + kSBuf;
    uint64_t* xbar = drain + 1;                        // the shares of this CTA's tokens have arrived
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + S::misc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::misc + 4);

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int split = gridDim.x, rank = blockIdx.x;
    const int n0 = blockIdx.y * kTileM, t0 = blockIdx.z * NT;
    const int KB = p.K / kTileK;
    const int g0 = static_cast<int>(static_cast<long long>(rank) * KB / split);
    const int n = static_cast<int>(static_cast<long long>(rank + 1) * KB / split) - g0;   // this CTA's groups
    const int per = NT / split;                        // tokens that a CTA of the cluster owns

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&sfready[s], 1);
            mbar_init(&empty[s], MX ? 1 : 1 + kSEpiWarps);
        }
        for (int b = 0; b < kSBuf; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], kSEpiWarps);
        }
        mbar_init(drain, 1);
        mbar_init(xbar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        if (split > 1 && t0 + rank * per < p.T) mbar_arrive_expect_tx(xbar, static_cast<uint32_t>(NT * 512));
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmT);
        for (int i = 0; i < n && i < ST; ++i) tma_prefetch_2d(&tmW, (g0 + i) * kTileK, n0);   // toward L2, ahead of the wait
    }
    if (warp == 1) tmem_alloc(tmem_holder, S::tmem_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (split > 1) cluster_arrive();                   // this CTA has started (waited for before the exchange)
    pdl_wait_then_release();
    if (p.clear && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) *p.status = MOE_OK;
    const uint32_t tmem_base = *tmem_holder;
    float acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = 0.0f;

    if (warp == 0) {
        // ---------------------------------------------------------------------- TMA producer
        const uint32_t a_bytes = p.recipe == 2 ? kSA / 2 : kSA;   // E2M1 weights arrive packed
        const int n_pad = (p.N + kLinearPad - 1) / kLinearPad * kLinearPad;
        int it = 0;
        uint32_t s = 0, ph = 1;
        bool ok = true;
        for (; it < n; ++it) {
            const int kb = g0 + it;
            if (!mbar_wait(&empty[s], ph, abort_flag, p.status)) {
                ok = false;
                break;
            }
            uint8_t* st = smem + s * S::stage;
            if (!fault_skip_stage(p.fault, it) && elect_one()) {   // debug builds: an injected fault
                mbar_arrive_expect_tx(&full[s], a_bytes + S::bytes_b + kSSf + (MX ? 0 : NT * 4));
                tma_load_2d(st, &tmW, kb * kTileK, n0, &full[s]);
                tma_load_2d(st + S::b, &tmT, kb * kTileK, t0, &full[s]);
                if (MX) {
                    bulk_load(st + S::ws, static_cast<const uint8_t*>(p.w_scale) +
                                              (static_cast<size_t>(blockIdx.y) * KB + kb) * kSSf, kSSf, &full[s]);
                } else {
                    bulk_load(st + S::ws, static_cast<const float*>(p.w_scale) + static_cast<size_t>(kb) * n_pad + n0,
                              kSSf, &full[s]);
                    bulk_load(st + S::ts, static_cast<const float*>(p.a_scale) + static_cast<size_t>(kb) * p.a_pad + t0,
                              NT * 4, &full[s]);
                }
            }
            __syncwarp();
            if (++s == ST) {
                s = 0;
                ph ^= 1;
            }
        }
        // the copies already issued land before their space is used again: the MMAs have read them, or after an abort
        for (int i = 0; i < ST && ok; ++i) {
            ok = mbar_wait(&empty[s], ph, abort_flag, p.status);
            if (++s == ST) {
                s = 0;
                ph ^= 1;
            }
        }
        if (!ok)
            for (int i = it > ST ? it - ST : 0; i < it; ++i) drain_wait(&full[i % ST], (i / ST) & 1);
    } else if (warp == 2) {
        if (MX) {
            // -------------------------------------------------------------------- token-scale atoms
            // lane i: the words of tokens i (and 32 + i); the scale rows reach 132 past T
            // (eight stages' words at a time, so that a load's latency is not paid per stage)
            const uint32_t* src = static_cast<const uint32_t*>(p.a_scale) + static_cast<size_t>(g0) * p.a_pad + t0 + lane;
            constexpr int kAhead = 8;
            for (int base = 0; base < n; base += kAhead) {
                uint32_t w0[kAhead], w1[kAhead];
#pragma unroll
                for (int d = 0; d < kAhead; ++d) {
                    const uint32_t* q = src + static_cast<size_t>(min(base + d, n - 1)) * p.a_pad;
                    w0[d] = __ldg(q);
                    w1[d] = NT == 64 ? __ldg(q + 32) : 0u;
                }
                bool ok = true;
#pragma unroll
                for (int d = 0; d < kAhead; ++d) {
                    const int it = base + d, s = it % ST;
                    if (it >= n || !ok) break;
                    if (it >= ST && !mbar_wait(&empty[s], ((it / ST) & 1) ^ 1, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    *reinterpret_cast<uint2*>(smem + s * S::stage + S::ts + 16 * lane) = make_uint2(w0[d], w1[d]);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // visible to tcgen05.cp
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sfready[s]);
                }
                if (!ok) break;
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------------- MMA issuer
        const uint32_t idesc = f8_idesc(kTileM, NT);
        const uint32_t afmt = p.recipe == 2 ? 5u : 0u;
        const uint64_t a_desc0 = sw128_kmajor_desc(smem_u32(smem)), b_desc0 = sw128_kmajor_desc(smem_u32(smem + S::b));
        const uint64_t sfa_desc0 = sf_atom_desc(smem_u32(smem + S::ws)), sfb_desc0 = sf_atom_desc(smem_u32(smem + S::ts));
        uint32_t s = 0, ph = 0, buf = 0, bph = 1;
        for (int it = 0; it < n; ++it) {
            if (!mbar_wait(&full[s], ph, abort_flag, p.status) || (MX && !mbar_wait(&sfready[s], ph, abort_flag, p.status)) ||
                (!MX && !mbar_wait(&tempty[buf], bph, abort_flag, p.status)))
                break;
            tc_fence_after();
            const uint32_t at = s * (S::stage >> 4);
            const uint64_t ad = a_desc0 + at, bd = b_desc0 + at;
            if (elect_one()) {
                if (MX) {
                    const uint32_t sfa_t = tmem_base + S::sf_col0 + s * 8, sfb_t = sfa_t + 4;
                    sf_copy(sfa_t, sfa_desc0 + at);
                    sf_copy(sfb_t, sfb_desc0 + at);
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k)
                        mma_mx(tmem_base, ad + 2 * k, bd + 2 * k, mx_block_idesc(k, afmt, 0u, kTileM, NT), sfa_t, sfb_t,
                               (it > 0 || k > 0) ? 1u : 0u);
                    if (it == n - 1) mma_commit(&tfull[0]);
                } else {
                    const uint32_t d = tmem_base + buf * NT;
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k) mma_f8(d, ad + 2 * k, bd + 2 * k, idesc, k > 0 ? 1u : 0u);
                    mma_commit(&tfull[buf]);
                }
                mma_commit(&empty[s]);
            }
            __syncwarp();
            if (++s == ST) {
                s = 0;
                ph ^= 1;
            }
            if (++buf == kSBuf) {
                buf = 0;
                bph ^= 1;
            }
        }
        if (elect_one()) mma_commit(drain);   // all MMAs issued by this warp have finished
        __syncwarp();
        drain_wait(drain, 0);
    } else if (warp >= 4) {
        // ---------------------------------------------------------------------- epilogue: the share's sums
        const int quad = warp & 3;      // TMEM lanes 32*quad .. = weight rows of the tile
        const uint32_t trow = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
        bool ok = true;
        if (MX) {
            if (n > 0) {
                ok = mbar_wait(&tfull[0], 0, abort_flag, p.status);
                if (__all_sync(0xffffffffu, ok)) {
                    tc_fence_after();
#pragma unroll
                    for (int h = 0; h < NT; h += 32) {
                        uint32_t v[32];
                        MOE_TMEM_LD32(trow + h, v);
                        MOE_TMEM_WAIT_LD(v);
#pragma unroll
                        for (int j = 0; j < 32; ++j) acc[h + j] = __uint_as_float(v[j]);
                    }
                }
            }
        } else {
            for (int it = 0; it < n; ++it) {
                const int s = it % ST, b = it % kSBuf;
                // the stage's scales (bulk copies), then the group's partial sums
                ok = mbar_wait(&full[s], (it / ST) & 1, abort_flag, p.status) &&
                     mbar_wait(&tfull[b], (it / kSBuf) & 1, abort_flag, p.status);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t st = smem_u32(smem + s * S::stage);
                const float ws = ld_shared_f32(st + S::ws + static_cast<uint32_t>((quad * 32 + lane) * 4));
#pragma unroll
                for (int h = 0; h < NT; h += 32) {
                    uint32_t v[32];
                    MOE_TMEM_LD32(trow + static_cast<uint32_t>(b * NT + h), v);
                    MOE_TMEM_WAIT_LD(v);
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 a4 = ld_shared_f32x4(st + S::ts + static_cast<uint32_t>((h + j) * 4));
                        acc[h + j] = fmaf(__uint_as_float(v[j]), a4.x * ws, acc[h + j]);
                        acc[h + j + 1] = fmaf(__uint_as_float(v[j + 1]), a4.y * ws, acc[h + j + 1]);
                        acc[h + j + 2] = fmaf(__uint_as_float(v[j + 2]), a4.z * ws, acc[h + j + 2]);
                        acc[h + j + 3] = fmaf(__uint_as_float(v[j + 3]), a4.w * ws, acc[h + j + 3]);
                    }
                }
                tc_fence_before();
                // the scales were read through the generic proxy; the next bulk copy into this stage
                // is an async-proxy write: order the reads before it
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&tempty[b]);
                    mbar_arrive(&empty[s]);
                }
            }
        }
        if (!__all_sync(0xffffffffu, ok)) {
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[j] = __int_as_float(0x7fc00000);   // a wait ran out: NaN
        }
    }
    __syncwarp();

    // -------------------------------------------------------------------------- the shares meet
    const int row = (warp & 3) * 32 + lane, col = n0 + row;
    if (split == 1) {
        if (warp >= 4 && col < p.N) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (t0 + j < p.T) finish_one(p, acc[j], t0 + j, col);
        }
    } else {
        // Two neighbouring columns a thread, tokens threadIdx / 64, + 4, ...; the first residuals are
        // fetched while the shares are on their way.
        const int c2 = (threadIdx.x & 63) * 2, tq = threadIdx.x >> 6, n2 = n0 + c2;
        const bool pair = p.N % 2 == 0;
        __nv_bfloat162 r0 = __floats2bfloat162_rn(0.0f, 0.0f), r1 = r0;
        const int ta = t0 + rank * per + tq, tb = ta + 4;
        if (p.res && pair && n2 < p.N) {
            if (tq < per && ta < p.T) r0 = *reinterpret_cast<const __nv_bfloat162*>(p.res + static_cast<size_t>(ta) * p.N + n2);
            if (tq + 4 < per && tb < p.T) r1 = *reinterpret_cast<const __nv_bfloat162*>(p.res + static_cast<size_t>(tb) * p.N + n2);
        }
        const float b0 = p.bias && n2 < p.N ? __bfloat162float(p.bias[n2]) : 0.0f;
        const float b1 = p.bias && n2 + 1 < p.N ? __bfloat162float(p.bias[n2 + 1]) : 0.0f;
        if (warp >= 4) {                               // this share's sums, [token][row], over the stages' space
            if (!MX) named_bar_sync(1, 32 * kSEpiWarps);   // no warp still reads a stage's scales
            float* own = reinterpret_cast<float*>(smem) + row;
#pragma unroll
            for (int j = 0; j < NT; ++j) own[j * 128] = acc[j];
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncthreads();
        cluster_wait();                                // every CTA of the cluster has set its barrier up
        if (warp == 4 && __any_sync(0xffffffffu, *abort_flag != 0)) {   // a copy that came late may have landed on them
            float* own = reinterpret_cast<float*>(smem);
#pragma unroll 1
            for (int i = lane; i < NT * 128; i += 32) own[i] = __int_as_float(0x7fc00000);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
        }
        if (warp == 4 && lane < split && t0 + lane * per < p.T) {   // lane r sends rank r its tokens
            const uint32_t bytes = static_cast<uint32_t>(per * 512);
            const uint32_t to = static_cast<uint32_t>(lane);
            bulk_send(cluster_addr(smem_u32(smem + S::part) + static_cast<uint32_t>(rank) * bytes, to),
                      smem_u32(smem) + to * bytes, bytes, cluster_addr(smem_u32(xbar), to));
        }
        __syncwarp();
        bool have = true;
        if (t0 + rank * per < p.T) {
            have = mbar_wait(xbar, 0, abort_flag, p.status);
            // the others send theirs all the same, at their own waits' limits: no copy is under way when a CTA leaves
            if (!have) drain_wait(xbar, 0, 2 * kWaitLimitNs);
        }
        __syncwarp();
        cluster_arrive();                              // this CTA holds its shares: its senders may leave
        const float* mine = reinterpret_cast<const float*>(smem + S::part) + c2;
        for (int jl = tq; jl < per; jl += 4) {
            const int t = t0 + rank * per + jl;
            if (t >= p.T || n2 >= p.N) break;
            float2 v = *reinterpret_cast<const float2*>(mine + jl * 128);
#pragma unroll 8
            for (int r = 1; r < split; ++r) {
                const float2 x = *reinterpret_cast<const float2*>(mine + (r * per + jl) * 128);
                v.x += x.x, v.y += x.y;
            }
            if (!have) v.x = v.y = __int_as_float(0x7fc00000);
            v.x = linear_act(v.x + b0, p.act), v.y = linear_act(v.y + b1, p.act);
            const size_t at = static_cast<size_t>(t) * p.N + n2;
            if (pair) {
                if (p.res) {
                    const float2 r = __bfloat1622float2(
                        jl == tq ? r0 : jl == tq + 4 ? r1 : *reinterpret_cast<const __nv_bfloat162*>(p.res + at));
                    v.x += r.x, v.y += r.y;
                }
                *reinterpret_cast<__nv_bfloat162*>(p.y + at) = __floats2bfloat162_rn(v.x, v.y);
            } else {
                if (p.res) v.x += __bfloat162float(p.res[at]);
                p.y[at] = __float2bfloat16_rn(v.x);
                if (n2 + 1 < p.N) {
                    if (p.res) v.y += __bfloat162float(p.res[at + 1]);
                    p.y[at + 1] = __float2bfloat16_rn(v.y);
                }
            }
        }
        __syncwarp();
        cluster_wait();                                // every copy out of this CTA has landed
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, S::tmem_cols);
    }
}

int linear_narrow_tokens(int T) { return T <= 32 ? 32 : 64; }

// The widest split that still lets every CTA run at once (two an SM) and gives each a K group.
int linear_narrow_split(int T, int N, int K, int num_sms) {
    const int nt = linear_narrow_tokens(T);
    const long long tiles = static_cast<long long>((N + kTileM - 1) / kTileM) * ((T + nt - 1) / nt);
    int split = 8;
    while (split > 1 && (tiles * split > 2LL * num_sms || split > K / kTileK)) split >>= 1;
    return split;
}

template <int NT, bool MX>
static cudaError_t launch_narrow_t(const LinearArgs& a, const LinearMaps& m, int split, cudaStream_t s) {
    constexpr uint32_t smem = SL<NT>::smem;
    cudaError_t e = cudaFuncSetAttribute(k_linear_narrow<NT, MX>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(split, (a.N + kTileM - 1) / kTileM, (a.T + NT - 1) / NT);
    cfg.blockDim = dim3(kSThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_linear_narrow<NT, MX>, m.w, m.x, a);
}

template <int NT>
static cudaError_t launch_narrow_n(const LinearArgs& a, const LinearMaps& m, int num_sms, cudaStream_t s) {
    const int split = linear_narrow_split(a.T, a.N, a.K, num_sms);
    return a.recipe == 0 ? launch_narrow_t<NT, false>(a, m, split, s)
                         : launch_narrow_t<NT, true>(a, m, split, s);
}

cudaError_t launch_linear_narrow(const LinearArgs& a, const LinearMaps& m, int num_sms, cudaStream_t s) {
    return linear_narrow_tokens(a.T) == 32 ? launch_narrow_n<32>(a, m, num_sms, s) : launch_narrow_n<64>(a, m, num_sms, s);
}

}  // namespace moe
