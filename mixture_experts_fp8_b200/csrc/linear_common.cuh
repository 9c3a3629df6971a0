// linear_common.cuh -- the epilogue of the dense product, shared by its kernels:
//   y[t, n] = bf16_rn( act( sum + bias[n] ) + residual[t, n] ),  one rounding at the end.
#pragma once

#include "block_kernels.h"
#include "gemm_common.cuh"

namespace moe {

// 0.5 v (1 + erf(v / sqrt 2)) = relu(v) - 0.5 |v| erfc(|v| / sqrt 2), so that the negative tail keeps its digits (as
// written, 1 + erf has lost a part in 20 at v = -5).  0.5 erfc(a / sqrt 2) is e^(-a^2/2) times a polynomial in
// t = 1 / (1 + 0.35 a), fitted here to 0.5 e^(a^2/2) erfc(a / sqrt 2) on [0, 16] by least squares reweighted toward
// the largest relative error, 4.5e-7 (7.4e-7 with fp32 steps).
__device__ __forceinline__ float gelu_erf(float v) {
    const float a = fabsf(v), t = __fdividef(1.0f, fmaf(0.35f, a, 1.0f));
    float q = 0.0479647337f;
    q = fmaf(q, t, -0.198432146f);
    q = fmaf(q, t, 0.234948159f);
    q = fmaf(q, t, -0.0123806731f);
    q = fmaf(q, t, 0.153811055f);
    q = fmaf(q, t, 0.133918516f);
    q = fmaf(q, t, 0.140193245f);
    q = fmaf(q, t, -2.30693386e-5f);
    const float tail = a * q * __expf(-0.5f * v * v);
    return v > 14.0f ? v : (v < 0.0f ? 0.0f : v) - tail;   // +inf stays; -inf is NaN, as in the product above
}

// cfg.activation: 0 none, 1 relu, 2 silu, 3 gelu (erf), 4 gelu (tanh form).  The last three take the hardware
// exponential and reciprocal (a few fp32 ulps, and as many as an exponential's argument has, far below the bf16
// rounding that follows); NaN stays NaN in every one.
template <int ACT>
__device__ __forceinline__ float linear_act_t(float v) {
    if (ACT == 1) return v < 0.0f ? 0.0f : v;
    if (ACT == 2) return silu(v);
    if (ACT == 3) return gelu_erf(v);
    if (ACT == 4) {   // 0.5 (1 + tanh u) = 1 / (1 + e^-2u),  u = sqrt(2/pi) (v + 0.044715 v^3)
        const float u2 = 1.5957691f * fmaf(0.044715f * v * v, v, v);
        return __fdividef(v, 1.0f + __expf(-u2));
    }
    return v;
}

__device__ __forceinline__ float linear_act(float v, int act) {
    switch (act) {
        case 1: return linear_act_t<1>(v);
        case 2: return linear_act_t<2>(v);
        case 3: return linear_act_t<3>(v);
        case 4: return linear_act_t<4>(v);
        default: return v;
    }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---- The output goes through shared memory, a subtile of 32 rows x C columns bf16 a warp: the residual is
// fetched into it while the sums are still being made, each lane replaces its row's residual by the
// result, and the tile leaves by TMA stores (N a multiple of 8; each warp on its own) or by coalesced
// stores (any N).  Laid out as the TMA box has it: C = 48, rows of 96 bytes as they are (a quarter warp's
// 16-byte accesses meet two at a time); C = 32, rows of 64 bytes with the 64-byte swizzle (they do not
// meet; 512-byte aligned).
//
// Any N: the four warps with the same 32 rows (a quad, kQuarters subtiles side by side) fetch and store
// whole tile rows together, 8 rows a warp, by aligned words: a row that starts at an odd element is
// handled one column apart.  (With each warp storing its own C columns, and odd rows by halves of words,
// most sectors were partial writes: 12900 cycles to fetch and 8500 to store a 128 x 192 tile.)
constexpr int kQuarters = 4;

template <int C>
struct Sub {
    static_assert(C == 32 || C == 48, "subtile columns");
    static constexpr int cols = C, chunks = C / 8, words = C / 2;
    static constexpr uint32_t bytes = 32 * C * 2;
    static __device__ __forceinline__ uint32_t chunk(int r, int j) {       // 8 columns of a row
        return static_cast<uint32_t>(r * C * 2 + (C == 32 ? (j ^ ((r >> 1) & 3)) : j) * 16);
    }
    static __device__ __forceinline__ uint32_t word(int r, int w) {        // 2 columns
        return chunk(r, w >> 2) + static_cast<uint32_t>((w & 3) * 4);
    }
};

__device__ __forceinline__ uint4 lds_u4(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts_u4(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts_u32(uint32_t a, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

__device__ __forceinline__ void sts_u16(uint32_t a, uint16_t v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(v) : "memory");
}

// Where an epilogue warp stands: its subtile and the quad's first (quarters are 4 subtiles apart), its
// quarter and quad, the rows' first token and the tile's and its own first column.
struct EpiAt {
    uint32_t sub, quad_sub;
    int qtr, quad, t0, tile_c0, c0;
};

// All four warps of the quad; true when every one says so.  (Each warp calls it once a tile until they
// leave together, so that none waits for one that has left.)
__device__ __forceinline__ bool quad_all(const EpiAt& at, bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.cta.red.and.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"(1 + at.quad), "r"(static_cast<uint32_t>(ok)) : "memory");
    return r != 0;
}

// Word W of tile row r (the quad's 32 rows, 2 columns a word).
template <int C>
__device__ __forceinline__ uint32_t quad_word(const EpiAt& at, int r, int W) {
    return at.quad_sub + static_cast<uint32_t>(W / Sub<C>::words) * (4 * Sub<C>::bytes) + Sub<C>::word(r, W % Sub<C>::words);
}

// Begin to fetch the residual (epilogue_residual_wait before use).  The subtiles are free: their stores have
// read them.  Rows that start at an odd element are fetched one column to the left; `last` then is the
// lane's row's last element, which that leaves out.
template <int C>
__device__ __forceinline__ void epilogue_residual(const LinearArgs& p, const EpiAt& at, uint32_t& last) {
    using S = Sub<C>;
    last = 0;
    if (!p.res) return;
    const int lane = threadIdx.x & 31;
    if (p.N % 8 == 0) {
        const int t = at.t0 + lane;
        if (t < p.T) {
            const __nv_bfloat16* row = p.res + static_cast<size_t>(t) * p.N;
#pragma unroll
            for (int j = 0; j < S::chunks; ++j) {
                const int c = at.c0 + 8 * j;
                if (c < p.N)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(at.sub + S::chunk(lane, j)), "l"(row + c)
                                 : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return;
    }
    constexpr int kLanes = kQuarters * S::words / 32;   // words of a row a lane
#pragma unroll 2
    for (int i = 0; i < 8; ++i) {
        const int r = 8 * at.qtr + i, t = at.t0 + r;
        if (t >= p.T) break;
        const int odd = p.N & t & 1;
        const __nv_bfloat16* row = p.res + static_cast<size_t>(t) * p.N + (at.tile_c0 - odd);
#pragma unroll
        for (int k = 0; k < kLanes; ++k) {
            const int W = 32 * k + lane, c = at.tile_c0 - odd + 2 * W;     // -1: the row before's last element
            const uint32_t dst = quad_word<C>(at, r, W);
            if (c + 1 < p.N)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(row + 2 * W) : "memory");
            else if (c < p.N)
                sts_u16(dst, *reinterpret_cast<const uint16_t*>(row + 2 * W));
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    const int t = at.t0 + lane, c = at.c0 + C - 1;
    if (t < p.T && (p.N & t & 1) && c < p.N)
        last = *reinterpret_cast<const uint16_t*>(p.res + static_cast<size_t>(t) * p.N + c);
}
// The residual is there, and (any N) the quad's warps are; false when one of them gave up.
__device__ __forceinline__ bool epilogue_residual_wait(const LinearArgs& p, const EpiAt& at, bool ok) {
    if (p.res) asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (p.N % 8) return quad_all(at, ok);
    return __all_sync(0xffffffffu, ok);
}

// The lane's row of the warp's subtile from acc.
template <int ACT, int C>
__device__ __forceinline__ void epilogue_sub_t(const LinearArgs& p, const EpiAt& at, uint32_t last, float* acc) {
    const int lane = threadIdx.x & 31;
    const bool odd = p.N & (at.t0 + lane) & 1;
#pragma unroll
    for (int j = 0; j < Sub<C>::chunks; ++j) {
        float* v = acc + 8 * j;
        const int c = at.c0 + 8 * j;
        if (p.bias) {
            if (c + 8 <= p.N) {
                add_bias8(v, ld_nc_u4(reinterpret_cast<const uint4*>(p.bias + c)));
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c + i < p.N) v[i] += __bfloat162float(p.bias[c + i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = linear_act_t<ACT>(v[i]);
        const uint32_t to = at.sub + Sub<C>::chunk(lane, j);
        if (p.res) {
            uint4 r = lds_u4(to);
            if (odd) {                                  // one column to the left: the next chunk's first word has the last
                const uint32_t n = j + 1 < Sub<C>::chunks ? lds_u32(at.sub + Sub<C>::chunk(lane, j + 1)) : last;
                r = make_uint4(__funnelshift_r(r.x, r.y, 16), __funnelshift_r(r.y, r.z, 16), __funnelshift_r(r.z, r.w, 16),
                               __funnelshift_r(r.w, n, 16));
            }
            add_bias8(v, r);
        }
        sts_u4(to, pack_bf16x8(v));
    }
}
template <int C>
__device__ __forceinline__ void epilogue_sub(const LinearArgs& p, const EpiAt& at, uint32_t last, float* acc) {
    switch (p.act) {
        case 1: return epilogue_sub_t<1, C>(p, at, last, acc);
        case 2: return epilogue_sub_t<2, C>(p, at, last, acc);
        case 3: return epilogue_sub_t<3, C>(p, at, last, acc);
        case 4: return epilogue_sub_t<4, C>(p, at, last, acc);
        default: return epilogue_sub_t<0, C>(p, at, last, acc);
    }
}

// Store to y.  tmY: y [T, N] bf16, box C x 32; used when N is a multiple of 8, and then asynchronous.
template <int C>
__device__ __forceinline__ void epilogue_store(const LinearArgs& p, const CUtensorMap* tmY, const EpiAt& at) {
    using S = Sub<C>;
    const int lane = threadIdx.x & 31;
    if (p.N % 8 == 0) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0 && at.t0 < p.T && at.c0 < p.N) {
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                             reinterpret_cast<uint64_t>(tmY)),
                         "r"(at.sub), "r"(at.c0), "r"(at.t0)
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        return;
    }
    quad_all(at, true);                                 // the quad's rows are whole
    constexpr int kLanes = kQuarters * S::words / 32, kRowWords = kQuarters * S::words;
#pragma unroll 2
    for (int i = 0; i < 8; ++i) {
        const int r = 8 * at.qtr + i, t = at.t0 + r;
        if (t >= p.T) break;
        const int odd = p.N & t & 1;
        __nv_bfloat16* row = p.y + static_cast<size_t>(t) * p.N + at.tile_c0;
#pragma unroll
        for (int k = 0; k < kLanes; ++k) {
            const int W = 32 * k + lane, c = at.tile_c0 + 2 * W + odd;
            uint32_t v = lds_u32(quad_word<C>(at, r, W));
            if (odd) {
                if (W == 0 && at.tile_c0 < p.N) *reinterpret_cast<uint16_t*>(row) = static_cast<uint16_t>(v);
                v >>= 16;
                if (W + 1 < kRowWords) v |= lds_u32(quad_word<C>(at, r, W + 1)) << 16;
            }
            if (c + 1 < p.N && (!odd || W + 1 < kRowWords)) *reinterpret_cast<uint32_t*>(row + 2 * W + odd) = v;
            else if (c < p.N) *reinterpret_cast<uint16_t*>(row + 2 * W + odd) = static_cast<uint16_t>(v);
        }
    }
    quad_all(at, true);                                 // the subtiles are free again
}
// Before the subtiles are written again: the stores have read them.
__device__ __forceinline__ void epilogue_store_wait() {
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
}
// Before the warp leaves.
__device__ __forceinline__ void epilogue_drain() {
    asm volatile("cp.async.wait_all;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// ---- single-thread roles: the whole warp runs the loop, so that addresses and descriptors stay in uniform
// registers, and one elected lane issues.  (With the loop in one lane of a divergent branch, issuing a
// stage's four MMAs and its commits took 350-550 cycles of moves to uniform registers.)
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0); }
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// ---- CTA pairs (cta_group::2): the even CTA issues the MMAs of both
__device__ __forceinline__ void tmem_alloc2(uint32_t* holder_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(holder_smem)),
                 "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Arrive on the barrier at this offset in both CTAs once the MMAs issued so far have finished.
__device__ __forceinline__ void mma_commit2(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_u32(bar)),
                 "h"(static_cast<uint16_t>(3)) : "memory");
}
// The same on this CTA's barrier alone.
__device__ __forceinline__ void mma_commit2_own(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ uint32_t pair_addr(uint32_t smem_addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr), "r"(rank));
    return r;
}
// A load into this CTA that counts on a barrier of the even CTA (bar: its cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
// Arrive on a barrier of either CTA of the pair, for what fences of their own order: an accumulator read
// out (tcgen05.fence), shared memory written for the other CTA's tcgen05 operations (fence.proxy.async).
// (A release at cluster scope here waits out the thread's loads in flight: about 1200 cycles.)
__device__ __forceinline__ void arrive_pair(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// After an abort, for copies whose barriers may never complete: long enough for any that is under way.
__device__ __forceinline__ void pause_for_copies() {
    const unsigned long long t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
}
// The end of a pair kernel's producer warp (it: stages issued; s, ph: the next one's place and parity): no copy is
// under way when the CTA leaves, whichever role gave up.  The MMAs have read the last stages, or else the even CTA's
// barriers, which count both CTAs' copies, complete.
template <int STAGES>
__device__ __forceinline__ void pair_copies_land(bool ok, uint64_t* full, uint64_t* empty, uint32_t it, uint32_t s, uint32_t ph,
                                                 uint32_t rank, volatile int* abort, int32_t* status) {
    if (it == 0 && ok) return;
    for (int i = 0; i < STAGES && ok; ++i) {
        ok = mbar_wait(&empty[s], ph, abort, status);   // no sleep: the kernel may end with this
        if (++s == STAGES) {
            s = 0;
            ph ^= 1;
        }
    }
    if (ok) return;
    if (rank == 0)
        for (uint32_t i = it < STAGES ? 0 : it - STAGES; i < it; ++i) drain_wait(&full[i % STAGES], (i / STAGES) & 1);
    pause_for_copies();
}

// Where an epilogue warp's waits ran out it leaves the unit in shared memory (owed[warp]; no unit at first), and at the
// kernel's end, where this takes no registers from the loop, writes NaN to its columns of that unit and of those that
// its pair owes after it: ROWS x N0 values a unit, the lane's rows one by one.
template <int C, int ROWS, int N0>
__device__ __forceinline__ void epilogue_owed(const LinearArgs& p, int u, int epi_warp, uint32_t rank) {
    const int mt = (p.T + ROWS - 1) / ROWS, total = mt * ((p.N + N0 - 1) / N0);
    const int quad = epi_warp & 3, qtr = epi_warp >> 2;
#pragma unroll 1
    for (; u < total; u += gridDim.x >> 1) {
        const int nb = u / mt, mb = u - nb * mt;
#pragma unroll 1
        for (int t = mb * ROWS + static_cast<int>(rank) * kTileM + quad * 32 + static_cast<int>(threadIdx.x & 31);
             t < min(p.T, (mb + 1) * ROWS); t += 2 * kTileM) {
            uint16_t* row = reinterpret_cast<uint16_t*>(p.y) + static_cast<size_t>(t) * p.N;
#pragma unroll 1
            for (int c0 = nb * N0 + C * qtr; c0 < (nb + 1) * N0; c0 += 4 * C)
#pragma unroll 1
                for (int c = c0; c < min(p.N, c0 + C); ++c) row[c] = 0x7fc0;
        }
    }
}

// Tiles of the pair kernels: 256 tokens, or two such blocks, x 128 columns (fp32 scales); 256 tokens x 192 or
// 256 columns (block-scaled).
constexpr int kPairM = 2 * kTileM;
constexpr int kPairN0 = 128, kPairNX = 192, kPairNW = 256;
// Columns of an output subtile.
constexpr int kSubCols0 = 32, kSubColsX = 48, kSubColsW = 32;

// Launch a pair kernel: one CTA an SM, clusters of two.
template <typename K>
inline cudaError_t launch_pair(K kernel, int threads, uint32_t smem, const LinearArgs& a, const LinearMaps& m,
                               int num_sms, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms / 2 * 2);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, m.x, m.w, m.sf, m.y, a);
}

}  // namespace moe
