// linear_mx.cu -- the dense FP8 product on the block-scaled tensor core instruction (moe_linear,
// recipes 1 and 2): E4M3 tokens with a UE8M0 scale per 32 columns, E4M3 or E2M1 weights with a UE8M0
// scale per 32 K-elements.  tcgen05.mma.kind::mxf8f6f4.block_scale applies 2^(ex + ew) to every
// 32-deep block itself and accumulates the whole K in TMEM, so nothing is promoted.
//
// Tiles of 128 tokens x 128 columns, persistent, two TMEM accumulators so that a tile's epilogue
// overlaps the next tile's MMAs.  Warp 0 loads by TMA, warp 1 issues, warp 2 builds the tokens'
// scale-factor atoms (word 4i + c of an atom = the four scale bytes of tile row 32c + i), warps 4-11
// are the epilogue.  Every wait is bounded.
#include "linear_common.cuh"

namespace moe {

namespace {

constexpr int kXStages = 5;
constexpr int kXThreads = 384;
constexpr int kXEpiWarps = 8;
constexpr int kXN = 128;
constexpr uint32_t kXA = kTileM * kTileK;         // 16 KB
constexpr uint32_t kXB = kXN * kTileK;            // 16 KB
constexpr uint32_t kXSf = 512;
constexpr uint32_t kXStage = kXA + kXB + 2 * kXSf + 1024;   // [A | B | SFA | SFB | pad]
constexpr uint32_t kXSfCol0 = 2 * kXN;            // scale factors after the two accumulators
constexpr uint32_t kXTmemCols = 512;
constexpr int kXStageCols = 16;
static_assert(kXSfCol0 + kXStages * 8 <= kXTmemCols, "TMEM");

struct XL {
    static constexpr uint32_t b = kXA;
    static constexpr uint32_t sfa = kXA + kXB;
    static constexpr uint32_t sfb = sfa + kXSf;
    static constexpr uint32_t stage = kXStages * kXStage;
    static constexpr uint32_t bars = stage + kXEpiWarps * 32 * (kXStageCols + 1) * 4;
    static constexpr uint32_t nbars = 3 * kXStages + 5;   // full, sfready, empty, tfull[2], tempty[2], drain
    static constexpr uint32_t misc = bars + nbars * 8;
    static constexpr uint32_t end = misc + 16;
};
static_assert(kXStage % 1024 == 0, "stage alignment");
constexpr uint32_t kXSmemBytes = XL::end + 1024;
static_assert(kXSmemBytes <= 232448, "shared memory");

}  // namespace

__global__ void __launch_bounds__(kXThreads, 1)
    k_linear_mx(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const LinearArgs p) {
    extern __shared__ uint8_t smem_raw[];
    const int mt = (p.T + kTileM - 1) / kTileM, nt = (p.N + kXN - 1) / kXN;
    const int total_units = mt * nt;
    const int KB = p.K / kTileK;

    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + XL::bars);
    uint64_t* sfready = full + kXStages;
    uint64_t* empty = sfready + kXStages;
    uint64_t* tfull = empty + kXStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + XL::misc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + XL::misc + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kXStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&sfready[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], kXEpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
    }
    if (warp == 1) tmem_alloc(tmem_holder, kXTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait_then_release();
    if (p.clear && blockIdx.x == 0 && threadIdx.x == 0) *p.status = MOE_OK;
    const uint32_t tmem_base = *tmem_holder;

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------------------------ TMA producer
            const uint32_t b_bytes = p.recipe == 2 ? kXB / 2 : kXB;   // E2M1 weights arrive packed
            uint32_t it = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < total_units && ok; u += gridDim.x) {
                const int nb = u / mt, mb = u - nb * mt;
                const uint8_t* sfb_src = static_cast<const uint8_t*>(p.w_scale) + static_cast<size_t>(nb) * KB * kXSf;
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    const int s = it % kXStages;
                    if (!mbar_wait<kProducerSleepNs>(&empty[s], ((it / kXStages) & 1) ^ 1, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    uint8_t* st = smem + s * kXStage;
                    mbar_arrive_expect_tx(&full[s], kXA + b_bytes + kXSf);
                    tma_load_2d(st, &tmA, kb * kTileK, mb * kTileM, &full[s]);
                    tma_load_2d(st + XL::b, &tmB, kb * kTileK, nb * kXN, &full[s]);
                    bulk_load(st + XL::sfb, sfb_src + static_cast<size_t>(kb) * kXSf, kXSf, &full[s]);
                }
            }
            if (!ok) {
                const uint32_t n = it < static_cast<uint32_t>(kXStages) ? it : kXStages;
                for (uint32_t i = it - n; i < it; ++i) drain_wait(&full[i % kXStages], (i / kXStages) & 1);
            }
        }
    } else if (warp == 2) {
        // ---------------------------------------------------------------------- token-scale atoms
        // lane i writes the atom's row i: the scale words of tile rows i, 32+i, 64+i, 96+i (the
        // scale rows reach 132 past T, so a ragged tile reads words that no stored row uses)
        uint32_t it = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < total_units && ok; u += gridDim.x) {
            const uint32_t* src = static_cast<const uint32_t*>(p.a_scale) + static_cast<size_t>(u % mt) * kTileM + lane;
            uint4 next = make_uint4(__ldg(src), __ldg(src + 32), __ldg(src + 64), __ldg(src + 96));
            for (int kb = 0; kb < KB; ++kb, ++it) {
                const uint4 w = next;
                if (kb + 1 < KB) {
                    src += p.a_pad;
                    next = make_uint4(__ldg(src), __ldg(src + 32), __ldg(src + 64), __ldg(src + 96));
                }
                const int s = it % kXStages;
                if (!mbar_wait<kProducerSleepNs>(&empty[s], ((it / kXStages) & 1) ^ 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                *reinterpret_cast<uint4*>(smem + s * kXStage + XL::sfa + 16 * lane) = w;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // visible to tcgen05.cp
                __syncwarp();
                if (lane == 0) mbar_arrive(&sfready[s]);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ------------------------------------------------------------------ MMA issuer
            const uint32_t bfmt = p.recipe == 2 ? 5u : 0u;
            uint32_t it = 0, tile = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < total_units && ok; u += gridDim.x, ++tile) {
                const int b = tile & 1;
                if (!mbar_wait<kIssuerSleepNs>(&tempty[b], ((tile >> 1) & 1) ^ 1, abort_flag, p.status)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + static_cast<uint32_t>(b * kXN);
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    const int s = it % kXStages;
                    if (!mbar_wait<kIssuerSleepNs>(&full[s], (it / kXStages) & 1, abort_flag, p.status) ||
                        !mbar_wait<kIssuerSleepNs>(&sfready[s], (it / kXStages) & 1, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t st = smem_u32(smem + s * kXStage);
                    const uint32_t sfa_t = tmem_base + kXSfCol0 + static_cast<uint32_t>(s * 8);
                    const uint32_t sfb_t = sfa_t + 4;
                    sf_copy(sfa_t, sf_atom_desc(st + XL::sfa));
                    sf_copy(sfb_t, sf_atom_desc(st + XL::sfb));
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k)
                        mma_mx(d, sw128_kmajor_desc(st + k * 32), sw128_kmajor_desc(st + XL::b + k * 32),
                               mx_block_idesc(k, 0u, bfmt, kTileM, kXN), sfa_t, sfb_t, (kb > 0 || k > 0) ? 1u : 0u);
                    mma_commit(&empty[s]);
                }
                if (!ok) break;
                mma_commit(&tfull[b]);
            }
            mma_commit(drain);
            drain_wait(drain, 0);
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------------------------- epilogue
        const int quad = warp & 3;
        const int h = (warp - 4) >> 2;             // columns h*64 .. h*64+63 of the tile
        float* stage = reinterpret_cast<float*>(smem + XL::stage) + (warp - 4) * 32 * (kXStageCols + 1);
        uint32_t tile = 0;
        for (int u = blockIdx.x; u < total_units; u += gridDim.x, ++tile) {
            const int nb = u / mt, mb = u - nb * mt;
            const int t0 = mb * kTileM + quad * 32, t = t0 + lane, c0 = nb * kXN + h * 64;
            const int b = tile & 1;
            if (!mbar_wait(&tfull[b], (tile >> 1) & 1, abort_flag, p.status)) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) +
                                   static_cast<uint32_t>(b * kXN + h * 64);
            uint32_t v[32], w[32];
            MOE_TMEM_LD32(taddr, v);
            MOE_TMEM_LD32(taddr + 32, w);
            MOE_TMEM_WAIT_LD(v);
            MOE_TMEM_WAIT_LD(w);
            float acc[64];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                acc[i] = __uint_as_float(v[i]);
                acc[32 + i] = __uint_as_float(w[i]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[b]);     // the accumulator may be refilled now
            if (p.N % 8 == 0) {
                if (t < p.T) {
                    linear_store32(p, acc, t, c0);
                    linear_store32(p, acc + 32, t, c0 + 32);
                }
            } else {
#pragma unroll
                for (int c = 0; c < 64; c += kXStageCols)
                    linear_store_any<kXStageCols>(p, stage, acc + c, t0, c0 + c);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, kXTmemCols);
    }
}

cudaError_t launch_linear_mx(const LinearArgs& a, const CUtensorMap& tmX, const CUtensorMap& tmW, int num_sms,
                             cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(k_linear_mx, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kXSmemBytes));
    if (e != cudaSuccess) return e;
    return launch_pdl(k_linear_mx, dim3(num_sms), dim3(kXThreads), kXSmemBytes, s, tmX, tmW, a);
}

}  // namespace moe
