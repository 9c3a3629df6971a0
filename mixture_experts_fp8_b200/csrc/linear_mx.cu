// linear_mx.cu -- the dense FP8 product on the block-scaled tensor core instruction (moe_linear,
// recipes 1 and 2): E4M3 tokens with a UE8M0 scale per 32 columns, E4M3 or E2M1 weights with a UE8M0
// scale per 32 K-elements.  tcgen05.mma.kind::mxf8f6f4.block_scale applies 2^(ex + ew) to every
// 32-deep block itself and accumulates the whole K in TMEM, so nothing is promoted.
//
// CTA pairs (cta_group::2), persistent: a tile is 256 tokens x 256 or 192 columns, each CTA of the pair
// holding 128 token rows and half of the weight rows.  What is taken to bound it, by a count of bytes (no
// counter shows the tensor core's operand reads), is shared memory: the MMAs of a 128-deep stage read the CTA's token rows and all of the tile's weight rows (48 KB at 256 columns, 40 at
// 192: 384 and 320 cycles), beside 32 (28) KB of TMA writes, 640 (544) cycles for MMAs of 512 (384).
// 192 columns leave TMEM for two accumulators beside the scale factors (12 columns a stage), so that a
// tile's epilogue overlaps the next tile's MMAs; 256 leave one, whose sums the epilogue takes into
// registers before it works on them, so that the MMAs wait for that alone.  (With 128 x 128 tiles of one CTA the same
// loop took 735 cycles a stage for MMAs of 256.)  Measured on normal data in short runs: 16384 x 4096 x 4096 211 us,
// 2.6 PFLOP/s (192 columns: 245), 4096 x 7168 x 7168 150 us, 2.8 PFLOP/s (165); at the power limit 245 (286) and 175
// (193).
//
// Scale factors: a CTA's SFA are its own rows', SFB the whole tile's in both CTAs; word 4i + c of a
// 512-byte atom = the four scale bytes of row 32c + i.  A 192-column tile's columns start in the middle of
// a weight atom when its index is odd: SFB then starts two TMEM columns in.
//
// Threads (640): warp 0 TMA producer, warp 1 MMA issuer (the even CTA's, for both), warp 2 the tokens'
// scale atoms, warp 3 idle, warps 4-19 epilogue (TMEM lanes 32 (w % 4).., 48 of the columns each, or
// twice 32).  Units go column block by column block, token blocks fastest.  Every wait is bounded.
#include "linear_common.cuh"

namespace moe {

namespace {

constexpr int kXThreads = 640;
constexpr int kXEpiWarps = 16;
constexpr int kXM = kPairM;
constexpr uint32_t kXA = kTileM * kTileK;         // 16 KB
constexpr uint32_t kXSf = 512;
constexpr uint32_t kXSfStage = 3 * kXSf;          // [SFA | SFB two atoms]
constexpr uint32_t kXTmemCols = 512;

// NX: columns of a tile.
template <int NX>
struct XL {
    static_assert(NX == kPairNX || NX == kPairNW, "tile columns");
    static constexpr int stages = NX == kPairNX ? 6 : 5;
    static constexpr int accs = NX == kPairNX ? 2 : 1;                        // accumulators
    static constexpr int sub_cols = NX == kPairNX ? kSubColsX : kSubColsW;    // of a subtile
    static constexpr int parts = NX / (4 * sub_cols);                         // a warp's subtiles, one after the other
    static constexpr uint32_t b_bytes = NX / 2 * kTileK;
    static constexpr uint32_t b = kXA;
    static constexpr uint32_t stage = kXA + b_bytes;
    static constexpr uint32_t sf_col0 = accs * NX;                            // scale factors after the accumulators
    static constexpr uint32_t out = stages * stage;                           // the epilogue's subtiles
    static constexpr uint32_t sf = out + kXEpiWarps * Sub<sub_cols>::bytes;
    static constexpr uint32_t bars = sf + stages * kXSfStage;
    static constexpr uint32_t nbars = 3 * stages + 5;     // full, sfready, empty, tfull[2], tempty[2], drain
    static constexpr uint32_t misc = bars + nbars * 8;
    static constexpr uint32_t owed = misc + 16;           // units that the epilogue warps gave up on
    static constexpr uint32_t end = owed + kXEpiWarps * 4;
    static constexpr uint32_t smem = end + 1024;
    static_assert(sf_col0 + stages * 12 <= kXTmemCols, "TMEM");
    static_assert(stage % 1024 == 0 && kXA % 1024 == 0 && out % 1024 == 0, "alignment");
    static_assert(smem <= 232448, "shared memory");
};

__device__ __forceinline__ void mma_mx2(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void sf_copy2(uint32_t tmem_col_addr, uint64_t sdesc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem_col_addr), "l"(sdesc) : "memory");
}

}  // namespace

template <int NX>
__global__ void __launch_bounds__(kXThreads, 1)
    k_linear_mx(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmSf, const __grid_constant__ CUtensorMap tmY, const LinearArgs p) {
    using X = XL<NX>;
    constexpr int kXStages = X::stages, kXN = NX, C = X::sub_cols;
    extern __shared__ uint8_t smem_raw[];
    const int mt = (p.T + kXM - 1) / kXM, nt = (p.N + kXN - 1) / kXN;
    const int total_units = mt * nt;
    const int KB = p.K / kTileK;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    // the same offsets in both CTAs: the dynamic shared memory starts at one address in every CTA
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + X::bars);     // the even CTA's count for both
    uint64_t* sfready = full + kXStages;                               // likewise
    uint64_t* empty = sfready + kXStages;                              // one in each CTA
    uint64_t* tfull = empty + kXStages;                                // one in each CTA
    uint64_t* tempty = tfull + 2;                                      // the even CTA's
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + X::misc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + X::misc + 4);
    int* owed = reinterpret_cast<int*>(smem + X::owed);

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kXStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&sfready[s], 2);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 2 * kXEpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
        prefetch_tmap(&tmSf);
        if (p.N % 8 == 0) prefetch_tmap(&tmY);
    }
    if (threadIdx.x < kXEpiWarps) owed[threadIdx.x] = INT32_MAX;
    if (warp == 1) tmem_alloc2(tmem_holder, kXTmemCols);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                                // both CTAs' barriers and TMEM are there
    tc_fence_after();
    pdl_wait_then_release();
    if (p.clear && blockIdx.x == 0 && threadIdx.x == 0) *p.status = MOE_OK;
    const uint32_t tmem_base = *tmem_holder;

    if (warp == 0) {
        // ---------------------------------------------------------------------- TMA producer
        const uint32_t b_bytes = p.recipe == 2 ? X::b_bytes / 2 : X::b_bytes;   // E2M1 weights arrive packed
        uint32_t it = 0, s = 0, ph = 1;
        bool ok = true;
        for (int u = pair; u < total_units && ok; u += pairs) {
            const int nb = u / mt, mb = u - nb * mt;
            const int row0 = mb * kXM + static_cast<int>(rank) * kTileM;
            const int brow0 = nb * kXN + static_cast<int>(rank) * (kXN / 2);
            for (int kb = 0; kb < KB; ++kb, ++it) {
                if (!mbar_wait<kProducerSleepNs>(&empty[s], ph, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                uint8_t* st = smem + s * X::stage;
                const uint32_t bar = pair_addr(smem_u32(&full[s]), 0);
                if (!fault_skip_stage(p.fault, it) && elect_one()) {   // debug builds: an injected fault
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * (kXA + b_bytes + 2 * kXSf));
                    tma_load_2d_pair(st, &tmA, kb * kTileK, row0, bar);
                    tma_load_2d_pair(st + X::b, &tmB, kb * kTileK, brow0, bar);
                    tma_load_3d_pair(smem + X::sf + s * kXSfStage + kXSf, &tmSf, 0, kb, nb * kXN / 128, bar);
                }
                __syncwarp();
                if (++s == kXStages) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        pair_copies_land<kXStages>(ok, full, empty, it, s, ph, rank, abort_flag, p.status);
    } else if (warp == 2) {
        // ---------------------------------------------------------------------- token-scale atoms
        // lane i writes the atom's row i: the scale words of tile rows i, 32+i, 64+i, 96+i (rows past T:
        // zero).  The words are fetched kSfAhead stages ahead of the stage being written (a register
        // ring), so that a load's latency is not paid per stage.
        constexpr int kSfAhead = 4;
        const int my_units = total_units > pair ? (total_units - 1 - pair) / pairs + 1 : 0;
        const long long n_stages = static_cast<long long>(my_units) * KB;
        int gu = pair, gkb = 0;                        // the fetch's own position
        auto fetch = [&]() {
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (gu < total_units) {
                const int r = (gu % mt) * kXM + static_cast<int>(rank) * kTileM + lane;
                const uint32_t* src = static_cast<const uint32_t*>(p.a_scale) + static_cast<size_t>(gkb) * p.a_pad + r;
                if (r < p.T) w.x = __ldg(src);
                if (r + 32 < p.T) w.y = __ldg(src + 32);
                if (r + 64 < p.T) w.z = __ldg(src + 64);
                if (r + 96 < p.T) w.w = __ldg(src + 96);
                if (++gkb == KB) {
                    gkb = 0;
                    gu += pairs;
                }
            }
            return w;
        };
        uint4 ring[kSfAhead];
#pragma unroll
        for (int d = 0; d < kSfAhead; ++d) ring[d] = fetch();
        uint32_t s = 0, ph = 1;
        bool ok = true;
        for (long long base = 0; base < n_stages && ok; base += kSfAhead) {
#pragma unroll
            for (int d = 0; d < kSfAhead; ++d) {
                if (base + d >= n_stages) break;
                const uint4 w = ring[d];
                ring[d] = fetch();
                if (!mbar_wait<kProducerSleepNs>(&empty[s], ph, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                *reinterpret_cast<uint4*>(smem + X::sf + s * kXSfStage + 16 * lane) = w;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // visible to tcgen05.cp
                __syncwarp();
                if (lane == 0) arrive_pair(pair_addr(smem_u32(&sfready[s]), 0));
                if (++s == kXStages) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // ------------------------------------------------------------------ MMA issuer, for the pair
            const uint32_t bfmt = p.recipe == 2 ? 5u : 0u;
            const uint64_t a_desc0 = sw128_kmajor_desc(smem_u32(smem)), b_desc0 = sw128_kmajor_desc(smem_u32(smem + X::b));
            const uint64_t sf_desc0 = sf_atom_desc(smem_u32(smem + X::sf));
            uint32_t s = 0, ph = 0, tile = 0;
            bool ok = true;
            for (int u = pair; u < total_units && ok; u += pairs, ++tile) {
                const int b = tile % X::accs;
                if (!mbar_wait<kIssuerSleepNs>(&tempty[b], ((tile / X::accs) & 1) ^ 1, abort_flag, p.status)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + static_cast<uint32_t>(b * kXN);
                const uint32_t sfb_off = 4 + (NX % 128 ? (u / mt & 1) * 2 : 0);
                for (int kb = 0; kb < KB; ++kb) {
                    if (!mbar_wait<kIssuerSleepNs>(&full[s], ph, abort_flag, p.status) ||
                        !mbar_wait<kIssuerSleepNs>(&sfready[s], ph, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = a_desc0 + s * (X::stage >> 4), bd = b_desc0 + s * (X::stage >> 4);
                    const uint64_t sfd = sf_desc0 + s * (kXSfStage >> 4);
                    const uint32_t sf_t = tmem_base + X::sf_col0 + s * 12;
                    if (elect_one()) {
                        sf_copy2(sf_t, sfd);
                        sf_copy2(sf_t + 4, sfd + (kXSf >> 4));
                        sf_copy2(sf_t + 8, sfd + 2 * (kXSf >> 4));
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k)
                            mma_mx2(d, ad + 2 * k, bd + 2 * k, mx_block_idesc(k, 0u, bfmt, kXM, kXN), sf_t, sf_t + sfb_off,
                                    (kb > 0 || k > 0) ? 1u : 0u);
                        mma_commit2(&empty[s]);
                        if (kb == KB - 1) mma_commit2(&tfull[b]);
                    }
                    __syncwarp();
                    if (++s == kXStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            if (elect_one()) mma_commit2_own(drain);
            __syncwarp();
            drain_wait(drain, 0);
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------------------------- epilogue
        const int quad = warp & 3;
        const int qtr = (warp - 4) >> 2;           // columns 48 qtr .. of the tile
        EpiAt at;
        at.qtr = qtr;
        at.quad = quad;
        at.quad_sub = smem_u32(smem + X::out) + static_cast<uint32_t>(quad) * Sub<C>::bytes;
        at.sub = at.quad_sub + static_cast<uint32_t>(4 * qtr) * Sub<C>::bytes;
        uint32_t tile = 0;
        for (int u = pair; u < total_units; u += pairs, ++tile) {
            const int nb = u / mt, mb = u - nb * mt;
            at.t0 = mb * kXM + static_cast<int>(rank) * kTileM + quad * 32;
            at.tile_c0 = nb * kXN;
            at.c0 = at.tile_c0 + C * qtr;
            const int b = tile % X::accs;
            uint32_t last;
            epilogue_store_wait();                 // the last tile's stores have read the subtile
            epilogue_residual<C>(p, at, last);
            const bool ok = mbar_wait(&tfull[b], (tile / X::accs) & 1, abort_flag, p.status);
            if (!epilogue_residual_wait(p, at, ok)) {
                if (lane == 0) owed[warp - 4] = u;
                break;
            }
            tc_fence_after();
            const uint32_t from = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(b * kXN + C * qtr);
            float acc[X::parts][C];
            if constexpr (X::parts == 1) {
                uint32_t v[32], w[16];
                MOE_TMEM_LD32(from, v);
                MOE_TMEM_LD16(from + 32, w);
                MOE_TMEM_WAIT_LD(v);
                MOE_TMEM_WAIT_LD16(w);
#pragma unroll
                for (int i = 0; i < 32; ++i) acc[0][i] = __uint_as_float(v[i]);
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[0][32 + i] = __uint_as_float(w[i]);
            } else {
                uint32_t v[32], w[32];
                MOE_TMEM_LD32(from, v);
                MOE_TMEM_LD32(from + 4 * C, w);
                MOE_TMEM_WAIT_LD(v);
                MOE_TMEM_WAIT_LD(w);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    acc[0][i] = __uint_as_float(v[i]);
                    acc[X::parts - 1][i] = __uint_as_float(w[i]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_pair(pair_addr(smem_u32(&tempty[b]), 0));   // the accumulator may be refilled now
            epilogue_sub<C>(p, at, last, acc[0]);
            epilogue_store<C>(p, &tmY, at);
            if constexpr (X::parts == 2) {
                at.tile_c0 += 4 * C;
                at.c0 += 4 * C;
                epilogue_store_wait();
                epilogue_residual<C>(p, at, last);
                epilogue_residual_wait(p, at, true);
                epilogue_sub<C>(p, at, last, acc[X::parts - 1]);
                epilogue_store<C>(p, &tmY, at);
            }
        }
        epilogue_drain();
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                                // neither CTA leaves while the other's MMAs or arrivals need it
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc2(tmem_base, kXTmemCols);
    }
    if (warp >= 4 && owed[warp - 4] < total_units) epilogue_owed<C, kXM, kXN>(p, owed[warp - 4], warp - 4, rank);
}

cudaError_t launch_linear_mx(const LinearArgs& a, const LinearMaps& m, int num_sms, cudaStream_t s) {
    return linear_mx_cols(a, num_sms) == kPairNW
               ? launch_pair(k_linear_mx<kPairNW>, kXThreads, XL<kPairNW>::smem, a, m, num_sms, s)
               : launch_pair(k_linear_mx<kPairNX>, kXThreads, XL<kPairNX>::smem, a, m, num_sms, s);
}

// The tile whose rounds are estimated to take less: a round is a time per K group and one for the tile's start and
// epilogue, 0.32 and 0.7 us with 192 columns, 0.38 and 0.9 with 256, fitted to 300 to 16384 tokens with K 512 to
// 7168.  Normal data, short runs: 16384 x 7168 x 2048 (7 rounds of 256, 10 of 192): 206 against 255 us; 512 x 2048 x
// 8192 (1 and 2): 12 against 14; but 1024 x 7168 x 2048 (1 and 1): 23.6 against 22.8, and 1237 x 768 x 4226 (2 and 2):
// 12.7 against 10.7.
int linear_mx_cols(const LinearArgs& a, int num_sms) {
    const long long pairs = num_sms / 2, mt = (a.T + kPairM - 1) / kPairM, KB = a.K / kTileK;
    auto rounds = [&](int cols) { return (mt * ((a.N + cols - 1) / cols) + pairs - 1) / pairs; };
    return rounds(kPairNW) * (38 * KB + 90) < rounds(kPairNX) * (32 * KB + 70) ? kPairNW : kPairNX;
}

}  // namespace moe
