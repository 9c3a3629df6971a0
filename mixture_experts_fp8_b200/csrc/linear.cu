// linear.cu -- the dense FP8 product with fp32 block scales (moe_linear, recipe 0), the weight
// transform of every recipe, and the choice of kernel.
//
//   y[t, n] = act( sum_g a_s[t,g] * w_s[g,n] * sum_{k in g} xq[t,k] * w[n,k] + b[n] ) + residual[t, n]
//
// The fp32 scales vary with the row, the column and the 128-deep group, so each group's partial
// leaves the tensor core and is promoted, acc += P * (a_s * w_s): two fp32 operations an element and
// group, 256 cycles for 128 x 128 at 128 a cycle, as long as the MMAs themselves.
//
// CTA pairs (cta_group::2), persistent: a tile is 128 columns of one or two row blocks of 256 tokens; each
// CTA of the pair holds 128 token rows a block and half of the weight rows, and promotes its own sums.
// Sums are handed over a step at a time: four 128-column TMEM buffers make two steps, and a step is two
// groups of one row block (the epilogue waits once, takes both partials into registers, 64 beside 32
// sums, hands the buffers back, and only then computes) or one group of two.  What bounds it is shared
// memory: a group of 128 x 128 sums reads the weight scales once a row (broadcasts, 270 cycles of its
// bandwidth), beside the operands' TMA writes (190) and the MMAs' reads (256).  Two row blocks share the
// loads of the weights and of their scales (a thread has a row of each).  The scales have a ring of
// their own, and an operand stage is free when its MMAs are done.  16384 x 4096 x 4096, codes of normal
// data, no epilogue inputs: 321 us, 1.7 PFLOP/s, in a short run at 1.9 GHz, and 375 us in a long one at the
// power limit (1.4 to 1.5 GHz); the tensor core active 45% of the time and the issue slots 56% (8192 tokens).
//
// Threads (640): warp 0 TMA producer, warp 1 MMA issuer (the even CTA's, for both), warp 2 scales,
// warp 3 idle, warps 4-19 epilogue (TMEM lanes 32 (w % 4).., 32 columns each).  Units go column block
// by column block, token blocks fastest, so that pairs working at the same time share weight tiles in
// L2.  Every wait is bounded.
#include "linear_common.cuh"

namespace moe {

namespace {

constexpr int kN = kPairN0;
constexpr int kSteps = 6;                              // scale slots, and barriers of finished steps
constexpr int kAhead = 3;                              // steps that the scales are fetched ahead
constexpr int kThreads = 640;
constexpr int kFirstEpiWarp = 4;
constexpr int kEpiWarps = 16;
// 640 threads launch with 96 registers each; warpgroup 0 keeps 32, the epilogue takes 112.
constexpr int kRegsLaunch = 96, kRegsLow = 32, kRegsHigh = 112;
static_assert(128 * kRegsLow + 512 * kRegsHigh == kThreads * kRegsLaunch, "register split");
constexpr uint32_t kABytes = kTileM * kTileK;
constexpr uint32_t kBBytes = kN / 2 * kTileK;
constexpr uint32_t kWsBytes = kN * 4;
constexpr uint32_t kSaBytes = kTileM * 4;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kStepCols = 2 * kN;

// RB: row blocks of a tile, 256 tokens each.
template <int RB>
struct L {
    static constexpr int stages = RB == 1 ? 7 : 4;
    static constexpr uint32_t stage = RB * kABytes + kBBytes;
    // a step's scales: the weights' of its groups and the rows' (RB 1: [weights, rows] of two groups; 2: [weights, rows, rows])
    static constexpr uint32_t group_scales = kWsBytes + kSaBytes;
    static constexpr uint32_t slot = RB == 1 ? 2 * group_scales : kWsBytes + 2 * kSaBytes;
    static constexpr uint32_t out = stages * stage;
    static constexpr uint32_t sc = out + kEpiWarps * Sub<kSubCols0>::bytes;
    static constexpr uint32_t bars = sc + kSteps * slot;
    // full[stages], empty[stages], tempty[2], tfull[kSteps], drain
    static constexpr uint32_t nbars = 2 * stages + kSteps + 3;
    static constexpr uint32_t misc = bars + nbars * 8;    // tmem holder, abort flag
    static constexpr uint32_t owed = misc + 16;           // units that the epilogue warps gave up on
    static constexpr uint32_t end = owed + kEpiWarps * 4;
    static constexpr uint32_t smem = end + 1024;          // + slack to align the base to 1024 bytes
    static_assert((bars + 16 * stages) % 16 == 0, "the two tempty barriers are one bit apart");
    static_assert(stage % 1024 == 0 && out % 512 == 0 && slot % 16 == 0, "alignment");
    static_assert(smem <= 232448, "shared memory");
};

__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

// A load at a constant offset from a shared-memory address (the offset stays in the instruction).
template <int OFF>
__device__ __forceinline__ float4 lds_f32x4_at(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4+%5];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a), "n"(OFF)
                 : "memory");
    return v;
}

// acc[j] += P[j] * (sa * ws[j]) from column 4 J on (packed fp32x2; each lane rounds as scalars would);
// OFF: the group's place in the scale slot.
template <int OFF, int J>
__device__ __forceinline__ void promote(float2 (&acc)[16], const uint32_t (&v)[32], uint32_t sc, float2 sa2) {
    if constexpr (J < 8) {
        const float4 w4 = lds_f32x4_at<OFF + 16 * J>(sc);
        const float2 s0 = __fmul2_rn(make_float2(w4.x, w4.y), sa2);
        const float2 s1 = __fmul2_rn(make_float2(w4.z, w4.w), sa2);
        acc[2 * J] = __ffma2_rn(make_float2(__uint_as_float(v[4 * J]), __uint_as_float(v[4 * J + 1])), s0, acc[2 * J]);
        acc[2 * J + 1] = __ffma2_rn(make_float2(__uint_as_float(v[4 * J + 2]), __uint_as_float(v[4 * J + 3])), s1,
                                    acc[2 * J + 1]);
        promote<OFF, J + 1>(acc, v, sc, sa2);
    }
}

// Two rows with the same columns, sixteen of them: acc[r][j] += P[r][j] * (s[r] * ws[j]) from column 4 J on; the weight
// scales are loaded once for both.
template <int OFF, int J>
__device__ __forceinline__ void promote2(float2* a0, float2* a1, const uint32_t (&v0)[16], const uint32_t (&v1)[16], uint32_t sc,
                                         float2 s0, float2 s1) {
    if constexpr (J < 4) {
        const float4 w4 = lds_f32x4_at<OFF + 16 * J>(sc);
        const float2 wa = make_float2(w4.x, w4.y), wb = make_float2(w4.z, w4.w);
        auto p2 = [](const uint32_t (&v)[16], int i) { return make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])); };
        a0[2 * J] = __ffma2_rn(p2(v0, 4 * J), __fmul2_rn(wa, s0), a0[2 * J]);
        a1[2 * J] = __ffma2_rn(p2(v1, 4 * J), __fmul2_rn(wa, s1), a1[2 * J]);
        a0[2 * J + 1] = __ffma2_rn(p2(v0, 4 * J + 2), __fmul2_rn(wb, s0), a0[2 * J + 1]);
        a1[2 * J + 1] = __ffma2_rn(p2(v1, 4 * J + 2), __fmul2_rn(wb, s1), a1[2 * J + 1]);
        promote2<OFF, J + 1>(a0, a1, v0, v1, sc, s0, s1);
    }
}

// One arrival from lane 0 of the warp on a barrier of the cluster (arrive_pair), predicated inside the asm.
__device__ __forceinline__ void arrive_pair_lane0(uint32_t bar, int lane) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"(lane)
        : "memory");
}

}  // namespace

template <int RB>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear_fp32(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap, const __grid_constant__ CUtensorMap tmY, const LinearArgs p) {
    using S = L<RB>;
    constexpr int kStages = S::stages, kM = RB * kPairM;
    constexpr int kGroups = RB == 1 ? 2 : 1;           // K groups of a step
    extern __shared__ uint8_t smem_raw[];
    const int mt = (p.T + kM - 1) / kM, nt = (p.N + kN - 1) / kN;
    const int total_units = mt * nt;
    const int KB = p.K / kTileK;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::bars);      // the even CTA's count for both
    uint64_t* empty = full + kStages;                                  // one in each CTA
    uint64_t* tempty = empty + kStages;                                // the even CTA's
    uint64_t* tfull = tempty + 2;                                      // in each CTA: a step's MMAs and scales
    uint64_t* drain = tfull + kSteps;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + S::misc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::misc + 4);
    int* owed = reinterpret_cast<int*>(smem + S::owed);

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < kSteps; ++s) mbar_init(&tfull[s], 2);      // the MMA commit, and the scales' producer
        for (int b = 0; b < 2; ++b) mbar_init(&tempty[b], 2 * kEpiWarps);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
        if (p.N % 8 == 0) prefetch_tmap(&tmY);
    }
    if (threadIdx.x < kEpiWarps) owed[threadIdx.x] = INT32_MAX;
    if (warp == 1) tmem_alloc2(tmem_holder, kTmemCols);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                                // both CTAs' barriers and TMEM are there
    tc_fence_after();
    pdl_wait_then_release();
    if (p.clear && blockIdx.x == 0 && threadIdx.x == 0) *p.status = MOE_OK;
    const uint32_t tmem_base = *tmem_holder;
    constexpr int MPG = kTileK / 32;

    if (warp < kFirstEpiWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
        if (warp == 0) {
            // -------------------------------------------------------------- TMA producer
            uint32_t it = 0, s = 0, ph = 1;
            bool ok = true;
            for (int u = pair; u < total_units && ok; u += pairs) {
                const int nb = u / mt, mb = u - nb * mt;
                const int row0 = mb * kM + static_cast<int>(rank) * kTileM;
                const int brow0 = nb * kN + static_cast<int>(rank) * (kN / 2);
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    if (!mbar_wait<kProducerSleepNs>(&empty[s], ph, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = pair_addr(smem_u32(&full[s]), 0);
                    if (!fault_skip_stage(p.fault, it) && elect_one()) {   // debug builds: an injected fault
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * S::stage);
#pragma unroll
                        for (int b = 0; b < RB; ++b)
                            tma_load_2d_pair(smem + s * S::stage + b * kABytes, &tmA, kb * kTileK, row0 + b * kPairM, bar);
                        tma_load_2d_pair(smem + s * S::stage + RB * kABytes, &tmB, kb * kTileK, brow0, bar);
                    }
                    __syncwarp();
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            pair_copies_land<kStages>(ok, full, empty, it, s, ph, rank, abort_flag, p.status);
        } else if (warp == 2) {
            // -------------------------------------------------------------- scales
            // Step g's scales go to slot g % kSteps and count on that slot's barrier.  The slot was last
            // read for step g - kSteps; the MMAs of step g - kAhead are issued only when every epilogue
            // warp has taken the partials of step g - kAhead - 2 (two steps of TMEM), and so has finished
            // step g - kAhead - 3 = g - kSteps.
            static_assert(kAhead + 3 == kSteps, "a slot is read out before it is filled again");
            const int n_pad = (p.N + kLinearPad - 1) / kLinearPad * kLinearPad;
            uint32_t it = 0;
            bool ok = true;
            for (int u = pair; u < total_units && ok; u += pairs) {
                const int nb = u / mt, mb = u - nb * mt;
                const int row0 = mb * kM + static_cast<int>(rank) * kTileM;
                uint32_t a_bytes[RB];                  // the scale rows reach 132 past T
#pragma unroll
                for (int b = 0; b < RB; ++b) a_bytes[b] = row0 + b * kPairM < p.T ? kSaBytes : 0u;
                const float* ws_src = static_cast<const float*>(p.w_scale) + nb * kN;
                const float* sa_src = static_cast<const float*>(p.a_scale) + row0;
                for (int kb = 0; kb < KB; kb += kGroups, ++it) {
                    if (it >= kAhead) {
                        const uint32_t g = it - kAhead;
                        if (!mbar_wait<kProducerSleepNs>(&tfull[g % kSteps], (g / kSteps) & 1, abort_flag, p.status)) {
                            ok = false;
                            break;
                        }
                    }
                    const int s = it % kSteps, n = min(kGroups, KB - kb);
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&tfull[s], static_cast<uint32_t>(n) * (kWsBytes + a_bytes[0] + (RB == 2 ? a_bytes[RB - 1] : 0u)));
                        for (int i = 0; i < n; ++i) {
                            uint8_t* slot = smem + S::sc + s * S::slot + i * S::group_scales;
                            bulk_load(slot, ws_src + static_cast<size_t>(kb + i) * n_pad, kWsBytes, &tfull[s]);
#pragma unroll
                            for (int b = 0; b < RB; ++b)
                                if (a_bytes[b])
                                    bulk_load(slot + kWsBytes + b * kSaBytes,
                                              sa_src + static_cast<size_t>(kb + i) * p.a_pad + b * kPairM, kSaBytes, &tfull[s]);
                        }
                    }
                    __syncwarp();
                }
            }
            // the last steps' copies land; after an abort their steps' barriers may never complete
            for (uint32_t g = it < kAhead ? 0 : it - kAhead; g < it && ok; ++g)
                ok = mbar_wait(&tfull[g % kSteps], (g / kSteps) & 1, abort_flag, p.status);
            if (!ok) pause_for_copies();
        } else if (warp == 1 && rank == 0) {
            // -------------------------------------------------------------- MMA issuer, for the pair
            const uint32_t idesc = f8_idesc(kPairM, kN);
            const uint64_t a_desc0 = sw128_kmajor_desc(smem_u32(smem));
            const uint64_t b_desc0 = sw128_kmajor_desc(smem_u32(smem + RB * kABytes));
            uint32_t s = 0, ph = 0, buf = 0, bph = 0, step = 0;
            bool ok = true;
            for (int u = pair; u < total_units && ok; u += pairs) {
                for (int kb = 0; kb < KB; ++kb) {
                    const int half = RB == 1 ? kb & 1 : 0;         // of the step's TMEM
                    if ((half == 0 && !mbar_wait<kIssuerSleepNs>(&tempty[buf], bph ^ 1, abort_flag, p.status)) ||
                        !mbar_wait<kIssuerSleepNs>(&full[s], ph, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = a_desc0 + s * (S::stage >> 4), bd = b_desc0 + s * (S::stage >> 4);
                    const uint32_t d = tmem_base + buf * kStepCols + half * kN;
                    const bool last = RB == 2 || half || kb == KB - 1;   // the step is complete
                    if (elect_one()) {
#pragma unroll
                        for (int b = 0; b < RB; ++b)
#pragma unroll
                            for (int m = 0; m < MPG; ++m)
                                mma_f8_pair(d + b * kN, ad + b * (kABytes >> 4) + 2 * m, bd + 2 * m, idesc, m > 0 ? 1u : 0u);
                        mma_commit2(&empty[s]);
                        if (last) mma_commit2(&tfull[step]);
                    }
                    __syncwarp();
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                    if (last) {
                        if (++step == kSteps) step = 0;
                        buf ^= 1;
                        bph ^= buf ^ 1;                // flips after both steps of TMEM were used
                    }
                }
            }
            if (elect_one()) mma_commit2_own(drain);
            __syncwarp();
            drain_wait(drain, 0);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
        // ------------------------------------------------------------------ epilogue
        const int quad = warp & 3;                     // TMEM lanes 32*quad .. 32*quad+31
        const int qtr = (warp - kFirstEpiWarp) >> 2;
        EpiAt at;
        at.qtr = qtr;
        at.quad = quad;
        at.quad_sub = smem_u32(smem + S::out) + static_cast<uint32_t>(quad) * Sub<kSubCols0>::bytes;
        at.sub = at.quad_sub + static_cast<uint32_t>(4 * qtr) * Sub<kSubCols0>::bytes;
        const uint32_t abort_at = smem_u32(smem + S::misc + 4);
        // the step's barrier, weight scales, TMEM and TMEM barrier (256 columns and 8 bytes apart)
        const uint32_t tf0 = smem_u32(tfull), tf_end = tf0 + 8 * kSteps;
        const uint32_t sc0 = smem_u32(smem + S::sc) + static_cast<uint32_t>(32 * qtr * 4);
        const uint32_t sa_off = kWsBytes + static_cast<uint32_t>((quad * 32 + lane - 32 * qtr) * 4);   // from there, the row's scale
        uint32_t tf_at = tf0, sc_at = sc0, ph = 0;
        uint32_t t_at = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(32 * qtr);
        uint32_t te_at = pair_addr(smem_u32(tempty), 0);
        bool ok = true;
        for (int u = pair; u < total_units; u += pairs) {
            const int nb = u / mt, mb = u - nb * mt;
            at.t0 = mb * kM + static_cast<int>(rank) * kTileM + quad * 32;
            at.tile_c0 = nb * kN;
            at.c0 = at.tile_c0 + 32 * qtr;
            uint32_t last;
            epilogue_store_wait();                     // the last tile's store has read the subtile
            epilogue_residual<kSubCols0>(p, at, last);
            float2 acc2[RB][16];
#pragma unroll
            for (int i = 0; i < 16 * RB; ++i) acc2[i / 16][i % 16] = make_float2(0.0f, 0.0f);
            for (int kb = 0; kb < KB; kb += kGroups) {
                if (!mbar_wait_at(tf_at, ph, abort_at, p.status)) {   // the partials and their scales
                    ok = false;
                    break;
                }
                tc_fence_after();
                if constexpr (RB == 1) {
                    const bool two = kb + 1 < KB;
                    uint32_t va[32], vb[32];
                    MOE_TMEM_LD32(t_at, va);
                    if (two) MOE_TMEM_LD32(t_at + kN, vb);
                    const float s0 = ld_shared_f32(sc_at + sa_off), s1 = two ? ld_shared_f32(sc_at + sa_off + S::group_scales) : 0.0f;
                    MOE_TMEM_WAIT_LD(va);
                    if (two) MOE_TMEM_WAIT_LD(vb);
                    // the warp holds its partials: hand the buffers back
                    tc_fence_before();
                    arrive_pair_lane0(te_at, lane);
                    promote<0, 0>(acc2[0], va, sc_at, make_float2(s0, s0));
                    if (two) promote<S::group_scales, 0>(acc2[0], vb, sc_at, make_float2(s1, s1));
                } else {
                    uint32_t va[16], vb[16];
                    MOE_TMEM_LD16(t_at, va);
                    MOE_TMEM_LD16(t_at + kN, vb);
                    const float s0 = ld_shared_f32(sc_at + sa_off), s1 = ld_shared_f32(sc_at + sa_off + kSaBytes);
                    MOE_TMEM_WAIT_LD16(va);
                    MOE_TMEM_WAIT_LD16(vb);
                    promote2<0, 0>(acc2[0], acc2[RB - 1], va, vb, sc_at, make_float2(s0, s0), make_float2(s1, s1));
                    MOE_TMEM_LD16(t_at + 16, va);
                    MOE_TMEM_LD16(t_at + 16 + kN, vb);
                    MOE_TMEM_WAIT_LD16(va);
                    MOE_TMEM_WAIT_LD16(vb);
                    tc_fence_before();
                    arrive_pair_lane0(te_at, lane);
                    promote2<64, 0>(acc2[0] + 8, acc2[RB - 1] + 8, va, vb, sc_at, make_float2(s0, s0), make_float2(s1, s1));
                }
                // the scales were read through the generic proxy; the next bulk copy into this slot is an
                // async-proxy write: order the reads before it (the next step's arrival carries that on)
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tf_at += 8;
                sc_at += S::slot;
                if (tf_at == tf_end) {
                    tf_at = tf0;
                    sc_at = sc0;
                    ph ^= 1;
                }
                t_at ^= kStepCols;
                te_at ^= 8;
            }
            ok = epilogue_residual_wait(p, at, ok);
            if (!ok) {
                if (lane == 0) owed[warp - kFirstEpiWarp] = u;
                break;
            }
            epilogue_sub<kSubCols0>(p, at, last, reinterpret_cast<float*>(acc2[0]));
            epilogue_store<kSubCols0>(p, &tmY, at);
            if constexpr (RB == 2) {                   // the second row block through the same subtile
                at.t0 += kPairM;
                epilogue_store_wait();
                epilogue_residual<kSubCols0>(p, at, last);
                epilogue_residual_wait(p, at, true);
                epilogue_sub<kSubCols0>(p, at, last, reinterpret_cast<float*>(acc2[RB - 1]));
                epilogue_store<kSubCols0>(p, &tmY, at);
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
        tmem_dealloc2(tmem_base, kTmemCols);
    }
    if (warp >= kFirstEpiWarp && owed[warp - kFirstEpiWarp] < total_units)
        epilogue_owed<kSubCols0, kM, kN>(p, owed[warp - kFirstEpiWarp], warp - kFirstEpiWarp, rank);
}

template <int RB>
static cudaError_t launch_fp32(const LinearArgs& a, const LinearMaps& m, int num_sms, cudaStream_t s) {
    // The register split above must fit what the block is launched with, or setmaxnreg.inc would
    // wait forever: refuse to launch otherwise.
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, k_linear_fp32<RB>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs * kThreads < kRegsLow * 128 + kRegsHigh * 512) return cudaErrorInvalidConfiguration;
    return launch_pair(k_linear_fp32<RB>, kThreads, L<RB>::smem, a, m, num_sms, s);
}

// Tiles of 512 tokens where their rounds are estimated to take no longer than those of 256: a round is a time per K
// group and one for the tile's start and epilogue, 0.58 and 2.5 us against 0.34 and 0.9, fitted to 2048 to 16384
// tokens with K 512 to 7168.  Normal data, short runs of 12 calls on three sets of buffers: 16384 x 4096 x 4096: 321 us
// against 335; 16384 x 7168 x 2048: 285 against 346; in 7 rounds instead of 13, 4096 x 7168 x 7168: 224 against 241;
// but in 3 instead of 5, 2560 x 4096 x 4096: 59 against 58, and with four groups, 8192 x 512 x 6144: 48 against 46.
// (Long runs, at the power limit: 375 and 380, 340 and 404, 260 and 279; 63 and 64, 51 and 50.)
cudaError_t launch_linear_fp32(const LinearArgs& a, const LinearMaps& m, int num_sms, cudaStream_t s) {
    const long long pairs = num_sms / 2, nt = (a.N + kN - 1) / kN, KB = a.K / kTileK;
    auto rounds = [&](int rows) { return ((a.T + rows - 1) / rows * nt + pairs - 1) / pairs; };
    return rounds(2 * kPairM) * (58 * KB + 250) <= rounds(kPairM) * (34 * KB + 90) ? launch_fp32<2>(a, m, num_sms, s)
                                                                                  : launch_fp32<1>(a, m, num_sms, s);
}

// The narrow kernel takes a product when its estimated time is below the pair kernel's.  Both estimates
// (ns) are a start and a time per K group of the busiest SM, fitted to products of 16 to 2048 tokens with
// K 512 to 7168 and N 512 to 12288 in a graph, the pair kernel's with tiles of 256 tokens and 128 or 192 columns
// alone (where a larger tile is chosen below, it takes less than this says); two CTAs that share an SM count as two
// rounds of its K groups.  Of 252 products 9 go to a kernel that is more than 8% slower: 512 x 7168 x 2048 with 4-bit
// weights to the pair kernel, 17.5 us against 15.4, 16 x 4096 x 12288 likewise, 14.7 against 9.5.  Narrow 3.3 us (32 tokens) or 5 us (64) for each round of two
// CTAs an SM, 0.32 us a group (block-scaled 0.26); pair 3.2 us and 0.28 us a group (4.2 us, 0.225 us).  At
// 64 x 2816 x 2816 that is 6.9 against 9.4 us (measured 7.8 and 9.5), at 256 tokens 12 against 9.4 (12.6
// and 9.8).
bool linear_is_narrow(int T, int N, int K, int recipe, int num_sms) {
    const long long KB = K / kTileK;
    const int nt = linear_narrow_tokens(T), split = linear_narrow_split(T, N, K, num_sms);
    const long long ctas = static_cast<long long>((N + kTileM - 1) / kTileM) * ((T + nt - 1) / nt) * split;
    if ((T + nt - 1) / nt > 65535) return false;       // grid.z
    const int wn = recipe == 0 ? kPairN0 : kPairNX;
    const long long units = static_cast<long long>((N + wn - 1) / wn) * ((T + kPairM - 1) / kPairM);
    const long long pairs = num_sms / 2;
    const long long narrow = (ctas + 2 * num_sms - 1) / (2 * num_sms) * (nt == 32 ? 3300 : 5000) +
                             (ctas + num_sms - 1) / num_sms * ((KB + split - 1) / split) * (recipe == 0 ? 320 : 260);
    const long long wide = (recipe == 0 ? 3200 : 4200) + (units + pairs - 1) / pairs * KB * (recipe == 0 ? 280 : 225);
    return narrow < wide;
}

LinearBoxes linear_boxes(const LinearArgs& a, int num_sms) {
    if (linear_is_narrow(a.T, a.N, a.K, a.recipe, num_sms))
        return {static_cast<uint32_t>(linear_narrow_tokens(a.T)), kTileM, 0, false};
    if (a.recipe == 0) return {kTileM, kPairN0 / 2, kSubCols0, true};
    return linear_mx_cols(a, num_sms) == kPairNW ? LinearBoxes{kTileM, kPairNW / 2, kSubColsW, true}
                                                 : LinearBoxes{kTileM, kPairNX / 2, kSubColsX, true};
}

cudaError_t launch_linear(const LinearArgs& a, const LinearMaps& m, int num_sms, cudaStream_t s) {
    if (linear_is_narrow(a.T, a.N, a.K, a.recipe, num_sms)) return launch_linear_narrow(a, m, num_sms, s);
    return a.recipe == 0 ? launch_linear_fp32(a, m, num_sms, s) : launch_linear_mx(a, m, num_sms, s);
}

// ------------------------------------------------------------------------------------------
// Weight transform (once per set of weights): codes [K, N] -> K-major [N, K] (4-bit codes stay two
// per byte, along K), scales fp32 [K/128, N] -> [K/128, n_pad], or UE8M0 [K/32, N] -> 512-byte atoms
// [n_pad/128][K/128] (byte 16i + 4c + k of an atom: column 32c + i, 32-deep block k).  Columns past N
// get a scale of zero; their codes are the tensor map's zero fill.
__global__ void __launch_bounds__(256) k_linear_codes(const uint8_t* src, uint8_t* dst, int K, int N, int fp4) {
    __shared__ uint8_t tile[64][65];
    const int k0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
    for (int i = threadIdx.x; i < 64 * 64; i += 256) {
        const int kk = i >> 6, nn = i & 63;
        if (n0 + nn < N) {
            const size_t at = static_cast<size_t>(k0 + kk) * N + n0 + nn;    // K is a multiple of 128
            tile[kk][nn] = fp4 ? (src[at >> 1] >> (4 * (nn & 1))) & 15 : src[at];
        }
    }
    __syncthreads();
    const int per = fp4 ? 32 : 64;                     // bytes of a K run of 64 codes
    for (int i = threadIdx.x; i < 64 * per; i += 256) {
        const int nn = i / per, j = i - nn * per;
        if (n0 + nn >= N) continue;
        if (fp4) dst[(static_cast<size_t>(n0 + nn) * K + k0) / 2 + j] = tile[2 * j][nn] | (tile[2 * j + 1][nn] << 4);
        else dst[static_cast<size_t>(n0 + nn) * K + k0 + j] = tile[j][nn];
    }
}

__global__ void __launch_bounds__(256) k_linear_scales(const void* src, void* dst, int K, int N, int n_pad, int recipe) {
    const size_t words = static_cast<size_t>(K / 128) * n_pad;
    for (size_t i = blockIdx.x * 256ull + threadIdx.x; i < words; i += static_cast<size_t>(gridDim.x) * 256) {
        if (recipe == 0) {
            const int n = static_cast<int>(i % n_pad);
            const size_t kb = i / n_pad;
            static_cast<float*>(dst)[i] = n < N ? static_cast<const float*>(src)[kb * N + n] : 0.0f;
        } else {                                       // word i of the atoms
            const int w = static_cast<int>(i & 127);
            const size_t atom = i >> 7;                // nb * (K/128) + kb
            const size_t kb = atom % (K / 128);
            const int n = static_cast<int>(atom / (K / 128)) * 128 + 32 * (w & 3) + (w >> 2);
            uint32_t v = 0;
            if (n < N)
                for (int k = 0; k < 4; ++k)
                    v |= static_cast<uint32_t>(static_cast<const uint8_t*>(src)[(kb * 4 + k) * N + n]) << (8 * k);
            static_cast<uint32_t*>(dst)[i] = v;
        }
    }
}

cudaError_t launch_linear_transform(const LinearTransformArgs& a, cudaStream_t s) {
    k_linear_codes<<<dim3((a.N + 63) / 64, a.K / 64), 256, 0, s>>>(a.w, a.w_t, a.K, a.N, a.recipe == 2);
    k_linear_scales<<<592, 256, 0, s>>>(a.ws, a.ws_t, a.K, a.N, linear_n_pad(a.N), a.recipe);
    return cudaGetLastError();
}

}  // namespace moe
