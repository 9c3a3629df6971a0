// linear.cu -- the dense FP8 product with fp32 block scales (moe_linear, recipe 0), the weight
// transform of every recipe, and the choice of kernel.
//
//   y[t, n] = act( sum_g a_s[t,g] * w_s[g,n] * sum_{k in g} xq[t,k] * w[n,k] + b[n] ) + residual[t, n]
//
// The fp32 scales vary with the row, the column and the 128-deep group, so each group's partial
// leaves the tensor core and is promoted, acc += P * (a_s * w_s): the FP32 pipe does as much work as
// the tensor core.  Persistent, one CTA per SM, tiles of 128 tokens x 256 columns, as the layer's
// wide GEMM lays them out: warp 0 loads by TMA, warp 1 issues tcgen05.mma.kind::f8f6f4 (M 128, N 256,
// K 32) into one of two 256-column TMEM buffers per group, warps 4-19 promote into registers and run
// the epilogue.  Units go column block by column block, token blocks fastest, so that CTAs working
// at the same time share a weight tile in L2.  Every wait is bounded.
#include "linear_common.cuh"

namespace moe {

namespace {

constexpr int kStages = 4;
constexpr int kThreads = 640;
constexpr int kFirstEpiWarp = 4;
constexpr int kEpiWarps = 16;
constexpr int kCols = kTileN / 4;                  // columns per epilogue thread (32 per half)
constexpr int kHalf = kTileN / 2;
// 640 threads launch with 96 registers each; warpgroup 0 keeps 32, the epilogue takes 112.
constexpr int kRegsLaunch = 96, kRegsLow = 32, kRegsHigh = 112;
static_assert(128 * kRegsLow + 512 * kRegsHigh == kThreads * kRegsLaunch, "register split");
constexpr uint32_t kABytes = kTileM * kTileK;
constexpr uint32_t kBBytes = kTileN * kTileK;
constexpr uint32_t kWsBytes = kTileN * 4;
constexpr uint32_t kSaBytes = kTileM * 4;
constexpr uint32_t kScaleSlot = 2048;
constexpr uint32_t kTmemCols = 2 * kTileN;
constexpr int kStageCols = 8;                      // columns a warp stages at once when N is not a multiple of 8

struct L {
    static constexpr uint32_t a = 0;
    static constexpr uint32_t b = a + kStages * kABytes;
    static constexpr uint32_t sc = b + kStages * kBBytes;
    static constexpr uint32_t stage = sc + kStages * kScaleSlot;
    static constexpr uint32_t full = stage + kEpiWarps * 32 * (kStageCols + 1) * 4;
    static constexpr uint32_t empty = full + 8 * kStages;
    static constexpr uint32_t tfull = empty + 8 * kStages;
    static constexpr uint32_t tempty = tfull + 16;
    static constexpr uint32_t drain = tempty + 16;
    static constexpr uint32_t misc = drain + 8;    // tmem holder, abort flag
    static constexpr uint32_t end = misc + 16;
};
static_assert(kWsBytes + kSaBytes <= kScaleSlot, "scale slot");
constexpr uint32_t kSmemBytes = L::end + 1024;     // + slack to align the base to 1024 bytes
static_assert(kSmemBytes <= 232448, "shared memory");

// acc[a0 + j] += P[j] * (sa * ws[j]) for j < 16 (packed fp32x2; each lane rounds as scalars would).
__device__ __forceinline__ void promote16(float2 (&acc)[kCols / 2], const uint32_t (&v)[16], uint32_t ws, int a0,
                                          float2 sa2) {
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
        const float4 w4 = ld_shared_f32x4(ws + 4 * j);
        const float2 s0 = __fmul2_rn(make_float2(w4.x, w4.y), sa2);
        const float2 s1 = __fmul2_rn(make_float2(w4.z, w4.w), sa2);
        acc[(a0 + j) / 2] = __ffma2_rn(make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), s0,
                                       acc[(a0 + j) / 2]);
        acc[(a0 + j) / 2 + 1] = __ffma2_rn(make_float2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])), s1,
                                           acc[(a0 + j) / 2 + 1]);
    }
}

}  // namespace

__global__ void __launch_bounds__(kThreads, 1)
    k_linear_fp32(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const LinearArgs p) {
    extern __shared__ uint8_t smem_raw[];
    const int mt = (p.T + kTileM - 1) / kTileM, nt = (p.N + kTileN - 1) / kTileN;
    const int total_units = mt * nt;
    const int KB = p.K / kTileK;
    const int n_pad = (p.N + kLinearPad - 1) / kLinearPad * kLinearPad;

    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::full);
    uint64_t* empty = reinterpret_cast<uint64_t*>(smem + L::empty);
    uint64_t* tfull = reinterpret_cast<uint64_t*>(smem + L::tfull);
    uint64_t* tempty = reinterpret_cast<uint64_t*>(smem + L::tempty);
    uint64_t* drain = reinterpret_cast<uint64_t*>(smem + L::drain);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::misc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::misc + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1 + kEpiWarps);   // the MMA commit + one arrival per epilogue warp
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], kEpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
    }
    if (warp == 1) tmem_alloc(tmem_holder, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait_then_release();
    if (p.clear && blockIdx.x == 0 && threadIdx.x == 0) *p.status = MOE_OK;
    const uint32_t tmem_base = *tmem_holder;
    constexpr int MPG = kTileK / 32;

    if (warp < kFirstEpiWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
        if (warp == 0 && lane == 0) {
            // -------------------------------------------------------------- TMA producer
            uint32_t it = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < total_units && ok; u += gridDim.x) {
                const int nb = u / mt, mb = u - nb * mt;
                const int row0 = mb * kTileM, brow0 = nb * kTileN;
                const float* ws_src = static_cast<const float*>(p.w_scale) + brow0;
                const float* sa_src = static_cast<const float*>(p.a_scale) + row0;
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    const int s = it % kStages;
                    if (!mbar_wait<kProducerSleepNs>(&empty[s], ((it / kStages) & 1) ^ 1, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[s], kABytes + kBBytes + kWsBytes + kSaBytes);
                    tma_load_2d(smem + L::a + s * kABytes, &tmA, kb * kTileK, row0, &full[s]);
                    tma_load_2d(smem + L::b + s * kBBytes, &tmB, kb * kTileK, brow0, &full[s]);
                    bulk_load(smem + L::sc + s * kScaleSlot, ws_src + static_cast<size_t>(kb) * n_pad, kWsBytes, &full[s]);
                    bulk_load(smem + L::sc + s * kScaleSlot + kWsBytes, sa_src + static_cast<size_t>(kb) * p.a_pad,
                              kSaBytes, &full[s]);
                }
            }
            if (!ok) {   // let the copies already issued land before the CTA leaves
                const uint32_t n = it < static_cast<uint32_t>(kStages) ? it : kStages;
                for (uint32_t i = it - n; i < it; ++i) drain_wait(&full[i % kStages], (i / kStages) & 1);
            }
        } else if (warp == 1 && lane == 0) {
            // -------------------------------------------------------------- MMA issuer
            const uint32_t idesc = f8_idesc(kTileM, kTileN);
            const uint64_t a_desc0 = sw128_kmajor_desc(smem_u32(smem + L::a));
            const uint64_t b_desc0 = sw128_kmajor_desc(smem_u32(smem + L::b));
            uint32_t s = 0, ph = 0, buf = 0, bph = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < total_units && ok; u += gridDim.x) {
                for (int kb = 0; kb < KB; ++kb) {
                    if (!mbar_wait<kIssuerSleepNs>(&full[s], ph, abort_flag, p.status) ||
                        !mbar_wait<kIssuerSleepNs>(&tempty[buf], bph ^ 1, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = a_desc0 + s * (kABytes >> 4), bd = b_desc0 + s * (kBBytes >> 4);
                    const uint32_t d = tmem_base + buf * static_cast<uint32_t>(kTileN);
#pragma unroll
                    for (int m = 0; m < MPG; ++m) mma_f8(d, ad + 2 * m, bd + 2 * m, idesc, m > 0 ? 1u : 0u);
                    mma_commit(&tfull[buf]);
                    mma_commit(&empty[s]);
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                    buf ^= 1;
                    bph ^= buf ^ 1;
                }
            }
            mma_commit(drain);
            drain_wait(drain, 0);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
        // ------------------------------------------------------------------ epilogue
        const int quad = warp & 3;                 // TMEM lanes 32*quad .. 32*quad+31
        const int qtr = (warp - kFirstEpiWarp) >> 2;
        const int row_in_tile = quad * 32 + lane;
        const uint32_t t_warp = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(32 * qtr);
        const uint32_t ws0 = smem_u32(smem + L::sc) + static_cast<uint32_t>(32 * qtr * 4);
        const uint32_t sa0 = smem_u32(smem + L::sc + kWsBytes) + static_cast<uint32_t>(row_in_tile * 4);
        const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
        const uint32_t tfull0 = smem_u32(tfull), tempty0 = smem_u32(tempty);
        const uint32_t abort_at = smem_u32(smem + L::misc + 4);
        uint32_t s = 0, ph = 0, buf = 0, bph = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < total_units && ok; u += gridDim.x) {
            float2 acc2[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) acc2[i] = make_float2(0.0f, 0.0f);
            float* acc = reinterpret_cast<float*>(acc2);
            for (int kb = 0; kb < KB; ++kb) {
                if (!mbar_wait_at(full0 + 8 * s, ph, abort_at, p.status) ||
                    !mbar_wait_at(tfull0 + 8 * buf, bph, abort_at, p.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t so = s * kScaleSlot;
                const float sa = ld_shared_f32(sa0 + so);
                const float2 sa2 = make_float2(sa, sa);
                const uint32_t ws = ws0 + so;
                const uint32_t taddr = t_warp + buf * static_cast<uint32_t>(kTileN);
                uint32_t va[16], vb[16];
                MOE_TMEM_LD16(taddr, va);
                MOE_TMEM_WAIT_LD16(va);
                MOE_TMEM_LD16(taddr + 16, vb);
                promote16(acc2, va, ws, 0, sa2);
                MOE_TMEM_WAIT_LD16(vb);
                MOE_TMEM_LD16(taddr + kHalf, va);
                promote16(acc2, vb, ws + 64, 16, sa2);
                MOE_TMEM_WAIT_LD16(va);
                MOE_TMEM_LD16(taddr + kHalf + 16, vb);
                promote16(acc2, va, ws + 4 * kHalf, 32, sa2);
                MOE_TMEM_WAIT_LD16(vb);
                tc_fence_before();
                mbar_arrive_lane0(tempty0 + 8 * buf, lane);
                promote16(acc2, vb, ws + 4 * kHalf + 64, 48, sa2);
                // the scales were read through the generic proxy; the next bulk copy into this
                // stage is an async-proxy write: order the reads before it
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive_lane0(empty0 + 8 * s, lane);
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1;
                }
                buf ^= 1;
                bph ^= buf ^ 1;
            }
            if (!ok) break;
            const int nb = u / mt, mb = u - nb * mt;
            const int t = mb * kTileM + row_in_tile;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c0 = nb * kTileN + h * kHalf + qtr * 32;
                if (c0 >= p.N) continue;
                if (p.N % 8 == 0) {
                    if (t < p.T) linear_store32(p, acc + 32 * h, t, c0);
                } else {
                    float* stage = reinterpret_cast<float*>(smem + L::stage) + (warp - kFirstEpiWarp) * 32 * (kStageCols + 1);
#pragma unroll
                    for (int c = 0; c < 32; c += kStageCols)
                        linear_store_any<kStageCols>(p, stage, acc + 32 * h + c, mb * kTileM + quad * 32, c0 + c);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

cudaError_t launch_linear_fp32(const LinearArgs& a, const CUtensorMap& tmX, const CUtensorMap& tmW, int num_sms,
                               cudaStream_t s) {
    // The register split above must fit what the block is launched with, or setmaxnreg.inc would
    // wait forever: refuse to launch otherwise.
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, k_linear_fp32);
    if (e != cudaSuccess) return e;
    if (fa.numRegs * kThreads < kRegsLow * 128 + kRegsHigh * 512) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(k_linear_fp32, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
    if (e != cudaSuccess) return e;
    return launch_pdl(k_linear_fp32, dim3(num_sms), dim3(kThreads), kSmemBytes, s, tmX, tmW, a);
}

// The narrow kernel takes a product when its estimated time is below the wide kernel's: both are
// (rounds of CTAs over the SMs) x (K groups of a CTA) x (time of a group).
bool linear_is_narrow(int T, int N, int K, int recipe, int num_sms) {
    const long long KB = K / kTileK;
    const int nt = linear_narrow_tokens(T), split = linear_narrow_split(T, N, K, num_sms);
    const long long tiles = static_cast<long long>((N + kTileM - 1) / kTileM) * ((T + nt - 1) / nt);
    if ((T + nt - 1) / nt > 65535) return false;       // grid.z
    const int wn = recipe == 0 ? kTileN : 128;
    const long long units = static_cast<long long>((N + wn - 1) / wn) * ((T + kTileM - 1) / kTileM);
    const long long narrow = (tiles * split + num_sms - 1) / num_sms * ((KB + split - 1) / split) * 700;
    const long long wide = (units + num_sms - 1) / num_sms * KB * (recipe == 0 ? 1550 : 700);
    return narrow < wide;
}

uint32_t linear_token_box(const LinearArgs& a, int num_sms) {
    return linear_is_narrow(a.T, a.N, a.K, a.recipe, num_sms) ? linear_narrow_tokens(a.T) : kTileM;
}
uint32_t linear_weight_box(const LinearArgs& a, int num_sms) {
    return a.recipe != 0 || linear_is_narrow(a.T, a.N, a.K, a.recipe, num_sms) ? 128 : kTileN;
}

cudaError_t launch_linear(const LinearArgs& a, const CUtensorMap& tmX, const CUtensorMap& tmW, int num_sms,
                          cudaStream_t s) {
    if (linear_is_narrow(a.T, a.N, a.K, a.recipe, num_sms)) return launch_linear_narrow(a, tmX, tmW, num_sms, s);
    return a.recipe == 0 ? launch_linear_fp32(a, tmX, tmW, num_sms, s) : launch_linear_mx(a, tmX, tmW, num_sms, s);
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
