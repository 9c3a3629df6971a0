// block_kernels.h -- host-side launchers of the kernels around the layer (internal header): the
// residual RMS norm, the dense FP8 product, the balance loss and the router's gradients.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

struct NormArgs {
    const __nv_bfloat16* x;     // [T, H]
    const void* res;            // [T, H] bf16 or fp32, or null
    const float* w;             // [H]
    void* res_out;              // as res, or null
    __nv_bfloat16* y;           // [T, H] or null
    uint8_t* xq;                // [T, H] or null
    uint32_t* xs;               // [H/128][a_pad] words
    int T, H, recipe, a_pad, res_fp32;
    float eps;
    int tpr;                    // threads per row (set by the launcher)
};

struct QuantRowsArgs {
    const __nv_bfloat16* x;     // [T, K]
    uint8_t* xq;                // [T, K]
    uint32_t* xs;               // [K/128][a_pad] words
    int32_t* status;            // cleared to MOE_OK
    int T, K, recipe, a_pad;
};

// Weight transform of one dense product: w [K, N] -> K-major rows, scales re-laid.
struct LinearTransformArgs {
    const uint8_t* w;
    const void* ws;
    uint8_t* w_t;
    void* ws_t;
    int K, N, recipe;
};

struct LinearArgs {
    int T, N, K, recipe, act;
    int a_pad;                  // row stride of the activation scales
    const void* a_scale;        // [K/128][a_pad] words
    const void* w_scale;        // recipe 0: fp32 [K/128][n_pad]; else 512-byte atoms [n_pad/128][K/128]
    const __nv_bfloat16* bias;  // [N] or null
    const __nv_bfloat16* res;   // [T, N] or null
    __nv_bfloat16* y;           // [T, N]
    int32_t* status;
    int clear;                  // the kernel clears the status word (it is the call's first)
    int fault;                  // MOE_FAULT_* (acted on only in a MOE_FAULT_INJECTION build)
};

// Output columns are padded to this in the transformed scales.
constexpr int kLinearPad = 256;
inline int linear_n_pad(int N) { return (N + kLinearPad - 1) / kLinearPad * kLinearPad; }

cudaError_t launch_add_rms_norm(NormArgs a, cudaStream_t s);
cudaError_t launch_quant_rows(const QuantRowsArgs& a, cudaStream_t s);
cudaError_t launch_linear_transform(const LinearTransformArgs& a, cudaStream_t s);
// The tensor maps of a product: x codes [T, K], w codes [N, K], the weights' scale atoms as 32-bit words
// [n_pad/128, K/128, 128] (the block-scaled pair kernel), y [T, N] (the pair kernels, N a multiple of 8).
struct LinearMaps {
    CUtensorMap x, w, sf, y;
};

// Which kernel takes a product: the narrow one (few tokens, K split over a cluster) or a pair kernel.
bool linear_is_narrow(int T, int N, int K, int recipe, int num_sms);
int linear_narrow_tokens(int T);
int linear_narrow_split(int T, int N, int K, int num_sms);
// Rows of the tensor maps' boxes, and columns of y's.
struct LinearBoxes {
    uint32_t x, w, y;
    bool pair;                  // the pair kernels' maps are needed too
};
int linear_mx_cols(const LinearArgs& a, int num_sms);   // columns of a block-scaled pair kernel's tile
LinearBoxes linear_boxes(const LinearArgs& a, int num_sms);
cudaError_t launch_linear(const LinearArgs& a, const LinearMaps& m, int num_sms, cudaStream_t s);
cudaError_t launch_linear_narrow(const LinearArgs& a, const LinearMaps& m, int num_sms, cudaStream_t s);
cudaError_t launch_linear_fp32(const LinearArgs& a, const LinearMaps& m, int num_sms, cudaStream_t s);
cudaError_t launch_linear_mx(const LinearArgs& a, const LinearMaps& m, int num_sms, cudaStream_t s);

// The balance loss takes the tokens in chunks, and a block the part of chunk c that is in sequence s, whose sums
// are slot c + s: walking the tokens in order raises c or s at every step, so no two parts share a slot.  As
// many slots as SMs (a block of 1024 threads each) while the sequences leave at least half of them to chunks.
inline int balance_chunk(int T, int S) {
    const int n = S <= 74 ? 149 - S : 75, c = (T + n - 1) / n;
    return c < 32 ? 32 : c;
}
inline int balance_slots(int T, int S) { return (T + balance_chunk(T, S) - 1) / balance_chunk(T, S) + S - 1; }
// No fewer than balance_slots, and more for more sequences: a workspace for S of them serves a smaller number.
inline int balance_max_slots(int T, int S) { return (T < 148 * 32 ? (T + 31) / 32 : 148) + S; }
// A slot's row of sums: its experts in groups of four.
inline __host__ __device__ int balance_row(int E) { return (E + 3) & ~3; }
// The gradients' chunks: a block of 8 warps each, as many as run at once (up to 64 experts four blocks an SM
// at 64 registers a thread, above two at 120).
inline int backward_chunk(int T, int E) {
    const int blocks = E <= 64 ? 592 : 296, c = (T + blocks - 1) / blocks;
    return c < 16 ? 16 : c;
}
inline int backward_chunks(int T, int E) { return (T + backward_chunk(T, E) - 1) / backward_chunk(T, E); }

struct BalanceArgs {
    const float* logits;        // [T, E]
    const int32_t* idx;         // [T, K]
    const uint8_t* mask;        // [T] or null: 0 = not counted
    const int32_t* off;         // [S + 1] or null (one sequence of all tokens)
    float* part_p;              // [slots][row] sums of p
    int32_t* part_n;            // [slots][row] counts
    int2* part_t;               // [slots] counted tokens, ids out of range
    float* seq_loss;            // [S]
    int32_t* ticket;
    int32_t* counts;            // [S, E]
    int32_t* tokens;            // [S + 1]
    float* mean;                // [S, E]
    float* loss;                // [1]
    int32_t* status;
    int T, E, K, S, routing, chunk, slots;
    float coef;
};

struct RouteBackwardArgs {
    const float* logits;        // [T, E]
    const int32_t* idx;         // [T, K]
    const float* dw;            // [T, K] or null
    const float* pes;           // [E] or null
    const float* dloss;         // [1] or null (no balance loss)
    const int32_t* counts;      // [S, E]
    const int32_t* tokens;      // [S + 1]
    const uint8_t* mask;
    const int32_t* off;
    float* dl;                  // [T, E]
    float* dpes;                // [E] or null
    float* part;                // [chunks][E] partial sums of dpes
    int T, E, K, S, routing, renorm, chunk, chunks;
    float rsf, coef;
};

cudaError_t launch_balance(const BalanceArgs& a, cudaStream_t s);
cudaError_t launch_route_backward(const RouteBackwardArgs& a, cudaStream_t s);

}  // namespace moe
