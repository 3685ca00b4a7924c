// Internal declarations of the bf16 products of training (grouped by expert,
// and with the tokens as the summed dimension) and of the SwiGLU gradient.
#pragma once

#include "w8.h"

namespace w4 {

// A checkpoint operand: e4m3 codes [R, K] with the scales of w8_quantize_rows;
// its values are bf16(code * 2^(scale - 127)), exact unless below bf16's normal range.
struct Bf16Rows {
  const void* p;          // bf16 rows, or codes where scales is given
  const uint8_t* scales;
};

// The aligned pairs of moe_align_block_size (P pairs, E experts, blocks of B).
struct Bf16Plan {
  const int32_t* sorted_ids;
  const int32_t* expert_ids;
  const int32_t* ntpp;
  int64_t P;
  int32_t E, B;
};

// threads of the largest launch (for the launch limit)
int64_t bf16_moe_threads(int64_t P, int32_t E, int64_t N, int64_t K, int32_t B);
int64_t bf16_wgrad_threads(int32_t E, int64_t N, int64_t K);
// fp32 values of the partial sums that a call with a workspace is split into (0: not)
int64_t bf16_moe_workspace(int64_t P, int32_t E, int64_t N, int64_t K, int32_t B);
int64_t bf16_sums_workspace(int64_t groups, int64_t sum, int64_t N, int64_t K);
// results of a workgroup, rows << 16 | columns, of a call with its workspace
int32_t bf16_moe_tile(int64_t P, int32_t E, int64_t N, int64_t K, int32_t B);
int32_t bf16_sums_tile(int64_t groups, int64_t sum, int64_t N, int64_t K);
// Y[f] = X[f / div] W_e^T (W [E, N, K]) or, transposed, X[f / div] W_e (W [E, K, N])
hipError_t launch_bf16_moe_gemm(const uint16_t* X, const uint16_t* W, uint16_t* Y,
                                const Bf16Plan& plan, int64_t N, int64_t K, int32_t div,
                                bool transposed, float* workspace, hipStream_t st);
// dW[e] = sum over e's pairs of dY[f / dy_div]^T X[f / x_div]
hipError_t launch_bf16_moe_wgrad(const uint16_t* dY, const Bf16Rows& X, uint16_t* dW,
                                 const Bf16Plan& plan, int64_t N, int64_t K, int32_t dy_div,
                                 int32_t x_div, float* workspace, hipStream_t st);
// C [N, K] = A [M, N]^T B [M, K]
hipError_t launch_bf16_gemm_tn(const uint16_t* A, const Bf16Rows& B, uint16_t* C, int64_t M,
                               int64_t N, int64_t K, float* workspace, hipStream_t st);
hipError_t launch_silu_mul_bwd(const Bf16Rows& H1, const uint16_t* dA, const float* weights,
                               int64_t R, int64_t I, uint16_t* dH1, uint16_t* A, float* dw,
                               hipStream_t st);
}  // namespace w4
