// Internal declarations of the 8-bit floating-point (W8A8) kernels and the
// scored router.
//
// Values: e4m3 codes (OCP, largest 448) with one power-of-two scale per
// block of 128 along K (activations) or 128 x 128 (weights), stored as its
// biased exponent b (e8m0: 2^(b - 127), 255 = NaN).  CDNA4's
// v_mfma_scale_f32_*_f8f6f4 takes such a byte per lane and 32 elements and
// applies it inside the matrix pipe, so the block scales cost no vector
// instruction and the accumulator is the matrix unit's own for the whole K.
#pragma once

#include "common.h"

namespace w4 {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

constexpr int kW8Block = 128;       // elements per scale along K, rows per weight scale
constexpr int kW8MaxK = 1 << 22;    // a tile of 256 rows spans less than 2^31 bytes

// scale bytes of a row: whole dwords, so that the scales of four K blocks
// are one aligned load
__host__ __device__ __forceinline__ int64_t w8_cols(int64_t K) { return (K + 511) / 512 * 4; }
__host__ __device__ __forceinline__ int64_t w8_blocks(int64_t n) { return (n + 127) / 128; }

// D[16x16] += A[16x128] * B[128x16] of e4m3 codes, fp32 accumulation, one
// scale byte per operand row (the low one of sa, sb).  Lane l supplies 32
// bytes of A row (l % 16) and of B column (l % 16); lanes l / 16 = 0..3
// split the 128 elements of the block between them, in any order that A and
// B share (one scale covers the whole block).  It receives
// D[4 (l / 16) + r][l % 16], r = 0..3.
// Precision: the unit cuts each product toward zero to 2^-13 of the largest
// in its group of eight consecutive bytes and adds the groups in fp32
// (measured; the older 16x16x32 fp8 form does the same).  Exact products
// would need the codes widened to bf16, at half the matrix rate and twice
// the operand traffic, to move a result by less than its bf16 rounding.
__device__ __forceinline__ f32x4 mfma8_16(i32x8 a, i32x8 b, f32x4 c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, (int)sa, 0, (int)sb);
}

__device__ __forceinline__ i32x8 join16(u32x4 lo, u32x4 hi) {
  return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w,
               (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// ---------------------------------------------------- quantization, shared --

// Scale byte of a block from the bits of its amax (fp32, sign cleared): with
// amax = m * 2^p, 1 <= m < 2, the exponent is p - 8, or p - 7 when m > 1.75
// (448 = 1.75 * 2^8), at least -127; Inf and NaN (which rank on top): 255.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  if (amax >= 0x7F800000u) return 255u;
  if (amax == 0u) return 127u;
  const int e = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(e, 0);
}

// 2^(127 - byte); the byte of a block is at most 247 (or 255: unused)
__device__ __forceinline__ float inv_scale(uint32_t byte) {
  return __uint_as_float((254u - min(byte, 253u)) << 23);
}

// four values times inv -> four e4m3 codes
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, r, true);
  return (uint32_t)r;
}

// silu(g) * u = g / (1 + e^-g) * u.  The exponential is 2^t with t = -g log2 e
// as a product and its remainder, so that it holds to about three units in the
// last place for every g (beyond the limits it is zero or infinite);
// v_exp_f32 and v_rcp_f32 give one unit each.  (The rounding to e4m3 that
// follows is 2^19 times coarser; with the exactly rounded division and expf the
// quantizer took 78 us at 32775 x 2000, 59 now.)  From t = 120 on the quotient
// and u are taken with 2^136 moved from one to the other: silu(g) itself is then
// below fp32's range, or near its end, while a large u brings the product back
// (t = 262, g = -181, is where the largest u no longer does).
__device__ __forceinline__ float silu_mul_fast(float g, float u) {
  constexpr float kLog2e = 1.44269502f, kRest = 1.92596299e-8f, kLn2 = 0.693147182f;
  const float c = __builtin_amdgcn_fmed3f(g, -1024.0f, 1024.0f);
  const float t = -c * kLog2e;
  const float r = __builtin_fmaf(-c, kLog2e, -t) - c * kRest;
  const bool far = t > 120.0f;
  const float one = far ? 0x1p-136f : 1.0f;
  const float e = __builtin_amdgcn_exp2f(far ? t - 136.0f : t) * __builtin_fmaf(r, kLn2, 1.0f);
  return g * __builtin_amdgcn_rcpf(e + one) * (u * one);
}

hipError_t launch_w8_quantize_rows(const uint16_t* X, int64_t M, int64_t K, uint8_t* X8,
                                   uint8_t* SX, hipStream_t st);
hipError_t launch_w8_quantize_blocks(const uint16_t* W, int64_t N, int64_t K, uint8_t* W8,
                                     uint8_t* SW, uint8_t* WT8, uint8_t* ST, hipStream_t st);
hipError_t launch_w8_silu_mul_quantize(const uint16_t* H1, int64_t R, int64_t I, uint8_t* A8,
                                       uint8_t* SA, hipStream_t st);
// threads the products' largest launch starts (for the launch limit)
int64_t w8_gemm_threads(int64_t M, int64_t N, int64_t K);
hipError_t launch_w8_gemm(const uint8_t* X8, const uint8_t* SX, const uint8_t* W8,
                          const uint8_t* SW, uint16_t* Y, int64_t M, int64_t N, int64_t K,
                          hipStream_t st);
int64_t w8_moe_threads(int64_t T, int32_t k, int32_t E, int64_t N, int64_t K, int32_t B,
                       int32_t x_row_div);
hipError_t launch_w8_moe_gemm(const uint8_t* X8, const uint8_t* SX, const uint8_t* W8,
                              const uint8_t* SW, const int32_t* sorted_ids,
                              const int32_t* expert_ids, const int32_t* ntpp, uint16_t* Y,
                              int64_t T, int32_t k, int32_t E, int64_t N, int64_t K, int32_t B,
                              int32_t x_row_div, hipStream_t st);
// the same for gate and up rows, SwiGLU and quantization in the epilogue; B a
// multiple of 256, I of 128, and X8 below 2 GiB
bool w8_moe_swiglu_fits(int64_t rows_x, int64_t I, int64_t K, int32_t B);
hipError_t launch_w8_moe_gemm_swiglu(const uint8_t* X8, const uint8_t* SX, const uint8_t* W8,
                                     const uint8_t* SW, const int32_t* sorted_ids,
                                     const int32_t* expert_ids, const int32_t* ntpp, uint8_t* A8,
                                     uint8_t* SA, int64_t T, int32_t k, int32_t E, int64_t I,
                                     int64_t K, int32_t B, int32_t x_row_div, hipStream_t st);
// the scored router
struct RouteRule {
  bool sigmoid;                     // scores: sigmoid, or softmax over the row
  int groups, topk_groups, group_top;
  bool renorm;
  float scale;
};
hipError_t launch_route_scored(const float* logits, const float* bias, int64_t T, int32_t E,
                               int32_t k, const RouteRule& r, int32_t* ids, float* w,
                               hipStream_t st);
hipError_t launch_route_scored_bwd(const float* logits, const int32_t* ids, const float* w,
                                   const float* dw, int64_t T, int32_t E, int32_t k,
                                   const RouteRule& r, float* dlogits, hipStream_t st);
}  // namespace w4
