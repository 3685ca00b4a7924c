// Gradient of the SwiGLU between the expert projections, with the top-k weight
// of the pair and with the input kept in bf16 or as a checkpoint of e4m3 codes.
//
// With h = (g, u), s = sigmoid(g), a = g s u, G the gradient of the down
// projection's input before the weight w is applied (out = sum_j w_j W a_j):
//   dg = w G u s (1 + g (1 - s)),   du = w G g s,   A = w a,   dw = sum_i G_i a_i
// so the backward needs neither the down product's output (dw = <dout, W a> = <W^T
// dout, a>) nor a stored a.
#include "bf16.h"

namespace w4 {

namespace {

struct Point {
  float dg, du, a, wa;     // a without the weight, and with it
};

// One element; G without the weight w.  The exponential is that of silu_mul_fast.  u is
// halved on the way to dg, since s (1 + g (1 - s)) reaches 1.1: with w G and w u below fp32's
// largest value no partial product passes it where the result (for dw: a) does not.
//
// FAR: gates below kFar, whose sigmoid is near fp32's smallest values or below them.  It
// carries 2^136, which the other factors give back piece by piece; dg takes the larger of
// u and w G first, so that neither product passes the range before the result does.  Gates
// below -181 give zeros (u and w G would have to be above 2^64 both for more).
constexpr float kFar = -83.0f;

template <bool FAR>
__device__ __forceinline__ Point swiglu_point(float g, float u, float G, float w) {
  constexpr float kLog2e = 1.44269502f, kRest = 1.92596299e-8f, kLn2 = 0.693147182f;
  const float c = __builtin_amdgcn_fmed3f(g, -1024.0f, 1024.0f);
  const float t = -c * kLog2e;
  const float r = __builtin_fmaf(-c, kLog2e, -t) - c * kRest;
  const float e = __builtin_amdgcn_exp2f(FAR ? t - 136.0f : t) * __builtin_fmaf(r, kLn2, 1.0f);
  const float q = __builtin_amdgcn_rcpf(e + (FAR ? 0x1p-136f : 1.0f));   // the sigmoid, or 2^136 times it
  const float gs = g * q, Gw = w * G;
  if constexpr (FAR) {                             // 1 - s is 1
    const bool more = __builtin_fabsf(u) > __builtin_fabsf(Gw);
    const float big = more ? u : Gw, small = more ? Gw : u;
    const float us = u * 0x1p-34f;
    return {q * (g + 1.0f) * (big * 0x1p-34f) * 0x1p-51f * (small * 0x1p-51f), Gw * 0x1p-51f * gs * 0x1p-85f,
            us * gs * 0x1p-102f, w * us * gs * 0x1p-102f};
  } else {
    // 1 - s = e^-g / (1 + e^-g): no cancellation for large g
    const float part = q * __builtin_fmaf(g, e * q, 1.0f);
    return {0.5f * u * part * Gw * 2.0f, Gw * gs, u * gs, w * u * gs};
  }
}

template <bool C8>
__device__ __forceinline__ void load8(const Bf16Rows& o, int64_t row, int64_t cols, int64_t c, float* v) {
  if constexpr (!C8) {
    const u32x4 x = *(const u32x4*)((const uint16_t*)o.p + row * cols + c);
    const uint32_t d[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(d[i]);
      v[2 * i + 1] = bf16_hi(d[i]);
    }
  } else {
    const u32x2 x = *(const u32x2*)((const uint8_t*)o.p + row * cols + c);
    const float s = __uint_as_float((uint32_t)o.scales[row * w8_cols(cols) + (c >> 7)] << 23);
    const uint32_t d[2] = {x.x, x.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = __builtin_bit_cast(
          uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d[i], s, false));
      const uint32_t hi = __builtin_bit_cast(
          uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d[i], s, true));
      v[4 * i] = bf16_lo(lo);
      v[4 * i + 1] = bf16_hi(lo);
      v[4 * i + 2] = bf16_lo(hi);
      v[4 * i + 3] = bf16_hi(hi);
    }
  }
}

template <bool C8>
__device__ __forceinline__ void load4(const Bf16Rows& o, int64_t row, int64_t cols, int64_t c, float* v) {
  uint32_t lo, hi;
  if constexpr (!C8) {
    const u32x2 x = *(const u32x2*)((const uint16_t*)o.p + row * cols + c);
    lo = x.x;
    hi = x.y;
  } else {
    const uint32_t x = *(const uint32_t*)((const uint8_t*)o.p + row * cols + c);
    const float s = __uint_as_float((uint32_t)o.scales[row * w8_cols(cols) + (c >> 7)] << 23);
    lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, s, false));
    hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, s, true));
  }
  v[0] = bf16_lo(lo);
  v[1] = bf16_hi(lo);
  v[2] = bf16_lo(hi);
  v[3] = bf16_hi(hi);
}

__device__ __forceinline__ u32x2 pack4(const float* v) {
  return u32x2{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
}

__device__ __forceinline__ u32x4 pack8(const float* v) {
  return u32x4{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]), pk_bf16(v[4], v[5]), pk_bf16(v[6], v[7])};
}

}  // namespace

// One workgroup per row, eight elements a thread and pass (16-byte loads and stores of
// bf16, 8 of codes); dw's terms meet in a fixed order (a thread's own, its wave's by
// exchange, the waves' in order), in fp32.  An element of I moves 10 bytes from codes, 12
// from bf16 (with A).  Memory bounds rows of about 500 and more: 32775 rows of 2000 take
// 115 us from codes (5.7 TB/s, above the copy rate since a stream that is mostly stores runs
// faster) and 142 from bf16 (5.5), 32768 rows of 768 49 and 60.  Shorter rows leave threads
// without work, and the beginning of a workgroup bounds them: 32768 rows of 256 39 and 36 us,
// of 64 32 and 30.  64 rows of 2048: 4 us, a launch and a row's chain of loads.
// Far gates are computed apart, in fewer registers (scales selected for every element: 125
// us, and 94 registers with both forms side by side); a hundredth of them among the 32775 x
// 2000 gates makes it 162 us, nothing else 174.
template <bool C8>
__global__ __launch_bounds__(256) void k_silu_mul_bwd(Bf16Rows H1, const uint16_t* __restrict__ dA,
                                                      const float* __restrict__ weights, int64_t R,
                                                      int64_t I, uint16_t* __restrict__ dH1,
                                                      uint16_t* __restrict__ A,
                                                      float* __restrict__ dw) {
  __shared__ float part[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t row = blockIdx.x; row < R; row += gridDim.x) {
    const float w = weights ? weights[row] : 1.0f;
    float sum = 0.0f;
    for (int64_t i = 8 * threadIdx.x; i < I; i += 8 * 256) {
      float g[8], u[8], d[8], dg[8], du[8], a[8];
      load8<C8>(H1, row, 2 * I, i, g);
      load8<C8>(H1, row, 2 * I, I + i, u);
      load8<false>({dA, nullptr}, row, I, i, d);
      bool far = false;
#pragma unroll
      for (int q = 0; q < 8; ++q) far |= g[q] < kFar;
      if (far) {                                   // hardly ever: four at a time, for the registers' sake
        int c = (int)i;
        asm volatile("" : "+v"(c));                // addresses formed here, not kept by every pass
#pragma unroll 1
        for (int last = c + 8; c < last; c += 4) {
          load4<C8>(H1, row, 2 * I, c, g);
          load4<C8>(H1, row, 2 * I, I + c, u);
          load4<false>({dA, nullptr}, row, I, c, d);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const Point p = g[q] < kFar ? swiglu_point<true>(g[q], u[q], d[q], w) : swiglu_point<false>(g[q], u[q], d[q], w);
            sum = __builtin_fmaf(d[q], p.a, sum);
            dg[q] = p.dg;
            du[q] = p.du;
            a[q] = p.wa;
          }
          *(u32x2*)(dH1 + row * 2 * I + c) = pack4(dg);
          *(u32x2*)(dH1 + row * 2 * I + I + c) = pack4(du);
          if (A) *(u32x2*)(A + row * I + c) = pack4(a);
        }
        continue;
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const Point p = swiglu_point<false>(g[q], u[q], d[q], w);
        sum = __builtin_fmaf(d[q], p.a, sum);
        dg[q] = p.dg;
        du[q] = p.du;
        a[q] = p.wa;
      }
      *(u32x4*)(dH1 + row * 2 * I + i) = pack8(dg);
      *(u32x4*)(dH1 + row * 2 * I + I + i) = pack8(du);
      if (A) *(u32x4*)(A + row * I + i) = pack8(a);
    }
    if (dw) {
#pragma unroll
      for (int x = 32; x > 0; x >>= 1) sum += __shfl_xor(sum, x);
      __syncthreads();
      if (lane == 0) part[wave] = sum;
      __syncthreads();
      if (threadIdx.x == 0) dw[row] = part[0] + part[1] + part[2] + part[3];
    }
  }
}

hipError_t launch_silu_mul_bwd(const Bf16Rows& H1, const uint16_t* dA, const float* weights,
                               int64_t R, int64_t I, uint16_t* dH1, uint16_t* A, float* dw,
                               hipStream_t st) {
  const dim3 g((unsigned)(R < (1 << 23) ? R : (1 << 23))), b(256);
  if (H1.scales)
    hipLaunchKernelGGL(k_silu_mul_bwd<true>, g, b, 0, st, H1, dA, weights, R, I, dH1, A, dw);
  else
    hipLaunchKernelGGL(k_silu_mul_bwd<false>, g, b, 0, st, H1, dA, weights, R, I, dH1, A, dw);
  return hipGetLastError();
}

}  // namespace w4
