// Quantization to e4m3 codes with power-of-two block scales.
//
// Per block (128 consecutive k of a row, or 128 x 128 of a weight):
//   e    = the smallest integer >= -127 with amax <= 448 * 2^e (0 when amax = 0)
//   code = e4m3_rne(x * 2^-e)
// amax of bf16 or fp32 values comes from an integer maximum of their bits
// without the sign, which also ranks Inf and NaN on top: such a block gets
// the NaN scale and NaN codes.  x * 2^-e is exact and at most 448, so the only
// rounding is that of the conversion.
#include "w8.h"

namespace w4 {

namespace {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(
      uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, false);
}

// maximum over each row of 16 lanes, in every lane of the row
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = max(v, dpp<0xB1>(v));    // quad_perm [1, 0, 3, 2]
  v = max(v, dpp<0x4E>(v));    // quad_perm [2, 3, 0, 1]
  v = max(v, dpp<0x141>(v));   // row_half_mirror
  return max(v, dpp<0x140>(v));   // row_mirror
}

// Largest |x| of eight bf16, as bits of that bf16.
__device__ __forceinline__ uint32_t amax8(u32x4 v) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  const uint32_t a = pk_max_u16(pk_max_u16(v.x & kAbs, v.y & kAbs), pk_max_u16(v.z & kAbs, v.w & kAbs));
  return max(a & 0xFFFFu, a >> 16);
}

__device__ __forceinline__ u32x2 codes8(u32x4 v, uint32_t byte) {
  const float inv = inv_scale(byte);
  u32x2 r = {codes4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y), inv),
             codes4(bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w), inv)};
  return byte == 255u ? u32x2{0x7F7F7F7Fu, 0x7F7F7F7Fu} : r;
}

// workgroups for `units` waves: one round, or a stride where the launch would
// pass 2^32 threads
unsigned row_grid(int64_t units) {
  const int64_t g = (units + 3) / 4;
  return (unsigned)(g < (1 << 23) ? g : (1 << 23));
}

}  // namespace

// ------------------------------------------------------------------- rows --
// One wave per 512 elements of a row (four blocks, one dword of scales): 16
// lanes hold a block, eight elements each, so that a block's maximum is four
// lane exchanges and each lane reads 16 bytes and writes 8.  Bound by bytes, and
// by the launch where they are few: 2050 x 5120 (32 MB) 8 us, 32 x 4096 2.5 us.
__global__ __launch_bounds__(256) void k_w8_quantize_rows(const uint16_t* __restrict__ X,
                                                          int64_t units, int quads, int64_t K,
                                                          uint8_t* __restrict__ X8,
                                                          uint8_t* __restrict__ SX) {
  const int lane = threadIdx.x & 63;
  for (int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); unit < units;
       unit += (int64_t)gridDim.x * 4) {
    const int64_t m = unit / quads;
    const int64_t k = (unit - m * quads) * 512 + 8 * lane;
    u32x4 v = u32x4{0u, 0u, 0u, 0u};
    if (k < K) v = *(const u32x4*)(X + m * K + k);
    const uint32_t byte = scale_byte(row16_max(amax8(v)) << 16);
    if (k < K) *(u32x2*)(X8 + m * K + k) = codes8(v, byte);
    if ((lane & 15) == 0) SX[unit * 4 + (lane >> 4)] = (uint8_t)byte;   // past K: zeros, 127
  }
}

hipError_t launch_w8_quantize_rows(const uint16_t* X, int64_t M, int64_t K, uint8_t* X8,
                                   uint8_t* SX, hipStream_t st) {
  const int64_t quads = w8_cols(K) / 4, units = M * quads;
  hipLaunchKernelGGL(k_w8_quantize_rows, dim3(row_grid(units)), dim3(256), 0, st, X,
                     units, (int)quads, K, X8, SX);
  return hipGetLastError();
}

// ----------------------------------------------------------------- blocks --
// One workgroup per 128 x 128 block: thread t holds eight elements of rows
// t / 16 + 16 i, i = 0..7.  TR also writes the transposed codes through LDS.
// The grid covers whole dwords of scales in both directions; workgroups past
// the blocks write padding (1.0).  The block stays in registers between its
// maximum and its codes: W is read once.  Bound by bytes: 14336 x 4096 with the
// transpose, 235 MB, 45 us (5.2 TB/s; 52 with the call and cold caches).
template <bool TR>
__global__ __launch_bounds__(256) void k_w8_quantize_blocks(const uint16_t* __restrict__ W,
                                                            int64_t N, int64_t K,
                                                            uint8_t* __restrict__ W8,
                                                            uint8_t* __restrict__ SW,
                                                            uint8_t* __restrict__ WT8,
                                                            uint8_t* __restrict__ ST, int gx) {
  constexpr int PAD = 16;
  __shared__ uint32_t wmax[4];
  __shared__ __attribute__((aligned(16))) uint8_t tile[TR ? 128 : 1][128 + PAD];
  const int tid = threadIdx.x;
  const int64_t bk = blockIdx.x % gx, bn = blockIdx.x / gx;
  const int64_t nb = w8_blocks(N), kb = w8_blocks(K), sk = w8_cols(K), sn = w8_cols(N);
  const int64_t n0 = bn * 128, k0 = bk * 128 + 8 * (tid % 16);
  u32x4 v[8];
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = n0 + tid / 16 + 16 * i;
    v[i] = (n < N && k0 < K) ? *(const u32x4*)(W + n * K + k0) : u32x4{0u, 0u, 0u, 0u};
    a = max(a, amax8(v[i]));
  }
  a = row16_max(a);
  a = max(a, (uint32_t)__shfl_xor((int)a, 16));
  a = max(a, (uint32_t)__shfl_xor((int)a, 32));
  if ((tid & 63) == 0) wmax[tid >> 6] = a;
  __syncthreads();
  a = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
  const uint32_t byte = scale_byte(a << 16);
  if (tid == 0) {
    if (bn < nb && bk < sk) SW[bn * sk + bk] = (uint8_t)byte;
    if constexpr (TR) {
      if (bk < kb && bn < sn) ST[bk * sn + bn] = (uint8_t)byte;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = tid / 16 + 16 * i;
    const u32x2 q = codes8(v[i], byte);
    if (n0 + r < N && k0 < K) *(u32x2*)(W8 + (n0 + r) * K + k0) = q;
    if constexpr (TR) *(u32x2*)&tile[r][8 * (tid % 16)] = q;
  }
  if constexpr (TR) {
    __syncthreads();
    // 16 consecutive n of one k per thread and pass (N % 16 == 0)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = tid / 8 + 32 * i, r0 = 16 * (tid % 8);
      const int64_t k = bk * 128 + c;
      if (k >= K || n0 + r0 >= N) continue;
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) w[j] |= (uint32_t)tile[r0 + 4 * j + b][c] << (8 * b);
      }
      *(u32x4*)(WT8 + k * N + n0 + r0) = u32x4{w[0], w[1], w[2], w[3]};
    }
  }
}

hipError_t launch_w8_quantize_blocks(const uint16_t* W, int64_t N, int64_t K, uint8_t* W8,
                                     uint8_t* SW, uint8_t* WT8, uint8_t* ST, hipStream_t st) {
  const int64_t gx = w8_cols(K);
  const int64_t gy = WT8 ? w8_cols(N) : w8_blocks(N);
  const dim3 g((unsigned)(gx * gy)), b(256);
  if (WT8)
    hipLaunchKernelGGL(k_w8_quantize_blocks<true>, g, b, 0, st, W, N, K, W8, SW, WT8, ST, (int)gx);
  else
    hipLaunchKernelGGL(k_w8_quantize_blocks<false>, g, b, 0, st, W, N, K, W8, SW, nullptr, nullptr,
                       (int)gx);
  return hipGetLastError();
}

// ------------------------------------------------------ SwiGLU + quantize --
// a = silu(g) * u in fp32, quantized per 128 elements of the row; one wave
// per 512 outputs, as in the row quantizer.  Bound by bytes: 32775 x 2000,
// 329 MB, 59 us (5.5 TB/s); 2048 x 2048 6 us.
__global__ __launch_bounds__(256) void k_w8_silu_mul_quantize(const uint16_t* __restrict__ H1,
                                                              int64_t units, int quads, int64_t I,
                                                              uint8_t* __restrict__ A8,
                                                              uint8_t* __restrict__ SA) {
  const int lane = threadIdx.x & 63;
  for (int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); unit < units;
       unit += (int64_t)gridDim.x * 4) {
    const int64_t r = unit / quads;
    const int64_t i = (unit - r * quads) * 512 + 8 * lane;
    float a[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = 0.0f;
    if (i < I) {
      const u32x4 gv = *(const u32x4*)(H1 + r * 2 * I + i);
      const u32x4 uv = *(const u32x4*)(H1 + r * 2 * I + I + i);
      const uint32_t g[4] = {gv.x, gv.y, gv.z, gv.w}, u[4] = {uv.x, uv.y, uv.z, uv.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[2 * j] = silu_mul_fast(bf16_lo(g[j]), bf16_lo(u[j]));
        a[2 * j + 1] = silu_mul_fast(bf16_hi(g[j]), bf16_hi(u[j]));
      }
    }
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(a[j]) & 0x7FFFFFFFu);
    const uint32_t byte = scale_byte(row16_max(amax));
    if (i < I) {
      const float inv = inv_scale(byte);
      u32x2 q = {codes4(a[0], a[1], a[2], a[3], inv), codes4(a[4], a[5], a[6], a[7], inv)};
      if (byte == 255u) q = u32x2{0x7F7F7F7Fu, 0x7F7F7F7Fu};
      *(u32x2*)(A8 + r * I + i) = q;
    }
    if ((lane & 15) == 0) SA[unit * 4 + (lane >> 4)] = (uint8_t)byte;
  }
}

hipError_t launch_w8_silu_mul_quantize(const uint16_t* H1, int64_t R, int64_t I, uint8_t* A8,
                                       uint8_t* SA, hipStream_t st) {
  const int64_t quads = w8_cols(I) / 4, units = R * quads;
  hipLaunchKernelGGL(k_w8_silu_mul_quantize, dim3(row_grid(units)), dim3(256), 0, st,
                     H1, units, (int)quads, I, A8, SA);
  return hipGetLastError();
}

}  // namespace w4
