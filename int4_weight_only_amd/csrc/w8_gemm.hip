// W8A8 products: e4m3 codes with block scales, fp32 accumulation, bf16 out.
//
//   Y[m, n] = bf16( sum_k X8[m, k] 2^SX[m, k/128] W8[n, k] 2^SW[n/128, k/128] )
//
// dense (w8a8_gemm) and grouped over aligned expert blocks (w8a8_moe_gemm).
#include "w8.h"

namespace w4 {

namespace {

// Where a tile's activation rows come from and its output rows go.
struct Grouped {
  const int32_t* sorted_ids;
  const int32_t* expert_ids;
  const int32_t* ntpp;
  int P, E, B, div;     // pairs T k, experts, rows per aligned block, pairs per X row
};

}  // namespace

// ----------------------------------------------------------- split-K tile --
// A workgroup of NW waves computes 16 MT rows of X times 16 NT rows of W.
// The waves split the K blocks between them (wave w takes a contiguous run),
// each reads its operands from memory straight into the MFMA registers (no
// LDS: nothing is shared between waves but the final sum), and the partial
// sums are joined through LDS in wave order, so a result does not depend on
// timing.  Lane (r = l % 16, h = l / 16) reads the 16-byte pieces h and
// 4 + h of its row's 128: a load instruction covers 16 rows x 64 bytes, two
// complete each row's 128-byte line.  Rows past the end repeat the last one
// and are not stored; pieces past K are zero.
template <int MT, int NT, int NW, bool GROUPED>
__global__ __launch_bounds__(NW * 64) void k_w8_split(const uint8_t* __restrict__ X8,
                                                      const uint8_t* __restrict__ SX,
                                                      const uint8_t* __restrict__ W8,
                                                      const uint8_t* __restrict__ SW,
                                                      uint16_t* __restrict__ Y, int64_t M,
                                                      int64_t N, int K, int ntiles, Grouped gr) {
  constexpr int BM = 16 * MT, BN = 16 * NT;
  __shared__ __attribute__((aligned(16))) f32x4 part[NW][MT * NT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, h = lane >> 4;
  const int64_t slot = blockIdx.x / ntiles;
  const int64_t n0 = (int64_t)(blockIdx.x % ntiles) * BN;
  const int nb = (K + 127) / 128;
  const int64_t cols = w8_cols(K);

  if constexpr (GROUPED) {
    const int64_t first = slot * BM;
    if (first >= gr.ntpp[0]) return;
    const int e = gr.expert_ids[first / gr.B];
    if (e < 0 || e >= gr.E || (uint32_t)gr.sorted_ids[first] >= (uint32_t)gr.P) return;
    W8 += (int64_t)e * N * K;
    SW += (int64_t)e * w8_blocks(N) * cols;
  }
  // row of X / Y that tile row 16 i + r16 stands for; out of range: -1
  int64_t yrow[MT];
  const uint8_t* xp[MT];
  const uint8_t* sxp[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    int64_t x;
    if constexpr (GROUPED) {
      const int f = gr.sorted_ids[slot * BM + 16 * i + r16];
      const bool ok = (uint32_t)f < (uint32_t)gr.P;
      yrow[i] = ok ? f : -1;
      x = ok ? f / gr.div : 0;
    } else {
      const int64_t m = slot * BM + 16 * i + r16;
      yrow[i] = m < M ? m : -1;
      x = m < M ? m : M - 1;
    }
    xp[i] = X8 + x * K + 16 * h;
    sxp[i] = SX + x * cols;
  }
  const uint8_t* wp[NT];
  const uint8_t* swp[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t n = min(n0 + 16 * j + r16, N - 1);
    wp[j] = W8 + n * K + 16 * h;
    swp[j] = SW + (n >> 7) * cols;
  }

  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int per = (nb + NW - 1) / NW;
  const int b_lo = min(nb, wave * per), b_hi = min(nb, b_lo + per);
  const int full = K / 128;
  const u32x4 zero = u32x4{0u, 0u, 0u, 0u};
  auto block = [&](int b, bool whole) __attribute__((always_inline)) {
    const int64_t k = (int64_t)b * 128;
    const bool in0 = whole || k + 16 * h < K, in1 = whole || k + 64 + 16 * h < K;
    i32x8 x[MT], w[NT];
    uint32_t sx[MT], sw[NT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      x[i] = join16(in0 ? *(const u32x4*)(xp[i] + k) : zero, in1 ? *(const u32x4*)(xp[i] + k + 64) : zero);
      sx[i] = sxp[i][b];
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      w[j] = join16(in0 ? *(const u32x4*)(wp[j] + k) : zero, in1 ? *(const u32x4*)(wp[j] + k + 64) : zero);
      sw[j] = swp[j][b];
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = mfma8_16(w[j], x[i], acc[i][j], sw[j], sx[i]);
  };
  for (int b = b_lo; b < min(b_hi, full); ++b) block(b, true);
  if (full < b_hi && full >= b_lo) block(full, false);

#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) part[wave][i * NT + j][lane] = acc[i][j];
  __syncthreads();
  // lane holds n = n0 + 16 j + 4 h + 0..3 of row yrow[i]
  const bool vec = (N & 3) == 0 && ((uintptr_t)Y & 7) == 0;
#pragma unroll
  for (int t = 0; t < MT * NT; ++t) {
    if (t % NW != wave) continue;
    f32x4 s = part[0][t][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) s += part[w][t][lane];
    const int i = t / NT, j = t % NT;
    int64_t row = -1;
#pragma unroll
    for (int q = 0; q < MT; ++q) row = q == i ? yrow[q] : row;
    const int64_t n = n0 + 16 * j + 4 * h;
    if (row < 0 || n >= N) continue;
    uint16_t* y = Y + row * N + n;
    const u32x2 o = {pk_bf16(s.x, s.y), pk_bf16(s.z, s.w)};
    if (vec) {
      *(u32x2*)y = o;
    } else {
      y[0] = (uint16_t)o.x;
      if (n + 1 < N) y[1] = (uint16_t)(o.x >> 16);
      if (n + 2 < N) y[2] = (uint16_t)o.y;
      if (n + 3 < N) y[3] = (uint16_t)(o.y >> 16);
    }
  }
}

namespace {

template <int MT, int NT, int NW, bool GROUPED>
hipError_t split(const uint8_t* X8, const uint8_t* SX, const uint8_t* W8, const uint8_t* SW,
                 uint16_t* Y, int64_t M, int64_t N, int64_t K, int64_t slots, const Grouped& gr,
                 hipStream_t st) {
  const int64_t ntiles = (N + 16 * NT - 1) / (16 * NT);
  hipLaunchKernelGGL((k_w8_split<MT, NT, NW, GROUPED>), dim3((unsigned)(ntiles * slots)),
                     dim3(NW * 64), 0, st, X8, SX, W8, SW, Y, M, N, (int)K, (int)ntiles, gr);
  return hipGetLastError();
}

}  // namespace

int64_t w8_gemm_threads(int64_t M, int64_t N, int64_t K) {
  return ((M + 63) / 64) * ((N + 31) / 32) * 512;
}

hipError_t launch_w8_gemm(const uint8_t* X8, const uint8_t* SX, const uint8_t* W8,
                          const uint8_t* SW, uint16_t* Y, int64_t M, int64_t N, int64_t K,
                          hipStream_t st) {
  const Grouped none = {};
  if (M <= 16) return split<1, 2, 8, false>(X8, SX, W8, SW, Y, M, N, K, 1, none, st);
  if (M <= 32) return split<2, 2, 8, false>(X8, SX, W8, SW, Y, M, N, K, 1, none, st);
  return split<4, 2, 8, false>(X8, SX, W8, SW, Y, M, N, K, (M + 63) / 64, none, st);
}

int64_t w8_moe_threads(int64_t T, int32_t k, int32_t E, int64_t N, int64_t K, int32_t B) {
  return (T * k + (int64_t)E * (B - 1) + 15) / 16 * ((N + 31) / 32) * 256;
}

hipError_t launch_w8_moe_gemm(const uint8_t* X8, const uint8_t* SX, const uint8_t* W8,
                              const uint8_t* SW, const int32_t* sorted_ids,
                              const int32_t* expert_ids, const int32_t* ntpp, uint16_t* Y,
                              int64_t T, int32_t k, int32_t E, int64_t N, int64_t K, int32_t B,
                              int32_t x_row_div, hipStream_t st) {
  const Grouped gr = {sorted_ids, expert_ids, ntpp, (int)(T * k), E, B, x_row_div};
  const int64_t cap = (T * k + (int64_t)E * (B - 1) + B - 1) / B * B;
  if (B % 64 == 0)
    return split<4, 2, 4, true>(X8, SX, W8, SW, Y, 0, N, K, cap / 64, gr, st);
  if (B % 32 == 0)
    return split<2, 2, 4, true>(X8, SX, W8, SW, Y, 0, N, K, cap / 32, gr, st);
  return split<1, 2, 4, true>(X8, SX, W8, SW, Y, 0, N, K, cap / 16, gr, st);
}

}  // namespace w4
