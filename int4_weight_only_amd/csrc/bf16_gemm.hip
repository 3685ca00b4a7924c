// bf16 products of training: grouped by expert over aligned blocks, and with
// the rows (tokens) as the summed dimension.
//
//   rows grouped      Y[f] = X[f / div] W_e^T, or X[f / div] W_e
//   sums grouped      dW[e] = sum over e's pairs f of dY[f / a]^T X[f / b]
//   dense sums        C = A^T B
//
// Bf16 operands, fp32 accumulation in a fixed order, one rounding to bf16.  The
// second operand of a sum may be a checkpoint of e4m3 codes.
#include "bf16.h"

namespace w4 {

namespace {

// Which dimension the expert's pairs are.
enum Group { kDense, kRows, kSums };

struct Job {
  const uint16_t* A;        // [*, K] rows summed along, or (TA) [*, M] with the sum down the rows
  Bf16Rows B;
  uint16_t* C;
  int64_t M, N, K;          // C is M x N (kRows: M slots; a row of C a pair), K the summed dimension
  Bf16Plan g;
  int32_t a_div, b_div;     // pairs per row of A, of B
};

// First of n ascending numbers that is not below e, by 64 probes at a time;
// always within [0, n], whatever the numbers are.
template <typename Below>
__device__ __forceinline__ int first_not(int n, Below below) {
  const int lane = threadIdx.x & 63;
  int lo = 0, len = n;
  while (len > 0) {
    const int step = (len + 63) / 64;
    const int at = lane * step;
    const int below_n = __popcll(__ballot(at < len && below(lo + at)));
    if (below_n == 0) break;
    const int end = min(below_n * step, len);
    lo += (below_n - 1) * step + 1;
    len = end - ((below_n - 1) * step + 1);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// The slots of expert e: [first, first + count).
struct Segment {
  int first, count;
};
__device__ __forceinline__ Segment segment(const Bf16Plan& g, int64_t cap, int e) {
  const int nblk = (int)(min(max((int64_t)g.ntpp[0], (int64_t)0), cap) / g.B);
  const int lo = first_not(nblk, [&](int b) { return g.expert_ids[b] < e; });
  const int hi = first_not(nblk, [&](int b) { return g.expert_ids[b] <= e; });
  if (hi <= lo) return {0, 0};
  const int last = (hi - 1) * g.B;
  const int tail =
      first_not(g.B, [&](int i) { return (uint32_t)g.sorted_ids[last + i] < (uint32_t)g.P; });
  return {lo * g.B, last - lo * g.B + tail};
}

// Eight consecutive values of a row as bf16.
template <bool C8>
__device__ __forceinline__ u32x4 eight(const Bf16Rows& o, int64_t row, int64_t cols, int64_t c) {
  if constexpr (!C8) {
    return *(const u32x4*)((const uint16_t*)o.p + row * cols + c);
  } else {
    const u32x2 q = *(const u32x2*)((const uint8_t*)o.p + row * cols + c);
    const float s = __uint_as_float((uint32_t)o.scales[row * w8_cols(cols) + (c >> 7)] << 23);
    u32x4 r;
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.x, s, false));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.x, s, true));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.y, s, false));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.y, s, true));
    return r;
  }
}

}  // namespace

// ------------------------------------------------------------ simple tile --
// 64 x 64 of C by four waves of 32 x 32, 32 of the summed dimension a step
// through LDS as [row][k], 64-bit addresses throughout.
template <Group G, bool TA, bool TB, bool C8>
__global__ __launch_bounds__(256) void k_bf16_simple(Job j) {
  constexpr int PAD = 8;
  __shared__ __attribute__((aligned(16))) uint16_t as[64][32 + PAD], bs[64][32 + PAD];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r16 = lane & 15, h = lane >> 4;
  const int64_t nt = (j.N + 63) / 64, mt = (j.M + 63) / 64;
  int64_t tile = blockIdx.x, e = 0;
  if constexpr (G == kSums) {
    e = tile / (mt * nt);
    tile -= e * mt * nt;
  }
  const int64_t m0 = tile / nt * 64, n0 = tile % nt * 64;
  Segment seg = {0, 0};
  int64_t steps = (j.K + 31) / 32, cap = 0;
  if constexpr (G != kDense) cap = (j.g.P + (int64_t)j.g.E * (j.g.B - 1) + j.g.B - 1) / j.g.B * j.g.B;
  if constexpr (G == kRows) {
    if (m0 >= min((int64_t)j.g.ntpp[0], cap)) return;
    e = j.g.expert_ids[m0 / j.g.B];
    if (e < 0 || e >= j.g.E) return;
    j.B.p = (const uint16_t*)j.B.p + e * j.N * j.K;
  }
  if constexpr (G == kSums) {
    seg = segment(j.g, cap, (int)e);
    steps = (seg.count + 31) / 32;
    j.C += e * j.M * j.N;
  }
  auto pair = [&](int64_t slot) { return (uint32_t)j.g.sorted_ids[slot]; };
  // row of the operand that summed index k stands for; -1: none
  auto sum_row = [&](int64_t k, int div) -> int64_t {
    if constexpr (G == kSums) {
      if (k >= seg.count) return -1;
      const uint32_t f = pair(seg.first + k);
      return f < (uint32_t)j.g.P ? (int64_t)(f / (uint32_t)div) : -1;
    } else {
      return k < j.K ? k : -1;
    }
  };
  f32x4 acc[2][2] = {};
  const u32x4 zero = {0u, 0u, 0u, 0u};
  for (int64_t s = 0; s < steps; ++s) {
    const int64_t k0 = s * 32;
    __syncthreads();
    if constexpr (!TA) {
      const int r = tid >> 2, c = 8 * (tid & 3);
      int64_t row = m0 + r < j.M ? m0 + r : -1;
      if constexpr (G == kRows) {
        const uint32_t f = pair(m0 + r);
        row = f < (uint32_t)j.g.P ? (int64_t)(f / (uint32_t)j.a_div) : -1;
      }
      *(u32x4*)&as[r][c] = row >= 0 && k0 + c < j.K ? eight<false>({j.A, nullptr}, row, j.K, k0 + c) : zero;
    } else {
      const int k = tid >> 3, c = 8 * (tid & 7);
      const int64_t row = sum_row(k0 + k, j.a_div);
      const u32x4 v = row >= 0 && m0 + c < j.M ? eight<false>({j.A, nullptr}, row, j.M, m0 + c) : zero;
      const uint16_t* q = (const uint16_t*)&v;
      for (int i = 0; i < 8; ++i) as[c + i][k] = q[i];
    }
    if constexpr (!TB) {
      const int r = tid >> 2, c = 8 * (tid & 3);
      *(u32x4*)&bs[r][c] =
          n0 + r < j.N && k0 + c < j.K ? eight<false>(j.B, n0 + r, j.K, k0 + c) : zero;
    } else {
      const int k = tid >> 3, c = 8 * (tid & 7);
      const int64_t row = sum_row(k0 + k, j.b_div);
      const u32x4 v = row >= 0 && n0 + c < j.N ? eight<C8>(j.B, row, j.N, n0 + c) : zero;
      const uint16_t* q = (const uint16_t*)&v;
      for (int i = 0; i < 8; ++i) bs[c + i][k] = q[i];
    }
    __syncthreads();
    u32x4 a[2], b[2];
    for (int i = 0; i < 2; ++i) {
      a[i] = *(const u32x4*)&as[32 * (wave >> 1) + 16 * i + r16][8 * h];
      b[i] = *(const u32x4*)&bs[32 * (wave & 1) + 16 * i + r16][8 * h];
    }
    for (int i = 0; i < 2; ++i)
      for (int n = 0; n < 2; ++n) acc[i][n] = mfma16(b[n], a[i], acc[i][n]);
  }
  // lane holds columns 4 h .. + 3 of row r16 of each 16 x 16
  for (int i = 0; i < 2; ++i) {
    int64_t row = m0 + 32 * (wave >> 1) + 16 * i + r16;
    if constexpr (G == kRows) {
      const uint32_t f = pair(row);
      row = f < (uint32_t)j.g.P ? (int64_t)f : -1;
    } else if (row >= j.M) {
      row = -1;
    }
    if (row < 0) continue;
    for (int n = 0; n < 2; ++n)
      for (int v = 0; v < 4; ++v) {
        const int64_t c = n0 + 32 * (wave & 1) + 16 * n + 4 * h + v;
        if (c < j.N) j.C[row * j.N + c] = to_bf16(acc[i][n][v]);
      }
  }
}

namespace {

int64_t moe_cap(int64_t P, int32_t E, int32_t B) {
  return (P + (int64_t)E * (B - 1) + B - 1) / B * B;
}

template <Group G, bool TA, bool TB, bool C8>
hipError_t run_simple(const Job& j, int64_t tiles, hipStream_t st) {
  hipLaunchKernelGGL((k_bf16_simple<G, TA, TB, C8>), dim3((unsigned)tiles), dim3(256), 0, st, j);
  return hipGetLastError();
}

int64_t simple_tiles(int64_t M, int64_t N) { return ((M + 63) / 64) * ((N + 63) / 64); }

}  // namespace

int64_t bf16_moe_threads(int64_t P, int32_t E, int64_t N, int64_t K, int32_t B) {
  return simple_tiles(moe_cap(P, E, B), N) * 256;
}
int64_t bf16_wgrad_threads(int32_t E, int64_t N, int64_t K) { return E * simple_tiles(N, K) * 256; }

hipError_t launch_bf16_moe_gemm(const uint16_t* X, const uint16_t* W, uint16_t* Y,
                                const Bf16Plan& plan, int64_t N, int64_t K, int32_t div,
                                bool transposed, hipStream_t st) {
  const int64_t cap = moe_cap(plan.P, plan.E, plan.B);
  const Job j = {X, {W, nullptr}, Y, cap, N, K, plan, div, 1};
  if (transposed) return run_simple<kRows, false, true, false>(j, simple_tiles(cap, N), st);
  return run_simple<kRows, false, false, false>(j, simple_tiles(cap, N), st);
}

hipError_t launch_bf16_moe_wgrad(const uint16_t* dY, const Bf16Rows& X, uint16_t* dW,
                                 const Bf16Plan& plan, int64_t N, int64_t K, int32_t dy_div,
                                 int32_t x_div, hipStream_t st) {
  const Job j = {dY, X, dW, N, K, 0, plan, dy_div, x_div};
  const int64_t tiles = plan.E * simple_tiles(N, K);
  if (X.scales) return run_simple<kSums, true, true, true>(j, tiles, st);
  return run_simple<kSums, true, true, false>(j, tiles, st);
}

hipError_t launch_bf16_gemm_tn(const uint16_t* A, const Bf16Rows& B, uint16_t* C, int64_t M,
                               int64_t N, int64_t K, hipStream_t st) {
  const Job j = {A, B, C, N, K, M, {}, 1, 1};
  if (B.scales) return run_simple<kDense, true, true, true>(j, simple_tiles(N, K), st);
  return run_simple<kDense, true, true, false>(j, simple_tiles(N, K), st);
}

}  // namespace w4
