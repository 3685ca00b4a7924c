// The scored router: softmax or sigmoid scores, a bias for the choice, the
// best groups of experts, the k largest in them, weights from the scores;
// and its gradient to the logits.
//
// Scores, choice values, group sums and weights are held in 64 bits: two
// choice values of a row are often closer than 32 bits of an exponential
// tell apart (sixteen thousand rows of 384 hold several such pairs), and a
// swapped expert is another result, not a rounding.  One wave per token.
#include <cfloat>

#include "w8.h"

namespace w4 {

namespace {

template <int CTRL>
__device__ __forceinline__ double dpp64(double a) {
  const uint64_t v = __builtin_bit_cast(uint64_t, a);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)v, CTRL, 0xF, 0xF, false);
  const uint32_t hi =
      (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(v >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// wave-wide reductions over quads, rows of 16 and rows; every lane ends with
// the result, in one fixed order
template <class Op>
__device__ __forceinline__ double wave_all(double a, Op op) {
  a = op(a, dpp64<0xB1>(a));
  a = op(a, dpp64<0x4E>(a));
  a = op(a, dpp64<0x141>(a));
  a = op(a, dpp64<0x140>(a));
  a = op(a, __shfl_xor(a, 16));
  return op(a, __shfl_xor(a, 32));
}
__device__ __forceinline__ double wave_max64(double a) {
  return wave_all(a, [](double x, double y) { return fmax(x, y); });
}
__device__ __forceinline__ double wave_sum64(double a) {
  return wave_all(a, [](double x, double y) { return x + y; });
}

// the logit as the score reads it: +-Inf as the largest numbers, except that
// NaN and -Inf mark a masked expert
__device__ __forceinline__ bool masked(float x) { return !(x > -INFINITY); }
__device__ __forceinline__ double number(float x) { return (double)fminf(x, FLT_MAX); }

// softmax: largest logit and sum of exponentials over the row's experts;
// sigmoid: unused
struct RowSum {
  double top, sum;
};

template <int NPER>
__device__ __forceinline__ RowSum row_sum(const float (&x)[NPER], int E, int lane) {
  double top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NPER; ++i)
    if (lane + 64 * i < E && !masked(x[i])) top = fmax(top, number(x[i]));
  top = wave_max64(top);
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < NPER; ++i)
    if (lane + 64 * i < E && !masked(x[i])) sum += exp(number(x[i]) - top);
  return {top, wave_sum64(sum)};
}

__device__ __forceinline__ double score(float x, bool sigmoid, const RowSum& rs) {
  if (masked(x)) return 0.0;
  return sigmoid ? 1.0 / (1.0 + exp(-number(x))) : exp(number(x) - rs.top) / rs.sum;
}

}  // namespace

// NPER: experts per lane; expert lane + 64 i is the lane's i-th
template <int NPER>
__global__ __launch_bounds__(256) void k_route_scored(const float* __restrict__ logits,
                                                      const float* __restrict__ bias, int T, int E,
                                                      int k, RouteRule rule,
                                                      int32_t* __restrict__ ids,
                                                      float* __restrict__ wts) {
  extern __shared__ double choice[];           // [4 waves][E]: only with groups
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * 4 + wave;
  if (t >= T) return;                          // whole waves; no barrier below
  const float* row = logits + (int64_t)t * E;
  float x[NPER];
#pragma unroll
  for (int i = 0; i < NPER; ++i) x[i] = lane + 64 * i < E ? row[lane + 64 * i] : -INFINITY;
  RowSum rs = {0.0, 1.0};
  if (!rule.sigmoid) rs = row_sum<NPER>(x, E, lane);
  double c[NPER];
  uint32_t live = 0, free = 0;
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const int e = lane + 64 * i;
    c[i] = -INFINITY;
    if (e >= E) continue;
    free |= 1u << i;
    const double v = score(x[i], rule.sigmoid, rs) + (bias ? (double)bias[e] : 0.0);
    if (!masked(x[i]) && v > -INFINITY) {      // a NaN bias masks too
      c[i] = v;
      live |= 1u << i;
    }
  }
  if (rule.groups > 1) {
    // lane g values group g; then its rank among the groups (ties to the
    // lower index) decides whether its experts stay
    double* mine = choice + (int64_t)wave * E;
#pragma unroll
    for (int i = 0; i < NPER; ++i)
      if (lane + 64 * i < E) mine[lane + 64 * i] = c[i];
    __builtin_amdgcn_wave_barrier();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const int per = E / rule.groups;
    double a = -INFINITY, b = -INFINITY;       // the two largest
    if (lane < rule.groups)
      for (int q = 0; q < per; ++q) {
        const double v = mine[lane * per + q];
        b = fmax(b, fmin(a, v));
        a = fmax(a, v);
      }
    const double value = rule.group_top == 2 && b > -INFINITY ? a + b : a;
    int rank = 0;
    for (int g = 0; g < rule.groups; ++g) {
      const double other = __shfl(value, g);
      rank += other > value || (other == value && g < lane);
    }
    const uint64_t keep = __ballot(lane < rule.groups && rank < rule.topk_groups);
#pragma unroll
    for (int i = 0; i < NPER; ++i)
      if (!((keep >> ((lane + 64 * i) / per)) & 1)) live &= ~(1u << i);
  }
  int my_id = 0;
  bool my_live = false;
  for (int j = 0; j < k; ++j) {
    double m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPER; ++i)
      if ((live >> i) & 1u) m = fmax(m, c[i]);
    m = wave_max64(m);
    const bool any = m > -INFINITY;
    int win = -1;
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      // no live expert left: the lowest index that no slot has taken
      const uint64_t b = __ballot(any ? ((live >> i) & 1u) && c[i] == m : (free >> i) & 1u);
      if (win < 0 && b) win = 64 * i + (int)__builtin_ctzll(b);
    }
    if (lane == (win & 63)) {
      live &= ~(1u << (win >> 6));
      free &= ~(1u << (win >> 6));
    }
    if (lane == j) {
      my_id = win;
      my_live = any;
    }
  }
  double s = 0.0;
  if (lane < k && my_live) s = score(row[my_id], rule.sigmoid, rs);
  if (rule.renorm) {
    const double sum = wave_sum64(s);
    s = sum > 0.0 ? s / sum : 0.0;
  }
  if (lane < k) {
    ids[(int64_t)t * k + lane] = my_id;
    wts[(int64_t)t * k + lane] = (float)((double)rule.scale * s);
  }
}

// Gradient: p over the picks (slots whose weight is zero took no part), then
// every expert sums the slots that name it, in slot order.
template <int NPER>
__global__ __launch_bounds__(256) void k_route_scored_bwd(const float* __restrict__ logits,
                                                          const int32_t* __restrict__ ids,
                                                          const float* __restrict__ wts,
                                                          const float* __restrict__ dw, int T,
                                                          int E, int k, RouteRule rule,
                                                          float* __restrict__ dlogits) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  const float* row = logits + (int64_t)t * E;
  const bool dense = !rule.sigmoid && !rule.renorm;   // every score moves every weight
  float x[NPER];
  RowSum rs = {0.0, 1.0};
  if (!rule.sigmoid) {
#pragma unroll
    for (int i = 0; i < NPER; ++i) x[i] = lane + 64 * i < E ? row[lane + 64 * i] : -INFINITY;
    rs = row_sum<NPER>(x, E, lane);
  }
  int id = -1;
  double s = 0.0, g = 0.0, rest = 1.0;
  if (lane < k) {
    const int e = ids[(int64_t)t * k + lane];
    if (e >= 0 && e < E && wts[(int64_t)t * k + lane] != 0.0f) {
      id = e;
      s = score(row[e], rule.sigmoid, rs);
      rest = score(-row[e], true, rs);         // 1 - sigmoid without its cancellation
      g = (double)rule.scale * (double)dw[(int64_t)t * k + lane];
    }
  }
  double d, all = 0.0;
  if (rule.renorm) {
    const double sum = wave_sum64(s);
    const double p = sum > 0.0 ? s / sum : 0.0;
    d = p * (g - wave_sum64(g * p)) * (rule.sigmoid ? rest : 1.0);
  } else if (rule.sigmoid) {
    d = g * s * rest;
  } else {
    d = g * s;
    all = wave_sum64(d);
  }
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const int e = lane + 64 * i;
    double v = dense && e < E ? -score(x[i], false, rs) * all : 0.0;
    for (int j = 0; j < k; ++j) {
      const double dj = __shfl(d, j);
      if (__shfl(id, j) == e) v += dj;
    }
    if (e < E) dlogits[(int64_t)t * E + e] = (float)v;
  }
}

namespace {

template <class F>
void by_experts(int E, F f) {
  if (E <= 64) f(std::integral_constant<int, 1>{});
  else if (E <= 128) f(std::integral_constant<int, 2>{});
  else if (E <= 256) f(std::integral_constant<int, 4>{});
  else if (E <= 384) f(std::integral_constant<int, 6>{});
  else if (E <= 512) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

}  // namespace

hipError_t launch_route_scored(const float* logits, const float* bias, int64_t T, int32_t E,
                               int32_t k, const RouteRule& r, int32_t* ids, float* w,
                               hipStream_t st) {
  const size_t lds = r.groups > 1 ? (size_t)4 * E * sizeof(double) : 0;
  by_experts(E, [&](auto n) {
    hipLaunchKernelGGL(k_route_scored<decltype(n)::value>, dim3((unsigned)((T + 3) / 4)), dim3(256),
                       lds, st, logits, bias, (int)T, (int)E, (int)k, r, ids, w);
  });
  return hipGetLastError();
}

hipError_t launch_route_scored_bwd(const float* logits, const int32_t* ids, const float* w,
                                   const float* dw, int64_t T, int32_t E, int32_t k,
                                   const RouteRule& r, float* dlogits, hipStream_t st) {
  by_experts(E, [&](auto n) {
    hipLaunchKernelGGL(k_route_scored_bwd<decltype(n)::value>, dim3((unsigned)((T + 3) / 4)),
                       dim3(256), 0, st, logits, ids, w, dw, (int)T, (int)E, (int)k, r, dlogits);
  });
  return hipGetLastError();
}

}  // namespace w4
