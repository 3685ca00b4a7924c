// The scored router: softmax or sigmoid scores, a bias for the choice, the
// best groups of experts, the k largest in them, weights from the scores;
// and its gradient to the logits.
//
// Scores, choice values, group sums and weights are held in 64 bits: two
// choice values of a row are often closer than 32 bits of an exponential
// tell apart (sixteen thousand rows of 384 hold several such pairs), and a
// swapped expert is another result, not a rounding.  Rows whose values 32 bits
// do tell apart, nearly all, are chosen by those.  One wave per token.
// 16384 x 384, sigmoid, bias: 18.7 us, 25.3 with 8 groups (the row's 1.5 KB would
// take 5 us): 430 and 565 vector instructions a row, many of them in chains of
// lane exchanges.  With groups the vector units issue in half to three fifths of
// the time; a wave spends half its cycles ready and not issuing, and a quarter in
// waits for memory and LDS.  72 us when every row is chosen in 64 bits.
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

// ------------------------------------------------------------- selection --
// NPER experts per lane; expert lane + 64 i is the lane's i-th, or NPER lane + i
// where the groups allow it.
// v: choice values, -Inf for masked experts.  Lane j < k gets pick j: its id, and
// whether it is one (slots without an expert left hold the lowest untaken
// indices).
//
// The quick form lets choice values from 32-bit exponentials decide where they
// are further apart than their errors can be; where some are not, the row is
// done again in 64 bits, where equal values also tie to the lower index.  A 32-bit score errs by less than 2.5e-7 (v_exp
// and v_rcp, one unit in the last place each; the rounding of the exponent's
// product counts by s (1 - s) |x| <= 0.23) and the sum with the bias by 2^-24
// of itself; softmax scores carry the error of their sum too, at most 1.7e-6 of
// a score for 1024 experts, and two of them add to at most one.  So two values are
// told apart if they differ by kApart (1 + |c|) and what their keys (below)
// leave of them, and two groups, whose worth may be the sum of two values, by
// 2 kApart (1 + |c|).
namespace {

constexpr float kApart = 2e-6f;

// slots of a lane, as a power of two
constexpr int slots_of(int nper) { return nper <= 1 ? 1 : nper <= 2 ? 2 : nper <= 4 ? 4 : nper <= 8 ? 8 : 16; }

__device__ __forceinline__ float wave_max_of(float a) {
  const auto x = [](int v, int w) { return fmaxf(__int_as_float(v), __int_as_float(w)); };
  a = x(__float_as_int(a), __builtin_amdgcn_mov_dpp(__float_as_int(a), 0xB1, 0xF, 0xF, false));
  a = x(__float_as_int(a), __builtin_amdgcn_mov_dpp(__float_as_int(a), 0x4E, 0xF, 0xF, false));
  a = x(__float_as_int(a), __builtin_amdgcn_mov_dpp(__float_as_int(a), 0x141, 0xF, 0xF, false));
  a = x(__float_as_int(a), __builtin_amdgcn_mov_dpp(__float_as_int(a), 0x140, 0xF, 0xF, false));
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(a), false, false);
  a = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(a), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ double wave_max_of(double a) { return wave_max64(a); }

// the value of one lane, the same one for the whole wave
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// a lane of the other half of 2 D lanes whose halves each hold one value
template <int D, class F>
__device__ __forceinline__ F from_other(F a) {
  if constexpr (D >= 16) {
    return __shfl_xor(a, D);
  } else {
    constexpr int ctrl = D == 1 ? 0xB1 : D == 2 ? 0x4E : D == 4 ? 0x141 : 0x140;
    if constexpr (sizeof(F) == 8) {
      return dpp64<ctrl>(a);
    } else {
      const int v = __float_as_int(a);
      return __int_as_float(__builtin_amdgcn_update_dpp(v, v, ctrl, 0xF, 0xF, true));
    }
  }
}
// the two largest, a >= b, of this and the other half
template <int D, class F>
__device__ __forceinline__ void join_two(F& a, F& b) {
  const F a2 = from_other<D>(a), b2 = from_other<D>(b);
  b = max(max(b, b2), min(a, a2));
  a = max(a, a2);
}

// Masks the experts of the groups that go; whether that is certain.
// `share` lanes, a power of two, hold each group's worth.  A lane's experts are
// `NPER` consecutive ones if `in_lanes`: its group is then `share` lanes' own
// registers.  Otherwise they are 64 apart and go through LDS.
template <int NPER, class F>
__device__ __forceinline__ bool limit_to_groups(F (&v)[NPER], F* mine, int E, const RouteRule& rule,
                                                int lane, bool in_lanes) {
  if (rule.groups == 1) return true;
  const F none = (F)-INFINITY;
  const int per = E / rule.groups;
  const int bits = 31 - __builtin_clz(64 / rule.groups), share = 1 << bits;
  const int g = lane >> bits;
  F a = none, b = none;                        // the two largest
  if (in_lanes) {
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      b = max(b, min(a, v[i]));
      a = max(a, v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPER; ++i)
      if (lane + 64 * i < E) mine[lane + 64 * i] = v[i];
    __builtin_amdgcn_wave_barrier();           // the wave's own LDS, in order
    if (g < rule.groups)
      for (int q = lane & (share - 1); q < per; q += share) {
        const F c = mine[g * per + q];
        b = max(b, min(a, c));
        a = max(a, c);
      }
    __builtin_amdgcn_wave_barrier();
  }
  if (share > 1) join_two<1>(a, b);
  if (share > 2) join_two<2>(a, b);
  if (share > 4) join_two<4>(a, b);
  if (share > 8) join_two<8>(a, b);
  if (share > 16) join_two<16>(a, b);
  const F worth = rule.group_top == 2 && b > none ? a + b : a;
  int rank = 0;
  for (int o = 0; o < rule.groups; ++o) {
    const F other = lane_value(worth, o << bits);
    rank += (other > worth) | ((other == worth) & (o < g));
  }
  const bool group = g < rule.groups;
  bool sure = true;
  if (sizeof(F) == 4 && rule.topk_groups < rule.groups) {
    // the worth of the last that stays and of the first that goes
    const uint64_t last = __ballot(group && rank == rule.topk_groups - 1);
    const uint64_t next = __ballot(group && rank == rule.topk_groups);
    const F in = lane_value(worth, (int)__builtin_ctzll(last));
    const F out = lane_value(worth, (int)__builtin_ctzll(next));
    if (out > none && !(in - out > (F)(2 * kApart) * (1 + fabs(in) + fabs(out)))) sure = false;
  }
  const uint64_t keep = __ballot(rank < rule.topk_groups);
  if (in_lanes) {
    const F limit = rank < rule.topk_groups ? (F)INFINITY : none;
#pragma unroll
    for (int i = 0; i < NPER; ++i) v[i] = min(v[i], limit);
  } else {
    // e / per as a product: exact for e, per <= 1024
    const uint32_t m = ((1u << 20) + per - 1) / per;
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      const int of = (int)(((lane + 64 * i) * m) >> 20) << bits;
      if (!((keep >> (of & 63)) & 1)) v[i] = none;
    }
  }
  return sure;
}

// A choice value as an integer of the same order, its low bits replaced by the
// slot it stands in: comparing, sorting and naming the winner are then integer
// maxima.  The slot moves the value by less than NPER units in the last place.
constexpr int kNone = INT32_MIN;
template <int NPER>
__device__ __forceinline__ int to_key(float c, int slot) {
  const int b = __float_as_int(c);
  const int ordered = b ^ ((b >> 31) & 0x7FFFFFFF);
  return c > -INFINITY ? ((ordered & ~(slots_of(NPER) - 1)) | slot) : kNone;
}
__device__ __forceinline__ float key_value(int key) {
  return __int_as_float(key ^ ((key >> 31) & 0x7FFFFFFF));
}

template <int CTRL>
__device__ __forceinline__ int max_with(int a) {
  return max(a, __builtin_amdgcn_update_dpp(a, a, CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ int wave_max_of(int a) {
  a = max_with<0xB1>(a);
  a = max_with<0x4E>(a);
  a = max_with<0x141>(a);
  a = max_with<0x140>(a);
  auto r = __builtin_amdgcn_permlane16_swap((uint32_t)a, (uint32_t)a, false, false);
  a = max((int)r[0], (int)r[1]);
  r = __builtin_amdgcn_permlane32_swap((uint32_t)a, (uint32_t)a, false, false);
  return max((int)r[0], (int)r[1]);
}

// sorts a lane's keys, largest first: Batcher's odd-even merge network, without
// the comparators that reach past the end
template <int NPER>
__device__ __forceinline__ void sort_keys(int (&v)[NPER]) {
#pragma unroll
  for (int p = 1; p < NPER; p *= 2)
#pragma unroll
    for (int q = p; q > 0; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < NPER; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < NPER && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const int hi = max(v[i + j], v[i + j + q]);
            v[i + j + q] = min(v[i + j], v[i + j + q]);
            v[i + j] = hi;
          }
}

// The quick form: false where values are too close or the masks leave fewer
// than k experts.  With each lane's keys sorted, a pick is the largest of the
// lanes' first ones and a shift in the lane that had it.
template <int NPER>
__device__ __forceinline__ bool choose(float (&c)[NPER], float* mine, int E, int k,
                                       const RouteRule& rule, int lane, bool in_lanes, int& my_id) {
  if (!limit_to_groups<NPER, float>(c, mine, E, rule, lane, in_lanes)) return false;
  int v[NPER];
#pragma unroll
  for (int i = 0; i < NPER; ++i) v[i] = to_key<NPER>(c[i], i);
  sort_keys<NPER>(v);
  int my_key = kNone;
  // one round more than picks: the first that stays out has to be apart too
  for (int j = 0; j <= k; ++j) {
    const int m = wave_max_of(v[0]);
    // one expert goes: an equal one stays, and shows as too close a call
    const int w = (int)__builtin_ctzll(__ballot(v[0] == m));
    // as masks: selections become an index into v, and that a chain of them
    const int won = lane == w ? -1 : 0;
#pragma unroll
    for (int i = 0; i < NPER; ++i) v[i] = ((i + 1 < NPER ? v[i + 1] : kNone) & won) | (v[i] & ~won);
    my_id = lane == j ? w : my_id;
    my_key = lane == j ? m : my_key;
  }
  const int slot = my_key & (slots_of(NPER) - 1);
  my_id = in_lanes ? NPER * my_id + slot : my_id + 64 * slot;
  const int next = __shfl_down(my_key, 1);
  const float a = key_value(my_key), b = key_value(next);
  const bool apart = next == kNone ? lane == k - 1 && my_key != kNone    // none left to be close to
                                   : a - b > kApart * (1.0f + fabsf(a) + fabsf(b)) +
                                                 slots_of(NPER) * 0x1p-23f * fmaxf(fabsf(a), fabsf(b));
  return __ballot(lane < k && !apart) == 0;
}

template <int NPER>
__device__ __forceinline__ void choose_exactly(double (&v)[NPER], double* mine, int E, int k,
                                               const RouteRule& rule, int lane, int& my_id,
                                               bool& my_live) {
  limit_to_groups<NPER, double>(v, mine, E, rule, lane, false);
  uint32_t free = 0;
#pragma unroll
  for (int i = 0; i < NPER; ++i) free |= lane + 64 * i < E ? 1u << i : 0u;
  for (int j = 0; j < k; ++j) {
    double m = v[0];
#pragma unroll
    for (int i = 1; i < NPER; ++i) m = fmax(m, v[i]);
    m = wave_max64(m);
    const bool any = m > -INFINITY;
    int win = -1;
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      const uint64_t b = __ballot(any ? v[i] == m : (free >> i) & 1u);
      if (win < 0 && b) win = 64 * i + (int)__builtin_ctzll(b);
    }
#pragma unroll
    for (int i = 0; i < NPER; ++i)
      if (win == lane + 64 * i) {
        v[i] = -INFINITY;
        free &= ~(1u << i);
      }
    if (lane == j) {
      my_id = win;
      my_live = any;
    }
  }
}

}  // namespace

namespace {

// A row's picks, for the wave that weighs them
struct Picked {
  RowSum rs;
  float x[16];
  int id[16];
};

// A lane's logits and biases, experts first, first + step, ...; a masked expert's
// bias is -Inf.
template <int NPER>
__device__ __forceinline__ void load_row(const float* row, const float* bias, int E, int first,
                                         int step, float (&x)[NPER], float (&add)[NPER]) {
  const uint32_t last = E - 1;
#pragma unroll
  for (int i = 0; i < NPER; ++i) x[i] = row[min((uint32_t)(first + step * i), last)];
#pragma unroll
  for (int i = 0; i < NPER; ++i) add[i] = 0.0f;
  if (bias) {
#pragma unroll
    for (int i = 0; i < NPER; ++i) add[i] = bias[min((uint32_t)(first + step * i), last)];
  }
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    x[i] = first + step * i < E ? x[i] : -INFINITY;
    // masked: by its logit or its bias
    add[i] = masked(x[i]) | masked(add[i]) ? -INFINITY : add[i];
  }
}

// sum over each row of 16 lanes, in every lane of it, in one fixed order
__device__ __forceinline__ double row16_sum64(double a) {
  a += dpp64<0xB1>(a);
  a += dpp64<0x4E>(a);
  a += dpp64<0x141>(a);
  return a + dpp64<0x140>(a);
}

}  // namespace

template <int NPER>
__global__ __launch_bounds__(256) void k_route_scored(const float* __restrict__ logits,
                                                      const float* __restrict__ bias, int T, int E,
                                                      int k, RouteRule rule,
                                                      int32_t* __restrict__ ids,
                                                      float* __restrict__ wts) {
  extern __shared__ double choice[];           // [4 waves][E]: only with groups
  __shared__ Picked picked[4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // rows past T: the last one again, not stored
  const int t = min((int)blockIdx.x * 4 + wave, T - 1);
  const float* row = logits + (int64_t)t * E;
  double* mine = choice + (int64_t)wave * E;
  // whole groups in neighbouring lanes: a lane holds consecutive experts
  const bool in_lanes = rule.groups > 1 && E == 64 * NPER && (rule.groups & (rule.groups - 1)) == 0;
  float x[NPER], add[NPER];
  load_row<NPER>(row, bias, E, in_lanes ? NPER * lane : lane, in_lanes ? 1 : 64, x, add);
  int my_id = 0;
  bool my_live = false, sure;
  float top = -INFINITY;                       // softmax: the row's largest logit
  {
    float c[NPER];
    if (rule.sigmoid) {
#pragma unroll
      for (int i = 0; i < NPER; ++i)
        c[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-x[i]));
    } else {
#pragma unroll
      for (int i = 0; i < NPER; ++i) {
        c[i] = masked(x[i]) ? -INFINITY : fminf(x[i], FLT_MAX);
        top = fmaxf(top, c[i]);
      }
      top = wave_max_of(top);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NPER; ++i) {
        c[i] = __expf(c[i] - top);
        sum += c[i];
      }
      sum += from_other<1>(sum);
      sum += from_other<2>(sum);
      sum += from_other<4>(sum);
      sum += from_other<8>(sum);
      sum += from_other<16>(sum);
      sum += from_other<32>(sum);
      const float inv = __builtin_amdgcn_rcpf(sum);
#pragma unroll
      for (int i = 0; i < NPER; ++i) c[i] *= inv;
    }
    // a masked expert's score may be anything, its value is -Inf
#pragma unroll
    for (int i = 0; i < NPER; ++i) c[i] = masked(add[i]) ? -INFINITY : c[i] + add[i];
    sure = choose<NPER>(c, (float*)mine, E, k, rule, lane, in_lanes, my_id);
    my_live = sure;
  }
  RowSum rs = {0.0, 1.0};
  if (!rule.sigmoid) {
    // renormalised: the picks' own largest logit will do, unless it is so far
    // below the row's that the scores are near zero in 64 bits too
    bool far = true;
    if (sure && rule.renorm) {
      const float best = wave_max_of(lane < k ? fminf(row[my_id], FLT_MAX) : -INFINITY);
      rs.top = (double)best;
      far = top - best >= 600.0f;
    }
    if (far) {
      load_row<NPER>(row, bias, E, lane, 64, x, add);
      rs = row_sum<NPER>(x, E, lane);
    }
  }
  if (!sure) {
    if (rule.sigmoid) load_row<NPER>(row, bias, E, lane, 64, x, add);
    double c[NPER];
#pragma unroll
    for (int i = 0; i < NPER; ++i)
      c[i] = masked(add[i]) ? -INFINITY : score(x[i], rule.sigmoid, rs) + (double)add[i];
    choose_exactly<NPER>(c, mine, E, k, rule, lane, my_id, my_live);
  }
  // the weights of four rows at once, 16 lanes each: their 64-bit exponentials
  // and divisions would take a wave per row as long as the choice
  if (lane < 16) {
    picked[wave].id[lane] = my_id;
    picked[wave].x[lane] = lane < k && my_live ? row[my_id] : -INFINITY;
    if (lane == 0) picked[wave].rs = rs;
  }
  __syncthreads();
  if (wave > 0) return;
  const Picked& p = picked[lane >> 4];
  const int j = lane & 15;
  double s = score(p.x[j], rule.sigmoid, p.rs);
  if (rule.renorm) {
    const double sum = row16_sum64(s);
    s = sum > 0.0 ? s / sum : 0.0;
  }
  const int64_t out = (int64_t)blockIdx.x * 4 + (lane >> 4);
  if (j < k && out < T) {
    ids[out * k + j] = p.id[j];
    wts[out * k + j] = (float)((double)rule.scale * s);
  }
}

// -------------------------------------------------------------- gradient --
// p over the picks (slots whose weight is zero took no part); the row is put
// together in LDS and written once.  Slots that name one expert twice add up in
// slot order.  16384 x 384: 9.4 us for 25 MB written and 6 read; the waves spend
// 77% of their cycles in waits, for the picks' logits, which come one by one, and
// for the wave that weighs them.  Softmax without renormalisation takes 25 us, a
// 64-bit exponential for every score.
template <int NPER>
__global__ __launch_bounds__(256) void k_route_scored_bwd(const float* __restrict__ logits,
                                                          const int32_t* __restrict__ ids,
                                                          const float* __restrict__ wts,
                                                          const float* __restrict__ dw, int T,
                                                          int E, int k, RouteRule rule,
                                                          float* __restrict__ dlogits) {
  __shared__ __attribute__((aligned(16))) float rows[4][64 * NPER];
  __shared__ RowSum sums[4];
  __shared__ double all_of[4];
  __shared__ float value[4][16];
  __shared__ int place[4][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // rows past T: the last one again, not stored
  const int t = min((int)blockIdx.x * 4 + wave, T - 1);
  const float* row = logits + (int64_t)t * E;
  float* mine = rows[wave];
  const bool dense = !rule.sigmoid && !rule.renorm;   // every score moves every weight
  float x[NPER];
  RowSum rs = {0.0, 1.0};
  if (dense) {
#pragma unroll
    for (int i = 0; i < NPER; ++i) x[i] = lane + 64 * i < E ? row[lane + 64 * i] : -INFINITY;
    rs = row_sum<NPER>(x, E, lane);
    if (lane == 0) sums[wave] = rs;
    __syncthreads();
  }
  // the picks of four rows at once, 16 lanes each
  if (wave == 0) {
    const int w = lane >> 4, j = lane & 15;
    const int64_t r = min((int64_t)blockIdx.x * 4 + w, (int64_t)T - 1);
    int id = -1;
    float y = -INFINITY;
    double g = 0.0;
    if (j < k) {
      const int e = ids[r * k + j];
      if (e >= 0 && e < E && wts[r * k + j] != 0.0f) {
        id = e;
        y = logits[r * E + e];
        g = (double)rule.scale * (double)dw[r * k + j];
      }
    }
    RowSum of = {0.0, 1.0};
    if (dense) {
      of = sums[w];
    } else if (!rule.sigmoid) {
      // renormalised softmax: only the picks' ratios count
      float top = masked(y) ? -INFINITY : fminf(y, FLT_MAX);
      for (int d = 1; d < 16; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
      of.top = (double)top;
    }
    const double s = score(y, rule.sigmoid, of);
    const double rest = rule.sigmoid ? score(-y, true, of) : 1.0;   // 1 - sigmoid, not cancelled
    double d, all = 0.0;
    if (rule.renorm) {
      const double sum = row16_sum64(s);
      const double p = sum > 0.0 ? s / sum : 0.0;
      d = p * (g - row16_sum64(g * p)) * rest;
    } else if (rule.sigmoid) {
      d = g * s * rest;
    } else {
      d = g * s;
      all = row16_sum64(d);
    }
    // the first slot of an expert sums those after it
    bool first = id >= 0;
    double v = 0.0;
    for (int q = 0; q < k; ++q) {
      const int other = __shfl(id, (lane & 48) + q);
      const double dq = __shfl(d, (lane & 48) + q);
      if (other == id) v += dq;
      if (other == id && q < j) first = false;
    }
    place[w][j] = first ? id : -1;
    value[w][j] = (float)(dense ? v - s * all : v);
    if (j == 0) all_of[w] = all;
  }
  if (!dense) {
#pragma unroll
    for (int i = 0; i < NPER; ++i) mine[lane + 64 * i] = 0.0f;
  }
  __syncthreads();
  if (dense) {
    const double all = all_of[wave];
#pragma unroll
    for (int i = 0; i < NPER; ++i) mine[lane + 64 * i] = (float)(-score(x[i], false, rs) * all);
    __builtin_amdgcn_wave_barrier();           // the wave's own LDS, in order
  }
  if (lane < 16 && place[wave][lane] >= 0) mine[place[wave][lane]] = value[wave][lane];
  __builtin_amdgcn_wave_barrier();
  if ((int)blockIdx.x * 4 + wave >= T) return;
  float* out = dlogits + (int64_t)t * E;
  if ((E & 3) == 0 && ((uintptr_t)dlogits & 15) == 0) {
    for (int q = lane; q < E / 4; q += 64) ((f32x4*)out)[q] = ((const f32x4*)mine)[q];
  } else {
#pragma unroll
    for (int i = 0; i < NPER; ++i)
      if (lane + 64 * i < E) out[lane + 64 * i] = mine[lane + 64 * i];
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
