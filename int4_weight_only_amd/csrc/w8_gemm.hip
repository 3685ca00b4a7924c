// W8A8 products: e4m3 codes with block scales, fp32 accumulation, bf16 out.
//
//   Y[m, n] = bf16( sum_k X8[m, k] 2^SX[m, k/128] W8[n, k] 2^SW[n/128, k/128] )
//
// dense (w8a8_gemm) and grouped over aligned expert blocks (w8a8_moe_gemm).
#include <algorithm>
#include <type_traits>

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

// Four consecutive outputs n .. n + 3 of a row; vec: whole and aligned.
__device__ __forceinline__ void store4(uint16_t* row, int64_t n, int64_t N, f32x4 s, bool vec) {
  if (n >= N) return;
  const u32x2 o = {pk_bf16(s.x, s.y), pk_bf16(s.z, s.w)};
  uint16_t* y = row + n;
  if (vec) {
    *(u32x2*)y = o;
    return;
  }
  y[0] = (uint16_t)o.x;
  if (n + 1 < N) y[1] = (uint16_t)(o.x >> 16);
  if (n + 2 < N) y[2] = (uint16_t)o.y;
  if (n + 3 < N) y[3] = (uint16_t)(o.y >> 16);
}

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
// Bound by W's bytes: 1 x 12288 x 4096, 50 MB, 10 us (5.1 TB/s).  Staging W
// through LDS would add a barrier to loads that nothing shares.
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
    if (row >= 0) store4(Y + row * N, n0 + 16 * j + 4 * h, N, s, vec);
  }
}

// ------------------------------------------------------------- LDS tile --
// A workgroup of four waves computes BM = 32 MI rows of X times BN = 32 NI
// rows of W, wave (wm, wn) of the 2 x 2 waves 16 MI x 16 NI of them as
// MI x NI tiles of v_mfma_scale_f32_16x16x128.  Both operands go from memory
// straight into LDS (16-byte buffer_load ... lds), one 128-byte K block per
// step, two stages; a row's eight 16-byte pieces are stored XOR-swizzled by
// (row / 2) % 8, so that an operand read of 16 rows spreads over the banks.
//
// Large tiles (NST 2 or 3 stages) multiply a step in four quarters, (X low, W
// low), (X low, W high), (X high, W high), (X high, W low), so that a wave holds
// its operands once and reads them during the quarters before: the high halves
// in the first, then, when the next stage has landed, its low halves in the
// third and fourth, into registers whose half is done (W's two sets swap roles
// every step).  After the first quarter a stage has been read and its buffer
// takes the loads of NST steps ahead, spread over the other three quarters: in
// one burst they queue behind each other and land too late (4096 x 14336 x
// 4096: 223 us with the loads in the third quarter, 209 spread; 157 us of
// 4096 x 4096 x 16384's 224 are left without the traffic).  Reading all of X at
// the end of a step keeps the LDS busy twice as long as the MFMAs of that time
// (8192^3: 464 us, 400 in quarters).  An odd number of steps is made even by one
// of zeros (pieces past K read zero).
//
// Small tiles (four stages) hold two steps' operands: one multiplies while the
// next is read, one barrier a step, and loads have three steps to land.
//
// The scales of four K blocks are one dword a row; they pass through a small
// LDS ring the same way.
//
// KG > 1: KG such groups of four waves share the tile and split the steps
// between them, each with stages of its own, where too few tiles would leave
// CUs idle; their sums are joined through LDS in group order.
// GROUPED: the rows of a tile are sorted pairs of one expert, gathered by the
// loads.
//
// Rates: 4096 x 14336 x 4096 203 to 217 us by card (2.2 to 2.4 PFLOP/s), 8192^3
// 398 us (2.76), grouped 16384 rows of 32 experts x [4096, 4096] 292 to 298 us
// with SwiGLU (fusing it took 40 us off the layer); bound by the feed of operands
// (above).
// 2048 rows of 128 experts x [4096, 4096] in 64 x 256 tiles read W at 5.3 TB/s.
//
// SWIGLU (256 x 256, grouped): W's 2 I rows are gate, then up; a tile takes 128
// of each, in the waves wn = 0 and 1, which exchange half of their bf16
// products through LDS; the row's 128 values of silu(g) * u are one scale
// block, so the tile quantizes them itself and writes codes and scales (Y is
// A8, one byte a value).
namespace {

constexpr uint32_t kOOB = 0x80000000u;   // byte offset past any buffer: reads 0

__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}

// p and bytes are the same in every lane; said so, or each load would loop
// over the resources of the lanes
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, int64_t bytes) {
  const uint64_t a = (uint64_t)p;
  const uint64_t u = (uint64_t)uniform((uint32_t)(a >> 32)) << 32 | uniform((uint32_t)a);
  return __builtin_amdgcn_make_buffer_rsrc((void*)u, (short)0, (int)uniform((uint32_t)bytes),
                                           0x00020000);
}

typedef __attribute__((address_space(3))) void* lds_ptr;

__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, void* lds, uint32_t off,
                                           uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)lds, 16, off, soff, 0, 0);
}
__device__ __forceinline__ void load_lds4(__amdgpu_buffer_rsrc_t r, void* lds, uint32_t off,
                                          uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)lds, 4, off, soff, 0, 0);
}

}  // namespace

template <int MI, int NI, int KG, int NST, bool GROUPED, bool SWIGLU = false>
__global__ __launch_bounds__(256 * KG, 1) void k_w8_tile(const uint8_t* __restrict__ X8,
                                                         const uint8_t* __restrict__ SX,
                                                         const uint8_t* __restrict__ W8,
                                                         const uint8_t* __restrict__ SW,
                                                         uint16_t* __restrict__ Y, int64_t M,
                                                         int64_t N, int K, Grouped gr,
                                                         uint8_t* __restrict__ SA_out) {
  constexpr int BM = 32 * MI, BN = 32 * NI;
  static_assert(!SWIGLU || (GROUPED && MI == 8 && NI == 8), "128 gate and 128 up rows");
  constexpr int XA = BM / 32, XB = BN / 32;        // 1 KB loads per wave and stage
  static_assert(MI % 2 == 0 && NI % 2 == 0 && MI <= 8 && NI <= 8, "halves; one scale of W a wave");
  static_assert(NST >= 2 && NST <= 4, "stages");
  // each stage an object of its own: the compiler then knows which loads an
  // operand read has to wait for
  constexpr int SA = BM * 128, SB = BN * 128;
  constexpr bool S3 = NST > 2, S4 = NST > 3;
  __shared__ __attribute__((aligned(16))) uint8_t as0_[KG][SA], as1_[KG][SA];
  __shared__ __attribute__((aligned(16))) uint8_t bs0_[KG][SB], bs1_[KG][SB];
  __shared__ __attribute__((aligned(16))) uint8_t as2_[KG][S3 ? SA : 16], as3_[KG][S4 ? SA : 16];
  __shared__ __attribute__((aligned(16))) uint8_t bs2_[KG][S3 ? SB : 16], bs3_[KG][S4 ? SB : 16];
  __shared__ __attribute__((aligned(16))) uint32_t rx_[KG][2][256], rw_[KG][2][64];

  const int lane = threadIdx.x & 63;
  const int kg = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) & 3);
  const int wm = wave >> 1, wn = wave & 1;
  const int r16 = lane & 15, h = lane >> 4;
  uint8_t* const as0 = as0_[kg];
  uint8_t* const as1 = as1_[kg];
  uint8_t* const as2 = as2_[kg];
  uint8_t* const as3 = as3_[kg];
  uint8_t* const bs0 = bs0_[kg];
  uint8_t* const bs1 = bs1_[kg];
  uint8_t* const bs2 = bs2_[kg];
  uint8_t* const bs3 = bs3_[kg];
  auto& rx = rx_[kg];
  auto& rw = rw_[kg];
  // tile order: XCD x (workgroups round-robin over 8) walks a contiguous
  // range of tiles in groups of 8 row blocks of X, which share operands in
  // its L2
  if constexpr (GROUPED) M = min(M, (int64_t)gr.ntpp[0]);
  const int64_t inner = N / 2;                     // SWIGLU: gate rows, up rows
  const int64_t mt = (M + BM - 1) / BM, nt = SWIGLU ? inner / 128 : (N + BN - 1) / BN;
  const int64_t tiles = mt * nt, per = (tiles + 7) / 8;
  const int64_t t = (blockIdx.x % 8) * per + blockIdx.x / 8;
  if (t >= tiles || blockIdx.x / 8 >= per) return;
  const int64_t band = t / (8 * nt), in_band = t - band * 8 * nt;
  const int gm = (int)min((int64_t)8, mt - band * 8);
  const int64_t m0 = (band * 8 + in_band % gm) * BM, n0 = in_band / gm * (SWIGLU ? 128 : BN);

  const int cols = (int)w8_cols(K);
  const int steps = (K + 127) / 128;
  // this group's steps, a multiple of the stages for every group (those past
  // its own part of K are zeros)
  constexpr int ROUND = NST == 3 ? 2 : NST;
  const int share = ((steps + KG - 1) / KG + ROUND - 1) / ROUND * ROUND;
  const int first = kg * share, last = first + share;
  const int k_end = min(K, last * 128);
  if constexpr (GROUPED) {
    const int e = gr.expert_ids[m0 / gr.B];
    if (e < 0 || e >= gr.E || (uint32_t)gr.sorted_ids[m0] >= (uint32_t)gr.P) return;
    W8 += (int64_t)e * N * K;
    SW += (int64_t)e * w8_blocks(N) * cols;
  }
  const int rows_x = GROUPED ? BM : (int)min((int64_t)BM, M - m0);
  const int rows_w = (int)min((int64_t)BN, N - n0);
  const int64_t x0 = GROUPED ? 0 : m0, all_x = GROUPED ? gr.P / gr.div : rows_x;
  const __amdgpu_buffer_rsrc_t ar = rsrc(X8 + x0 * K, all_x * K);
  // SWIGLU: waves 0 and 1 load the gate rows, 2 and 3 the up rows
  const int64_t w0 = SWIGLU && wave >= 2 ? inner + n0 : n0;
  const __amdgpu_buffer_rsrc_t br = rsrc(W8 + w0 * K, (int64_t)(SWIGLU ? 128 : rows_w) * K);
  const __amdgpu_buffer_rsrc_t sar = rsrc(SX + x0 * cols, all_x * cols);
  const int64_t up = SWIGLU ? inner / 128 : 1;     // the second scale's distance from the first
  const __amdgpu_buffer_rsrc_t sbr =
      rsrc(SW + (n0 >> 7) * cols,
           (SWIGLU ? up + 1 : ((n0 + rows_w - 1) >> 7) - (n0 >> 7) + 1) * cols);
  // row of X, from x0, that tile row r stands for; -1: none
  auto x_row = [&](int r) {
    if constexpr (GROUPED) {
      const int f = gr.sorted_ids[m0 + r];
      return (uint32_t)f < (uint32_t)gr.P ? f / gr.div : -1;
    } else {
      return r < rows_x ? r : -1;
    }
  };

  // load I of a stage fills its rows 8 I .. 8 I + 7: lane l writes slot l % 8
  // of row l / 8, which holds piece (l % 8) ^ ((row / 2) % 8)
  auto piece = [&](int I) { return (lane & 7) ^ ((4 * I + (lane >> 4)) & 7); };
  uint32_t aoff[XA], boff[XB];
#pragma unroll
  for (int i = 0; i < XA; ++i) {
    const int I = wave * XA + i, r = x_row(8 * I + (lane >> 3));
    aoff[i] = r >= 0 ? (uint32_t)r * (uint32_t)K + 16u * piece(I) : kOOB;
  }
#pragma unroll
  for (int i = 0; i < XB; ++i) {
    const int I = wave * XB + i, r = SWIGLU ? (8 * I + (lane >> 3)) & 127 : 8 * I + (lane >> 3);
    boff[i] = SWIGLU || r < rows_w ? (uint32_t)r * (uint32_t)K + 16u * piece(I) : kOOB;
  }
  // row of the scale ring this lane fills
  const int srow = 64 * wave < BM ? x_row(64 * wave + lane) : -1;
  const uint32_t sxoff = srow >= 0 ? (uint32_t)(srow * cols) : kOOB;
  const uint32_t swoff = lane < 2 ? (uint32_t)(lane * up * cols) : kOOB;   // past the end: 0

  // load i of a wave's XA + XB of a stage
  auto load_one = [&](int i, int step, uint8_t* sa, uint8_t* sb) __attribute__((always_inline)) {
    const uint32_t k0 = (uint32_t)step * 128u;
    const int left = k_end - (int)k0;              // pieces past the end read zero
    if (i < XA) {
      const int I = wave * XA + i;
      load_lds16(ar, sa + I * 1024, 16 * piece(I) < left ? aoff[i] : kOOB, k0);
    } else {
      const int I = wave * XB + i - XA;
      load_lds16(br, sb + I * 1024, 16 * piece(I) < left ? boff[i - XA] : kOOB, k0);
    }
  };
  // quads past K repeat the row's last one: what lies behind it is another
  // row's, and a NaN scale there would reach this row through 0 * NaN
  const int last_quad = (steps - 1) >> 2;
  auto load_scales = [&](int quad) __attribute__((always_inline)) {
    const uint32_t at = (uint32_t)min(quad, last_quad) * 4u;
    load_lds4(sar, rx[quad & 1] + 64 * wave, sxoff, at);
    load_lds4(sbr, rw[quad & 1], swoff, at);                    // by every wave, the same bytes
  };
  // operand tile i of a wave's rows (16 rows keep the swizzle of the first)
  auto read = [&](const uint8_t* s, int at, int i) __attribute__((always_inline)) {
    return join16(*(const u32x4*)(s + at + 2048 * i), *(const u32x4*)(s + (at ^ 64) + 2048 * i));
  };
  const int xrow = wm * 16 * MI + r16;
  const int swz = 16 * (h ^ (r16 >> 1));
  const int xat = xrow * 128 + swz, wat = (wn * 16 * NI + r16) * 128 + swz;

  // a zero that the compiler does not see as constant: it would split loop
  // variables that start at one into single registers
  f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  asm("" : "+v"(zero));
  f32x4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = zero;
  // small tiles hold two steps' operands (WHOLE), large ones halves
  constexpr bool WHOLE = MI + NI <= 8;
  static_assert(WHOLE == (NST == 4), "stages of the two schedules");
  static_assert(NST != 3 || KG == 1, "three stages: any even number of steps");
  constexpr int HI = WHOLE ? MI : MI / 2, HJ = WHOLE ? NI : NI / 2;
  i32x8 x[2][HI], w[2][HJ];
  uint32_t sx[MI], sw;
  // the dword that holds a step's scale, and its place in it (steps past K take
  // the last step's)
  auto read_sx = [&](int step, int i) __attribute__((always_inline)) {
    return rx[(step >> 2) & 1][xrow + 16 * i];
  };
  auto read_sw = [&](int step) __attribute__((always_inline)) {
    return rw[(step >> 2) & 1][(wn * 16 * NI) >> 7];
  };
  auto shift = [&](int step) { return 8 * (min(step, steps - 1) & 3); };
  auto fence = [] __attribute__((always_inline)) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };

  // one quarter: rows hi of X, hj of W (in register set set); READ(i) reads
  // operand tile i for a later quarter, LOADS calls load LOAD(i) per MFMA
  auto quarter = [&](auto HX, auto HW, int set, auto read_one, int reads, auto load, int loads)
      __attribute__((always_inline)) {
    constexpr int hx = decltype(HX)::value, hw = decltype(HW)::value;
#pragma unroll
    for (int i = 0; i < reads; ++i) read_one(i);
#pragma unroll
    for (int i = 0; i < loads; ++i) load(i);
#pragma unroll
    for (int q = 0; q < HI * HJ; ++q) {
      // the operand that arrives last goes slowest
      const int i = hx == 0 ? q % HI : q / HJ, j = hx == 0 ? q / HI : q % HJ;
      f32x4& d = acc[hx * HI + i][hw * HJ + j];
      d = mfma8_16(w[set][j], x[hx][i], d, sw, sx[hx * HI + i]);
    }
#pragma unroll
    for (int q = 0; q < HI * HJ; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);          // one MFMA
      if (q < 2 * reads) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one LDS read
      if (q < loads) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);       // one load
    }
    fence();
  };
  using std::integral_constant;
  constexpr integral_constant<int, 0> lo{};
  constexpr integral_constant<int, 1> hi{};
  auto none = [](int) {};

  // small tiles, one step: its operands are in set S; the next one's are read
  // into the other while they multiply
  auto body_whole = [&](auto Q, int step, uint8_t* sa, uint8_t* sb, uint8_t* na, uint8_t* nb)
      __attribute__((always_inline)) {
    constexpr int q = decltype(Q)::value, s = q & 1;
    uint32_t nsx[MI], nsw;
    const int sh = shift(step + 1);
    // the loads of the two steps after the next may be in flight (the scales
    // came with the quad's first step)
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NST - 2) * (XA + XB) + (q == 1 || q == 2 ? 2 : 0))
                 : "memory");
    __builtin_amdgcn_s_barrier();
    fence();
    if (q == 0) load_scales(step / 4 + 1);
    nsw = read_sw(step + 1);
#pragma unroll
    for (int i = 0; i < MI; ++i) nsx[i] = read_sx(step + 1, i);
#pragma unroll
    for (int j = 0; j < NI; ++j) w[1 - s][j] = read(nb, wat, j);
#pragma unroll
    for (int i = 0; i < MI; ++i) x[1 - s][i] = read(na, xat, i);
    fence();
#pragma unroll
    for (int i = 0; i < XA + XB; ++i) load_one(i, step + NST, sa, sb);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = mfma8_16(w[s][j], x[s][i], acc[i][j], sw, sx[i]);
#pragma unroll
    for (int q = 0; q < MI * NI; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                    // one MFMA
      if (q < XA + XB) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);   // one load
    }
    fence();
#pragma unroll
    for (int i = 0; i < MI; ++i) sx[i] = nsx[i] >> sh;
    sw = nsw >> sh;
  };

  // one step on stage (sa, sb); (na, nb) is the next one's; the step's low
  // half of W is in set S
  auto body_halves = [&](auto S, int step, uint8_t* sa, uint8_t* sb, uint8_t* na, uint8_t* nb)
      __attribute__((always_inline)) {
    constexpr int s = decltype(S)::value;
    constexpr int L2 = (XA + XB) * 3 / 8, L3 = (XA + XB) * 3 / 8;   // loads per quarter
    uint32_t nsx[MI], nsw;
    const int sh = shift(step + 1);
    // read the rest of this stage; when everyone has, its buffer is free
    quarter(lo, lo, s,
            [&](int i) {
              if (i < HJ)
                w[1 - s][i] = read(sb, wat, HJ + i);
              else
                x[1][i - HJ] = read(sa, xat, HI + i - HJ);
            },
            HJ + HI, none, 0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    fence();
    load_scales((step + 1) / 4 + 1);
    quarter(lo, hi, 1 - s, none, 0, [&](int i) { load_one(i, step + NST, sa, sb); }, L2);
    // the next stage has landed; the loads just issued, and with three stages
    // those of the step before, may be in flight
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NST - 2) * (XA + XB + 2) + 2 + L2) : "memory");
    __builtin_amdgcn_s_barrier();
    fence();
    quarter(hi, hi, 1 - s, [&](int i) { x[0][i] = read(na, xat, i); }, HI,
            [&](int i) { load_one(L2 + i, step + NST, sa, sb); }, L3);
    nsw = read_sw(step + 1);
#pragma unroll
    for (int i = 0; i < MI; ++i) nsx[i] = read_sx(step + 1, i);
    quarter(hi, lo, s, [&](int i) { w[1 - s][i] = read(nb, wat, i); }, HJ,
            [&](int i) { load_one(L2 + L3 + i, step + NST, sa, sb); }, XA + XB - L2 - L3);
#pragma unroll
    for (int i = 0; i < MI; ++i) sx[i] = nsx[i] >> sh;
    sw = nsw >> sh;
  };

  // (the scales of the first two quads, some of them more than once)
  auto load_stage = [&](int step, int quad, uint8_t* sa, uint8_t* sb) __attribute__((always_inline)) {
    load_scales(quad);
#pragma unroll
    for (int i = 0; i < XA + XB; ++i) load_one(i, step, sa, sb);
  };
  load_stage(first, first / 4, as0, bs0);
  load_stage(first + 1, first / 4 + 1, as1, bs1);
  if constexpr (S3) load_stage(first + 2, first / 4 + 1, as2, bs2);
  if constexpr (S4) load_stage(first + 3, first / 4 + 1, as3, bs3);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NST - 1) * (XA + XB + 2)) : "memory");
  __builtin_amdgcn_s_barrier();
  fence();
#pragma unroll
  for (int i = 0; i < MI; ++i) sx[i] = read_sx(first, i) >> shift(first);
  sw = read_sw(first) >> shift(first);
#pragma unroll
  for (int i = 0; i < HI; ++i) x[0][i] = read(as0, xat, i);
#pragma unroll
  for (int j = 0; j < HJ; ++j) w[0][j] = read(bs0, wat, j);
  fence();
  for (int step = first; step < last; step += NST == 3 ? 6 : NST) {
    if constexpr (NST == 3) {
      body_halves(lo, step, as0, bs0, as1, bs1);
      body_halves(hi, step + 1, as1, bs1, as2, bs2);
      if (step + 2 >= last) break;
      body_halves(lo, step + 2, as2, bs2, as0, bs0);
      body_halves(hi, step + 3, as0, bs0, as1, bs1);
      if (step + 4 >= last) break;
      body_halves(lo, step + 4, as1, bs1, as2, bs2);
      body_halves(hi, step + 5, as2, bs2, as0, bs0);
    } else if constexpr (WHOLE) {
      body_whole(lo, step, as0, bs0, as1, bs1);
      body_whole(hi, step + 1, as1, bs1, as2, bs2);
      body_whole(integral_constant<int, 2>{}, step + 2, as2, bs2, as3, bs3);
      body_whole(integral_constant<int, 3>{}, step + 3, as3, bs3, as0, bs0);
    } else {
      body_halves(lo, step, as0, bs0, as1, bs1);
      body_halves(hi, step + 1, as1, bs1, as0, bs0);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // loads past the end drained

  if constexpr (KG > 1) {
    // one column of tiles per round through the stages that are done with
    f32x4(*part)[4][MI][64] = (f32x4(*)[4][MI][64])as0_;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      __syncthreads();
      if (kg > 0) {
#pragma unroll
        for (int i = 0; i < MI; ++i) part[kg][wave][i][lane] = acc[i][j];
      }
      __syncthreads();
      if (kg == 0) {
#pragma unroll
        for (int g = 1; g < KG; ++g)
#pragma unroll
          for (int i = 0; i < MI; ++i) acc[i][j] += part[g][wave][i][lane];
      }
    }
    if (kg > 0) return;
  }
  if constexpr (SWIGLU) {
    // wave wn keeps the row tiles 4 wn .. 4 wn + 3 and gives the others away, two
    // tiles a round
    uint32_t(*give)[2][NI][64][2] = (uint32_t(*)[2][NI][64][2])as0_;
    auto half = [&](auto WN) __attribute__((always_inline)) {
      constexpr int own = decltype(WN)::value;
      const int64_t cols_i = w8_cols(inner);
#pragma unroll
      for (int rd = 0; rd < 2; ++rd) {
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int j = 0; j < NI; ++j) {
            const f32x4 v = acc[4 * (1 - own) + 2 * rd + q][j];
            *(u32x2*)give[2 * wm + own][q][j][lane] = u32x2{pk_bf16(v.x, v.y), pk_bf16(v.z, v.w)};
          }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int i = 4 * own + 2 * rd + q;
          const int row = gr.sorted_ids[m0 + xrow + 16 * i];
          float a[NI][4];
          uint32_t top = 0;
#pragma unroll
          for (int j = 0; j < NI; ++j) {
            const f32x4 v = acc[i][j];
            const u32x2 mine = {pk_bf16(v.x, v.y), pk_bf16(v.z, v.w)};
            const u32x2 other = *(const u32x2*)give[2 * wm + 1 - own][q][j][lane];
            const u32x2 g = own == 0 ? mine : other, u = own == 0 ? other : mine;
            a[j][0] = silu_mul_fast(bf16_lo(g.x), bf16_lo(u.x));
            a[j][1] = silu_mul_fast(bf16_hi(g.x), bf16_hi(u.x));
            a[j][2] = silu_mul_fast(bf16_lo(g.y), bf16_lo(u.y));
            a[j][3] = silu_mul_fast(bf16_hi(g.y), bf16_hi(u.y));
#pragma unroll
            for (int r = 0; r < 4; ++r) top = max(top, __float_as_uint(a[j][r]) & 0x7FFFFFFFu);
          }
          // the row's other values are in lanes 16, 32 and 48 further
          top = max(top, (uint32_t)__shfl_xor((int)top, 16));
          top = max(top, (uint32_t)__shfl_xor((int)top, 32));
          if ((uint32_t)row >= (uint32_t)gr.P) continue;
          const uint32_t byte = scale_byte(top);
          const float inv = inv_scale(byte);
          uint8_t* out = (uint8_t*)Y + (int64_t)row * inner + n0 + 4 * h;
#pragma unroll
          for (int j = 0; j < NI; ++j)
            *(uint32_t*)(out + 16 * j) =
                byte == 255u ? 0x7F7F7F7Fu : codes4(a[j][0], a[j][1], a[j][2], a[j][3], inv);
          if (h == 0) {
            uint8_t* s = SA_out + (int64_t)row * cols_i;
            s[n0 >> 7] = (uint8_t)byte;
            if (n0 + 128 == inner)
              for (int64_t c = inner / 128; c < cols_i; ++c) s[c] = 127;   // padding
          }
        }
      }
    };
    if (wn == 0)
      half(lo);
    else
      half(hi);
    return;
  }
  const bool vec = (N & 3) == 0 && ((uintptr_t)Y & 7) == 0;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    int64_t row = m0 + xrow + 16 * i;
    if constexpr (GROUPED) {
      row = gr.sorted_ids[row];
      if ((uint32_t)row >= (uint32_t)gr.P) continue;
    } else if (row >= M) {
      continue;
    }
#pragma unroll
    for (int j = 0; j < NI; ++j)
      store4(Y + row * N, n0 + wn * 16 * NI + 16 * j + 4 * h, N, acc[i][j], vec);
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

template <int MI, int NI, int KG, int NST, bool GROUPED>
hipError_t tile(const uint8_t* X8, const uint8_t* SX, const uint8_t* W8, const uint8_t* SW,
                uint16_t* Y, int64_t M, int64_t N, int64_t K, const Grouped& gr, hipStream_t st) {
  const int64_t tiles = ((M + 32 * MI - 1) / (32 * MI)) * ((N + 32 * NI - 1) / (32 * NI));
  hipLaunchKernelGGL((k_w8_tile<MI, NI, KG, NST, GROUPED>), dim3((unsigned)((tiles + 7) / 8 * 8)),
                     dim3(256 * KG), 0, st, X8, SX, W8, SW, Y, M, N, (int)K, gr, nullptr);
  return hipGetLastError();
}

// The kernels and what they cost.  Tiles: a round of one workgroup per CU takes
// step_us per 128-wide step and fixed_us besides (launch, first loads, stores),
// measured with every CU busy and operands that come from memory.  The split
// kernel reads 16 rows of X and 16 of W per workgroup at 12 TB/s (L2) after
// 3.5 us.
struct Kind {
  int bm, bn, kg;
  float step_us, fixed_us;
};
constexpr Kind kKinds[] = {
    {16, 16, 0, 0.0f, 3.5f},     // split
    {64, 64, 2, 0.32f, 6.0f},
    {64, 128, 1, 0.40f, 6.0f},
    {128, 128, 1, 0.60f, 6.0f},
    {128, 256, 1, 1.05f, 10.0f},
    {192, 256, 1, 1.10f, 11.0f},
    {256, 256, 1, 1.35f, 12.0f},
};

int64_t tiles_of(const Kind& t, int64_t M, int64_t N) {
  return ((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn);
}

float estimate(int kind, int64_t M, int64_t N, int64_t K) {
  const Kind& t = kKinds[kind];
  const int64_t tiles = tiles_of(t, M, N), steps = (K + 127) / 128;
  if (kind == 0) return t.fixed_us + (float)tiles * (float)K * (32.0f / 12e6f);
  const int64_t cus = cu_count(), rounds = (tiles + cus - 1) / cus;
  return (float)rounds * ((float)((steps + t.kg - 1) / t.kg) * t.step_us + t.fixed_us);
}

// The kernel that the estimate says is done first.  Few large tiles move the
// least data, but leave CUs idle where they are too few: 4096 x 14336 x 4096
// takes 209 us in 896 tiles of 256 x 256, 278 in 1792 of 128 x 256 and 356 in
// 3584 of 128 x 128; 1024 x 4096 x 4096 takes 51, 36 and 26 us.  192 rows fit
// where 256 leave a third of the CUs idle and 128 need a second round: 2304 x
// 4096 x 4096 takes 40.5 us, 47.5 without them.
int pick(int64_t M, int64_t N, int64_t K, float& us) {
  int best = -1;
  for (int i = M <= 64 ? 0 : 1; i < (M <= 16 ? 1 : 7); ++i) {
    const float e = estimate(i, M, N, K);
    if (best < 0 || e < us) {
      best = i;
      us = e;
    }
  }
  return best;
}

// The split kernel's rows of W and waves per workgroup.  64 rows of W per
// workgroup share their rows of X, which counts once there are some and N fills
// the CUs (12288 x 4096, 16 rows of X: 12.5 us, 15.9 in 16 rows of W; 8192 x 4096:
// 12.7 and 11.7; from 9728 on 64 would do for 8 rows and more, 13.3 and 16.4 us
// at 16); else 16, on 16 waves where there are few workgroups and 8 where there
// are many (4096 x 7168: 7.6 and 9.2 us; 12288 x 4096: 10.7 and 10.0, one row).
struct Split {
  int bn, waves;
};
Split split_of(int64_t M, int64_t N) {
  const int64_t cus = cu_count();
  if (M > 2 && M <= 16 && N >= 48 * cus) return {64, 8};
  return {16, N <= 32 * cus ? 16 : 8};
}

hipError_t run_kind(int kind, const uint8_t* X8, const uint8_t* SX, const uint8_t* W8,
                    const uint8_t* SW, uint16_t* Y, int64_t M, int64_t N, int64_t K,
                    hipStream_t st) {
  const Grouped none = {};
  switch (kind) {
    case 0: {
      const int64_t slots = (M + 15) / 16;
      const Split p = split_of(M, N);
      if (p.bn == 64)
        return split<1, 4, 8, false>(X8, SX, W8, SW, Y, M, N, K, slots, none, st);
      if (p.waves == 16)
        return split<1, 1, 16, false>(X8, SX, W8, SW, Y, M, N, K, slots, none, st);
      return split<1, 1, 8, false>(X8, SX, W8, SW, Y, M, N, K, slots, none, st);
    }
    case 1: return tile<2, 2, 2, 4, false>(X8, SX, W8, SW, Y, M, N, K, none, st);
    case 2: return tile<2, 4, 1, 4, false>(X8, SX, W8, SW, Y, M, N, K, none, st);
    case 3: return tile<4, 4, 1, 4, false>(X8, SX, W8, SW, Y, M, N, K, none, st);
    case 4: return tile<4, 8, 1, 3, false>(X8, SX, W8, SW, Y, M, N, K, none, st);
    case 5: return tile<6, 8, 1, 2, false>(X8, SX, W8, SW, Y, M, N, K, none, st);
    default: return tile<8, 8, 1, 2, false>(X8, SX, W8, SW, Y, M, N, K, none, st);
  }
}

// Rows to leave to a launch of their own: up to 16 past a multiple of 128,
// where a row of tiles for them would cost more (2050 x 4096 x 5120: 2048 rows
// and 2 instead of 9 x 256).
int64_t rest_rows(int64_t M, int64_t N, int64_t K) {
  const int64_t rest = M % 128;
  if (M <= 128 || rest == 0 || rest > 16) return 0;
  float whole, main, few;
  pick(M, N, K, whole);
  pick(M - rest, N, K, main);
  pick(rest, N, K, few);
  return main + few < whole ? rest : 0;
}

}  // namespace

int64_t w8_gemm_threads(int64_t M, int64_t N, int64_t K) {
  const int64_t rest = rest_rows(M, N, K);
  int64_t most = 0;
  for (const int64_t rows : {M - rest, rest}) {
    if (rows == 0) continue;
    float us;
    const Kind& t = kKinds[pick(rows, N, K, us)];
    const Split p = split_of(rows, N);
    most = std::max(most, t.kg == 0 ? (rows + 15) / 16 * ((N + p.bn - 1) / p.bn) * 64 * p.waves
                                    : (tiles_of(t, rows, N) + 7) * 256 * t.kg);
  }
  return most;
}

hipError_t launch_w8_gemm(const uint8_t* X8, const uint8_t* SX, const uint8_t* W8,
                          const uint8_t* SW, uint16_t* Y, int64_t M, int64_t N, int64_t K,
                          hipStream_t st) {
  float us;
  const int64_t rest = rest_rows(M, N, K), main = M - rest;
  const hipError_t e = run_kind(pick(main, N, K, us), X8, SX, W8, SW, Y, main, N, K, st);
  if (e != hipSuccess || rest == 0) return e;
  return run_kind(pick(rest, N, K, us), X8 + main * K, SX + main * w8_cols(K), W8, SW, Y + main * N,
                  rest, N, K, st);
}

namespace {

int64_t moe_rows(int64_t T, int32_t k, int32_t E, int32_t B) {
  return (T * k + (int64_t)E * (B - 1) + B - 1) / B * B;
}

// Rows of the grouped product's tiles: a divisor of B.  The tiles gather with
// 32-bit offsets into X; where X is larger, the split kernel (64-bit
// addresses) takes the blocks 16 rows at a time, ten times as long (2^20 rows of
// 2048 x 32 experts of [4096, 2048]: 93 ms, 9.7 with eight rows less).
int moe_tile_rows(int64_t rows_x, int64_t K, int32_t B) {
  if (rows_x * K >= (int64_t)kOOB) return 16;
  for (int bm = 256; bm >= 64; bm /= 2)
    if (B % bm == 0) return bm;
  return B % 32 == 0 ? 32 : 16;
}

// Columns of the grouped product's tiles.  64 rows: 256 columns read weights in
// longer runs, if there are tiles for all CUs (at most one expert a pair): 256 x 8
// pairs over 128 of [4096, 4096] take 402 us, 418 in 128 columns; 64 x 2 over 8 of
// [4096, 4096] 33 and 26.
int moe_tile_cols(int rows, int64_t T, int32_t k, int32_t E, int64_t N) {
  if (rows <= 32) return 32;
  if (rows > 64) return 256;
  const int64_t blocks = std::max(std::min((int64_t)E, T * k), T * k / 64);
  return blocks * ((N + 255) / 256) >= cu_count() ? 256 : 128;
}

}  // namespace

int64_t w8_moe_threads(int64_t T, int32_t k, int32_t E, int64_t N, int64_t K, int32_t B,
                       int32_t x_row_div) {
  const int rows = moe_tile_rows(T * k / x_row_div, K, B), cols = moe_tile_cols(rows, T, k, E, N);
  return (moe_rows(T, k, E, B) / rows * ((N + cols - 1) / cols) + 7) * 256;
}

hipError_t launch_w8_moe_gemm(const uint8_t* X8, const uint8_t* SX, const uint8_t* W8,
                              const uint8_t* SW, const int32_t* sorted_ids,
                              const int32_t* expert_ids, const int32_t* ntpp, uint16_t* Y,
                              int64_t T, int32_t k, int32_t E, int64_t N, int64_t K, int32_t B,
                              int32_t x_row_div, hipStream_t st) {
  const Grouped gr = {sorted_ids, expert_ids, ntpp, (int)(T * k), E, B, x_row_div};
  const int64_t cap = moe_rows(T, k, E, B);
  const int rows = moe_tile_rows(T * k / x_row_div, K, B);
  switch (rows) {
    case 16: return split<1, 2, 4, true>(X8, SX, W8, SW, Y, 0, N, K, cap / 16, gr, st);
    case 32: return split<2, 2, 4, true>(X8, SX, W8, SW, Y, 0, N, K, cap / 32, gr, st);
    case 64:
      if (moe_tile_cols(rows, T, k, E, N) == 256)
        return tile<2, 8, 1, 3, true>(X8, SX, W8, SW, Y, cap, N, K, gr, st);
      return tile<2, 4, 1, 4, true>(X8, SX, W8, SW, Y, cap, N, K, gr, st);
    case 128: return tile<4, 8, 1, 3, true>(X8, SX, W8, SW, Y, cap, N, K, gr, st);
    default: return tile<8, 8, 1, 2, true>(X8, SX, W8, SW, Y, cap, N, K, gr, st);
  }
}

bool w8_moe_swiglu_fits(int64_t rows_x, int64_t I, int64_t K, int32_t B) {
  return I % 128 == 0 && moe_tile_rows(rows_x, K, B) == 256;
}

hipError_t launch_w8_moe_gemm_swiglu(const uint8_t* X8, const uint8_t* SX, const uint8_t* W8,
                                     const uint8_t* SW, const int32_t* sorted_ids,
                                     const int32_t* expert_ids, const int32_t* ntpp, uint8_t* A8,
                                     uint8_t* SA, int64_t T, int32_t k, int32_t E, int64_t I,
                                     int64_t K, int32_t B, int32_t x_row_div, hipStream_t st) {
  const Grouped gr = {sorted_ids, expert_ids, ntpp, (int)(T * k), E, B, x_row_div};
  const int64_t cap = moe_rows(T, k, E, B), tiles = cap / 256 * (I / 128);
  hipLaunchKernelGGL((k_w8_tile<8, 8, 1, 2, true, true>), dim3((unsigned)((tiles + 7) / 8 * 8)),
                     dim3(256), 0, st, X8, SX, W8, SW, (uint16_t*)A8, cap, 2 * I, (int)K, gr, SA);
  return hipGetLastError();
}

}  // namespace w4
