// bf16 products of training: grouped by expert over aligned blocks, and with
// the rows (tokens) as the summed dimension.
//
//   rows grouped      Y[f] = X[f / div] W_e^T, or X[f / div] W_e
//   sums grouped      dW[e] = sum over e's pairs f of dY[f / a]^T X[f / b]
//   dense sums        C = A^T B
//
// Bf16 operands, fp32 accumulation in a fixed order, one rounding to bf16 (the type of
// the activations, gradients and master weights here).  The second operand of a sum
// may be a checkpoint of e4m3 codes.
//
// Kernels: k_bf16_tile (tiles of 64 x 64 to 256 x 256), k_bf16_short (results that are
// large next to their sums), k_bf16_join (sums in parts).  The host picks by what each
// is estimated to take (choose).
#include <algorithm>
#include <type_traits>

#include "bf16.h"

namespace w4 {

namespace {

// Which dimension the expert's pairs are.
enum Group { kDense, kRows, kSums };

// f / d for f < 2^31, with m = floor((2^32 - 1) / d): the high product is the
// quotient or one less.
struct Div {
  uint32_t d, m;
};
__device__ __forceinline__ int div_by(uint32_t f, Div v) {
  const uint32_t q = __umulhi(f, v.m);
  return (int)(f - q * v.d >= v.d ? q + 1 : q);
}

struct Job {
  const uint16_t* A;        // [*, K] rows summed along, or (TA) [*, M] with the sum down the rows
  Bf16Rows B;
  uint16_t* C;
  int64_t M, N, K;          // C is M x N (kRows: M slots; a row of C a pair), K the summed dimension
  Bf16Plan g;
  int32_t a_div, b_div;     // pairs per row of A, of B
  float* part;              // splits > 1: that many partial sums of each C, fp32, one after another
  int32_t splits;
  int32_t blocks;           // blocks that there may be: cap / B
  Div by_a, by_b;           // a_div, b_div
  Div by_block;             // B
  // a tile kernel's: columns of tiles (8 of them a band), tiles of an XCD for a sum
  int32_t mt, nt, per;
  Div by_band, by_per, by_splits;
  int32_t run;              // k_bf16_short: tiles of a workgroup, side by side (nt counts such runs)
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

// The blocks of expert e: [first, last).  Both ends are searched for together (the
// loads of a pass depend on the pass before, about 0.7 us each).
struct Blocks {
  int first, last;
};
__device__ __forceinline__ Blocks blocks_of(const Job& j, int e) {
  const Bf16Plan& g = j.g;
  const int lane = threadIdx.x & 63;
  const int total = g.ntpp[0];
  const int all = j.blocks;
  auto key = [&](int b) { return (uint32_t)g.expert_ids[b]; };     // -1 past the end: last
  int lo, hi;
  if (all <= 64 * 64) {
    const int step = (all + 63) / 64;
    const uint32_t k = lane * step < all ? key(lane * step) : ~0u;
    const int below_lo = __popcll(__ballot(k < (uint32_t)e)), below_hi = __popcll(__ballot(k <= (uint32_t)e));
    lo = max((below_lo - 1) * step + 1, 0);
    hi = max((below_hi - 1) * step + 1, 0);
    if (step > 1) {
      const uint32_t a = lane < step - 1 && lo + lane < all ? key(lo + lane) : ~0u;
      const uint32_t b = lane < step - 1 && hi + lane < all ? key(hi + lane) : ~0u;
      lo += below_lo == 0 ? 0 : __popcll(__ballot(a < (uint32_t)e));
      hi += below_hi == 0 ? 0 : __popcll(__ballot(b <= (uint32_t)e));
    }
  } else {
    lo = first_not(all, [&](int b) { return key(b) < (uint32_t)e; });
    hi = first_not(all, [&](int b) { return key(b) <= (uint32_t)e; });
  }
  hi = __builtin_amdgcn_readfirstlane(min(hi, div_by((uint32_t)max(total, 0), j.by_block)));
  lo = __builtin_amdgcn_readfirstlane(min(lo, hi));
  return {lo, hi};
}

// Pairs in an expert's last block: a prefix of its slots.
__device__ __forceinline__ int pairs_of_block(const Bf16Plan& g, int block) {
  const int lane = threadIdx.x & 63;
  int n = 0;
  for (int i = 0; i < g.B; i += 256) {
    uint32_t f[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int at = i + 64 * q + lane;
      f[q] = at < g.B ? (uint32_t)g.sorted_ids[block * g.B + at] : ~0u;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) n += __popcll(__ballot(f[q] < (uint32_t)g.P));
  }
  return __builtin_amdgcn_readfirstlane(n);
}

// The lower and the upper two of four e4m3 codes times a power of two, as bf16.
__device__ __forceinline__ uint32_t cvt2(uint32_t codes, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, s, false));
}
__device__ __forceinline__ uint32_t cvt2h(uint32_t codes, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, s, true));
}

}  // namespace

// --------------------------------------------------------------- LDS tile --
// A workgroup of four waves computes BM = 32 MI rows of C times BN = 32 NI
// columns, wave (wm, wn) of the 2 x 2 waves 16 MI x 16 NI of them as MI x NI tiles
// of v_mfma_f32_16x16x32_bf16.  Both operands go from memory straight into LDS
// (16-byte buffer_load ... lds), 64 of the summed dimension per step.  An operand
// whose rows run along the sum is stored [row][64], its eight 16-byte pieces
// XOR-swizzled by (row / 2) % 8.  One whose rows run across it (TA, TB: weights in
// the input gradient, both operands of a weight gradient) is stored as it lies in
// memory, [64][BM or BN], in units of 32 bytes XOR-swizzled by its row, and read
// through ds_read_b64_tr_b16, which hands four rows of 16 columns to 16 lanes
// column-wise: the transposition costs no instruction, and the swizzle spreads the
// eight rows that 32 lanes read over all banks (no bank conflicts measured).
//
// What bounds it.  Long sums on many tiles (256 x 256): the matrix unit and the loads
// that feed it, 1.45 us per round and 64 of the sum (1.6 PFLOP/s while running), and
// about 9 us per round to begin and to store, which nothing hides on a CU that holds
// one workgroup.  4096 x 8 pairs over 64 of [4096, 2048]: 587 us (937 TFLOP/s), the input
// gradient 597, with the experts' last blocks half empty; weight gradient over 32 of
// [4096, 4096]: 1165 (944); dense sums 4096^3: 100 us (1370 TFLOP/s).  The matrix unit
// is busy 61% of the CUs' cycles by rows, 44% in sums.
// Few pairs: the experts' weights from memory (8 pairs of 8 [1024, 1024]: 6.5 us;
// 256 x 2 pairs over 64 of [4096, 2048]: 209 us, 5.1 TB/s).
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

// Small tiles leave room for others on their CU: one loads or stores while another
// multiplies.
constexpr int workgroups_per_cu(int mi, int ni) {
  return mi * ni <= 4 ? 4 : mi * ni <= 8 ? 3 : mi * ni <= 16 ? 2 : 1;
}

// Order of the large tiles of a product by rows: groups of rows x cols tiles, `across`
// of them side by side, `groups` in all; what an XCD holds at a time (32) where there
// is enough, else about four groups for each.
struct Order {
  int rows, cols, across, groups;
};
__host__ __device__ __forceinline__ Order order(int mt, int nt) {
  const int rows = mt < 8 ? mt : 8, share = mt * nt / (32 * rows);
  const int cols = share < 1 ? 1 : share < 4 ? share : 4;
  const int across = (nt + cols - 1) / cols;
  return {rows, cols, across, (mt + rows - 1) / rows * across};
}

typedef __attribute__((address_space(3))) void* lds_ptr;
typedef short i16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, void* lds, uint32_t off,
                                           uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)lds, 16, off, soff, 0, 0);
}

// What a lane without a row reads where addresses have 64 bits.
__device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {0u, 0u, 0u, 0u};

// 16 bytes at the index'th 16 bytes from base; kOOB (and what is added to it): zeros.
typedef const __attribute__((address_space(1))) uint8_t* global_ptr;
__device__ __forceinline__ global_ptr wide_address(const uint8_t* base, uint32_t index) {
  return (global_ptr)((int)index >= 0 ? (uint64_t)base + ((uint64_t)index << 4) : (uint64_t)kZeros);
}
__device__ __forceinline__ void load_lds16_wide(const uint8_t* base, void* lds, uint32_t index) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)wide_address(base, index),
                                   (lds_ptr)lds, 16, 0, 0);
}

// Four rows of 16 columns, column-wise: lane c of each 16 gets column c.
__device__ __forceinline__ u32x2 read_tr(const uint8_t* s) {
  return __builtin_bit_cast(
      u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                 (__attribute__((address_space(3))) i16x4*)(__attribute__((address_space(3))) void*)s));
}

// Outputs of two neighbouring tiles of 16 columns: lane (r16, h) gives columns
// 4 h .. 4 h + 3 of row r16 of each and gets eight consecutive ones, of the first
// tile in h = 0, 1 and of the second in h = 2, 3, so that a store covers 64 bytes of
// a row instead of 32.
__device__ __forceinline__ u32x4 join_tiles(f32x4 a, f32x4 b) {
  typedef uint32_t u2 __attribute__((ext_vector_type(2)));
  u2 x = {pk_bf16(a.x, a.y), pk_bf16(b.x, b.y)}, y = {pk_bf16(a.z, a.w), pk_bf16(b.z, b.w)};
  x = __builtin_amdgcn_permlane32_swap(x.x, x.y, false, false);
  y = __builtin_amdgcn_permlane32_swap(y.x, y.y, false, false);
  x = __builtin_amdgcn_permlane16_swap(x.x, x.y, false, false);
  y = __builtin_amdgcn_permlane16_swap(y.x, y.y, false, false);
  return u32x4{x.x, y.x, x.y, y.y};
}

// Eight consecutive outputs n .. n + 7 of a row; vec: N is a multiple of 8, and the
// address of 16 bytes.
__device__ __forceinline__ void store8(uint16_t* row, int64_t n, int64_t N, u32x4 v, bool vec) {
  if (n >= N) return;
  if (vec) {
    *(u32x4*)(row + n) = v;
    return;
  }
  const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (n + i < N) row[n + i] = (uint16_t)(d[i >> 1] >> (16 * (i & 1)));
}

// Swizzle of a row (of the summed dimension) in units of 32 bytes: the eight
// rows {0..3, 8..11} (or {4..7, 12..15}) that 32 lanes read together get eight
// different places in 256 bytes.
template <int RB>
__device__ __forceinline__ int tr_swizzle(int row) {
  return RB >= 256 ? (row & 3) | ((row >> 3) & 1) << 2 : ((row >> 1) & 1) | ((row >> 3) & 1) << 1;
}

struct Operand {           // 16 rows x 64 of the sum: two MFMA operands
  u32x4 lo, hi;
};

}  // namespace

// A step is multiplied in four quarters, (A low, B low), (A low, B high), (A high, B
// high), (A high, B low), so that a wave holds its operands once and reads them during
// the quarters before: the high halves in the first, then, when the next stage has
// landed, its low halves in the third and fourth, into registers whose half is done
// (B's two sets swap roles every step).  After the first quarter a stage has been read
// and its buffer takes the loads of two steps ahead, spread over the other three
// quarters.  An odd number of steps is made even by one of zeros.
//
// Splits: workgroups that take a run of the steps each and leave fp32 sums to be
// joined (k_bf16_join).
//
// kRows: the rows of a tile are sorted pairs of one expert, gathered by the loads.
// kSums: the summed rows of both operands are the pairs of one expert, which
// are turned into byte offsets a step ahead of the loads.
//
// C8: B is a checkpoint.  Its codes come into registers, 16 of a row with their
// scale a lane, become bf16 by v_cvt_scalef32_pk_bf16_fp8 (which applies the power of
// two) and go into the stage as bf16 rows would, so that each element is converted
// once a workgroup and memory sees half the bytes.
//
// WIDE: offsets count 16 bytes and addresses have 64 bits, for operands of 2 GiB and
// more, which buffer loads do not reach.
template <int MI, int NI, Group G, bool TA, bool TB, bool C8, bool WIDE = false>
__global__ __launch_bounds__(256, workgroups_per_cu(MI, NI)) void k_bf16_tile(Job j) {
  constexpr int BM = 32 * MI, BN = 32 * NI;
  constexpr int XA = BM / 32, XB = C8 ? 0 : BN / 32;   // 1 KB loads per wave and stage
  constexpr int XC = C8 ? BN / 64 : 0;             // 16 codes each, and their scales
  static_assert(!C8 || (TA && TB), "rows across the sum");
  static_assert(MI % 2 == 0 && NI % 2 == 0 && MI <= 8 && NI <= 8, "halves");
  static_assert(!TA || (MI & (MI - 1)) == 0, "lanes of a row");
  static_assert(!TB || (NI & (NI - 1)) == 0, "lanes of a row");
  constexpr bool PARTS = MI * NI <= 16;            // large tiles are not for few results
  static_assert(G == kSums ? TA && TB : true, "pairs run across both operands");
  constexpr int SA = BM * 128, SB = BN * 128;
  // each stage an object of its own: the compiler then knows which loads an
  // operand read has to wait for
  __shared__ __attribute__((aligned(16))) uint8_t as0[SA], as1[SA];
  __shared__ __attribute__((aligned(16))) uint8_t bs0[SB], bs1[SB];
  __shared__ __attribute__((aligned(16))) u32x4 rows_[4][G == kSums ? 64 : 1];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) & 3);
  const int wm = wave >> 1, wn = wave & 1;
  const int r16 = lane & 15, h = lane >> 4;

  // tile order (workgroups go round-robin over 8 XCDs): the tiles that an XCD runs
  // at a time are groups of 8 row blocks by some columns, which share operands in
  // its L2.
  // (32-bit arithmetic and divisors prepared by the host: every tile begins with it)
  const int M = (int)j.M, nt = j.nt;
  constexpr bool DEALT = G == kRows && workgroups_per_cu(MI, NI) == 1;
  int mt = j.mt, m0, n0, e = 0, split = 0;
  if constexpr (DEALT) {
    // such groups are dealt to the XCDs in turn, over all the blocks that there may
    // be: how many there are need not be known to begin, and the last ones, which are
    // not there, are missed by every XCD alike
    const Order o = order(mt, nt);
    const int i = blockIdx.x / 8, size = o.rows * o.cols, round = i / size, w = i - round * size;
    const int group = round * 8 + blockIdx.x % 8, band = group / o.across;
    const int row = band * o.rows + w % o.rows, col = (group - band * o.across) * o.cols + w / o.rows;
    if (row >= mt || col >= nt) return;            // (with it the groups past the last)
    m0 = row * BM;
    n0 = col * BN;
  } else {
    // XCD x walks a contiguous range; an expert's tiles are spread over all XCDs,
    // since hot experts would keep one busy
    int per = j.per, at = blockIdx.x / 8, chunk = blockIdx.x % 8, part;   // which sum, or part of one
    if constexpr (G == kRows) {
      mt = (min(M, j.g.ntpp[0]) + BM - 1) / BM;
      per = max((mt * nt + 7) / 8, 1);
      part = at / per;
    } else {
      part = div_by((uint32_t)at, j.by_per);
    }
    at -= part * per;
    if constexpr (G == kSums) e = div_by((uint32_t)part, j.by_splits);
    split = part - e * j.splits;
    const int tiles = mt * nt;
    chunk = (chunk + 8 - (int)((uint32_t)part * (uint32_t)tiles % 8)) % 8;   // few tiles: another XCD for the next one
    const int t = chunk * per + at;
    if (t >= tiles || split >= j.splits) return;
    const int band = div_by((uint32_t)t, j.by_band), in_band = t - band * 8 * nt;
    const int gm = min(8, mt - band * 8);
    const int col = in_band / gm;
    m0 = (band * 8 + in_band - col * gm) * BM;
    n0 = col * BN;
  }

  int sum = G == kSums ? 0 : (int)j.K;             // length of the sum
  const int32_t* ids = j.g.sorted_ids;
  const uint16_t* A = j.A;
  const uint8_t* B = (const uint8_t*)j.B.p;
  constexpr int BB = C8 ? 1 : 2;                   // bytes of an element of B
  uint16_t* C = j.C;
  if constexpr (G == kRows) {
    const int total = j.g.ntpp[0];
    e = j.g.expert_ids[div_by((uint32_t)m0, j.by_block)];
    if (m0 >= total || e < 0 || e >= j.g.E || (uint32_t)ids[m0] >= (uint32_t)j.g.P) return;
    B += (int64_t)e * j.N * j.K * BB;
  }
  __amdgpu_buffer_rsrc_t ir = rsrc(nullptr, 0);
  // kSums: lane l's pair of a coming step, row l of the 64
  auto load_id = [&](int step) __attribute__((always_inline)) {
    return G == kSums ? (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(ir, (step * 64 + lane) * 4, 0, 0) : 0u;
  };
  uint32_t f[4] = {0u, 0u, 0u, 0u};                // the pairs of the first steps
  if constexpr (G == kSums) {
    const Blocks b = blocks_of(j, e);
    C += (int64_t)e * M * j.N;
    if (b.first == b.last) {                       // no pairs: zeros
      if (j.splits == 1) {
        for (int i = threadIdx.x; i < BM * (BN / 8); i += 256) {
          const int row = m0 + i / (BN / 8), col = n0 + i % (BN / 8) * 8;
          if (row < M && col < j.N) *(u32x4*)(C + (int64_t)row * j.N + col) = u32x4{0u, 0u, 0u, 0u};
        }
        return;
      }
    } else {
      const int start = b.first * j.g.B;
      ir = rsrc(ids + start, (int64_t)(b.last - b.first) * j.g.B * 4);
      if constexpr (!PARTS) {                      // on their way beside the last block's
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = load_id(i);
      }
      sum = (b.last - 1 - b.first) * j.g.B + pairs_of_block(j.g, b.last - 1);
    }
  }
  const int steps = (sum + 63) / 64;
  // this part's steps, an even number for every part (those past the sum are zeros)
  const int share = PARTS ? (div_by((uint32_t)(steps + j.splits - 1), j.by_splits) + 1) / 2 * 2 : (steps + 1) / 2 * 2;
  const int first = PARTS ? split * share : 0, last = first + share;
  const int k_end = min(sum, last * 64);

  const int64_t lda = TA ? M : j.K, ldb = TB ? j.N : j.K;     // elements of a row in memory
  const int pairs = (int)j.g.P;
  const int64_t rows_a = TA ? (G == kSums ? div_by((uint32_t)pairs, j.by_a) : sum)
                            : (G == kRows ? div_by((uint32_t)pairs, j.by_a) : min(BM, M - m0));
  const int64_t rows_b =
      TB ? (G == kSums ? div_by((uint32_t)pairs, j.by_b) : sum) : min((int64_t)BN, j.N - n0);
  // from the tile's first column (TA, TB) or row on
  const __amdgpu_buffer_rsrc_t ar =
      rsrc(A + (TA ? (int64_t)m0 : (G == kRows ? 0 : m0 * lda)), (rows_a * lda - (TA ? m0 : 0)) * 2);
  const __amdgpu_buffer_rsrc_t br =
      rsrc(B + (TB ? n0 : n0 * ldb) * BB, (rows_b * ldb - (TB ? n0 : 0)) * BB);
  const int64_t lds = w8_cols(j.N);                // C8: scales of a row
  const __amdgpu_buffer_rsrc_t sr =
      rsrc(C8 ? j.B.scales + (n0 >> 7) : nullptr, C8 ? rows_b * lds - (n0 >> 7) : 0);

  // Load I of a stage.  Rows along the sum: it fills rows 8 I .. 8 I + 7, lane l
  // slot l % 8 of row l / 8, which holds piece (l % 8) ^ ((row / 2) % 8).
  // Across: rows of RB bytes, lane l slot l % LR of row l / LR.
  constexpr int LRA = BM / 8, LRB = BN / 8;
  auto piece = [&](int I) { return (lane & 7) ^ ((4 * I + (lane >> 4)) & 7); };
  auto trow = [&](int I, int LR) { return I * (64 / LR) + lane / LR; };
  auto tcol = [&](int slot, int swz) { return 8 * (((slot >> 1) ^ swz) << 1 | (slot & 1)); };
  constexpr int CPR = BN / 16;                     // codes: lanes of a row
  auto crow = [&](int i) { return (i * 256 + wave * 64 + lane) / CPR; };
  // byte offset of the lane's 16 bytes at step 0 (WIDE: offset in units of 16, here and
  // below); of its column alone (kSums); past the end: kOOB
  const uint8_t* const abase = (const uint8_t*)(A + (TA ? (int64_t)m0 : (G == kRows ? 0 : m0 * lda)));
  const uint8_t* const bbase = B + (TB ? n0 : n0 * ldb) * BB;
  auto offset = [](int64_t bytes) __attribute__((always_inline)) {
    return WIDE ? (uint32_t)(bytes >> 4) : (uint32_t)bytes;
  };
  uint32_t aoff[XA], boff[C8 ? 1 : XB];
#pragma unroll
  for (int i = 0; i < XA; ++i) {
    const int I = wave * XA + i;
    if constexpr (TA) {
      const int row = trow(I, LRA), col = tcol(lane % LRA, tr_swizzle<2 * BM>(row));
      aoff[i] = m0 + col < M ? offset(((G == kSums ? 0 : row * lda) + col) * 2) : kOOB;
    } else {
      const int r = 8 * I + (lane >> 3);
      int64_t row = r < rows_a ? r : -1;
      if constexpr (G == kRows) {
        const uint32_t f = (uint32_t)ids[m0 + r];
        row = f < (uint32_t)j.g.P ? (int64_t)div_by(f, j.by_a) : -1;
      }
      aoff[i] = row >= 0 ? offset((row * lda + 8 * piece(I)) * 2) : kOOB;
    }
  }
#pragma unroll
  for (int i = 0; i < XB; ++i) {                   // (none of codes)
    const int I = wave * XB + i;
    if constexpr (TB) {
      const int row = trow(I, LRB), col = tcol(lane % LRB, tr_swizzle<2 * BN>(row));
      boff[i] = n0 + col < j.N ? offset(((G == kSums ? 0 : row * ldb) + col) * 2) : kOOB;
    } else {
      const int r = 8 * I + (lane >> 3);
      boff[i] = r < rows_b ? offset((r * ldb + 8 * piece(I)) * 2) : kOOB;
    }
  }
  // kSums: lane l holds the pair of row l of a coming step (loaded a step before it
  // is needed), turns it into the byte offsets of that row in A and B (kOOB: none),
  // and the loads' lanes take theirs out of a corner of LDS that is the wave's own
  uint32_t arow[G == kSums ? XA : 1], brow[G == kSums ? (C8 ? XC : XB) : 1], srow[C8 ? XC : 1];
  auto next_rows = [&](int step, uint32_t f) __attribute__((always_inline)) {
    if constexpr (G == kSums) {
      u32x4* q = rows_[wave];                  // a wave's LDS operations keep their order
      const bool ok = step * 64 + lane < k_end && f < (uint32_t)j.g.P;
      const uint32_t fb = (uint32_t)div_by(f, j.by_b);
      const uint32_t fa = (uint32_t)div_by(f, j.by_a);
      q[lane] = ok ? u32x4{WIDE ? offset(fa * lda * 2) : fa * (uint32_t)lda * 2u,
                           WIDE ? offset(fb * ldb * BB) : fb * (uint32_t)ldb * BB, C8 ? fb * (uint32_t)lds : 0u, 0u}
                   : u32x4{kOOB, kOOB, kOOB, 0u};
#pragma unroll
      for (int i = 0; i < XA; ++i) {
        const u32x2 o = *(const u32x2*)&q[trow(wave * XA + i, LRA)];
        arow[i] = o.x;
        if constexpr (XA == XB) brow[i] = o.y;
      }
      if constexpr (XA != XB && !C8) {
#pragma unroll
        for (int i = 0; i < XB; ++i) brow[i] = q[trow(wave * XB + i, LRB)].y;
      }
      if constexpr (C8) {
#pragma unroll
        for (int i = 0; i < XC; ++i) {
          const u32x4 o = q[crow(i)];
          brow[i] = o.y;
          srow[i] = o.z;
        }
      }
    }
  };
  // load i of the codes: 16 of row crow(i), from the lane's column on
  u32x4 code[C8 ? XC : 1];
  uint32_t scale[C8 ? XC : 1];
  const int ccol = 16 * (lane % CPR);
  const bool cok = n0 + ccol < j.N;
  const uint32_t cs = (uint32_t)(((n0 + ccol) >> 7) - (n0 >> 7));
  auto load_codes = [&](int step) __attribute__((always_inline)) {
    if constexpr (C8) {
#pragma unroll
      for (int i = 0; i < XC; ++i) {
        if constexpr (WIDE) {
          const int left = k_end - step * 64;
          const uint32_t from = G == kSums ? brow[i] : offset((left > 0 ? step * 64 + crow(i) : 0) * ldb);
          const bool ok = cok && (G == kSums || crow(i) < left);
          code[i] = *(const __attribute__((address_space(1))) u32x4*)wide_address(bbase, ok ? from + ccol / 16 : kOOB);
          scale[i] = __builtin_amdgcn_raw_buffer_load_b8(
              sr, G == kSums ? (int)(srow[i] + cs) : ok ? (int)((step * 64 + crow(i)) * (uint32_t)lds + cs) : (int)kOOB, 0, 0);
        } else if constexpr (G == kSums) {
          code[i] = __builtin_amdgcn_raw_buffer_load_b128(br, cok ? (int)(brow[i] + ccol) : (int)kOOB, 0, 0);
          scale[i] = __builtin_amdgcn_raw_buffer_load_b8(sr, (int)(srow[i] + cs), 0, 0);
        } else {
          const int left = k_end - step * 64;
          const uint32_t from = left > 0 ? (uint32_t)step * 64u : 0u;
          const bool ok = cok && crow(i) < left;
          code[i] = __builtin_amdgcn_raw_buffer_load_b128(
              br, ok ? (int)(crow(i) * (uint32_t)ldb + ccol) : (int)kOOB, (int)(from * (uint32_t)ldb), 0);
          scale[i] = __builtin_amdgcn_raw_buffer_load_b8(
              sr, ok ? (int)(crow(i) * (uint32_t)lds + cs) : (int)kOOB, (int)(from * (uint32_t)lds), 0);
        }
      }
    }
  };
  auto put_codes = [&](uint8_t* sb) __attribute__((always_inline)) {
    if constexpr (C8) {
#pragma unroll
      for (int i = 0; i < XC; ++i) {
        const int row = crow(i);
        u32x4* d = (u32x4*)(sb + row * 2 * BN + ((2 * ccol) ^ (32 * tr_swizzle<2 * BN>(row))));
        const float s = __uint_as_float(scale[i] << 23);
        const u32x4 c = code[i];
        d[0] = u32x4{cvt2(c.x, s), cvt2h(c.x, s), cvt2(c.y, s), cvt2h(c.y, s)};
        d[1] = u32x4{cvt2(c.z, s), cvt2h(c.z, s), cvt2(c.w, s), cvt2h(c.w, s)};
      }
    }
  };
  // load i of a wave's XA + XB of a stage
  auto load_one = [&](int i, int step, uint8_t* sa, uint8_t* sb) __attribute__((always_inline)) {
    const int k0 = step * 64, left = k_end - k0;   // what lies past the end reads zero,
    const uint32_t from = left > 0 ? (uint32_t)k0 * 2u : 0u;       // at offsets inside 32 bits
    if constexpr (WIDE) {
      const bool a = i < XA;
      const int I = a ? wave * XA + i : wave * XB + i - XA;
      const bool across = a ? TA : TB;
      const uint32_t own = a ? aoff[a ? i : 0] : boff[C8 || a ? 0 : i - XA];
      uint32_t index;
      if constexpr (G == kSums) {
        index = own != kOOB ? (a ? arow[a ? i : 0] : brow[C8 || a ? 0 : i - XA]) + own : kOOB;
      } else {
        const bool ok = own != kOOB && (across ? trow(I, a ? LRA : LRB) : 8 * piece(I)) < left;
        index = ok ? own + offset(across ? from * (a ? lda : ldb) : (int64_t)from) : kOOB;
      }
      load_lds16_wide(a ? abase : bbase, (a ? sa : sb) + I * 1024, index);
    } else if (i < XA) {
      const int I = wave * XA + i;
      if constexpr (G == kSums) {
        load_lds16(ar, sa + I * 1024, aoff[i] != kOOB ? arow[i] + aoff[i] : kOOB, 0);
      } else if constexpr (TA) {
        load_lds16(ar, sa + I * 1024, trow(I, LRA) < left ? aoff[i] : kOOB, from * (uint32_t)lda);
      } else {
        load_lds16(ar, sa + I * 1024, 8 * piece(I) < left ? aoff[i] : kOOB, from);
      }
    } else {
      const int b = i - XA, I = wave * XB + b;
      if constexpr (G == kSums) {
        load_lds16(br, sb + I * 1024, boff[b] != kOOB ? brow[b] + boff[b] : kOOB, 0);
      } else if constexpr (TB) {
        load_lds16(br, sb + I * 1024, trow(I, LRB) < left ? boff[b] : kOOB, from * (uint32_t)ldb);
      } else {
        load_lds16(br, sb + I * 1024, 8 * piece(I) < left ? boff[b] : kOOB, from);
      }
    }
  };
  constexpr int EX = G == kSums ? 1 : 0;           // a step's load of pairs
  // operand tile i of a wave's rows
  const int arow0 = wm * 16 * MI, brow0 = wn * 16 * NI;
  const int swz = 16 * (h ^ (r16 >> 1));
  const int at_a = TA ? (8 * h + (r16 >> 2)) * 2 * BM + (r16 & 3) * 8 : (arow0 + r16) * 128 + swz;
  const int at_b = TB ? (8 * h + (r16 >> 2)) * 2 * BN + (r16 & 3) * 8 : (brow0 + r16) * 128 + swz;
  const int swz_a = 32 * tr_swizzle<2 * BM>(8 * h + (r16 >> 2)), swz_b = 32 * tr_swizzle<2 * BN>(8 * h + (r16 >> 2));
  auto read_across = [&](const uint8_t* s, int RB) __attribute__((always_inline)) {
    const u32x2 a = read_tr(s), b = read_tr(s + 4 * RB), c = read_tr(s + 32 * RB), d = read_tr(s + 36 * RB);
    return Operand{u32x4{a.x, a.y, b.x, b.y}, u32x4{c.x, c.y, d.x, d.y}};
  };
  auto read_a = [&](const uint8_t* s, int i) __attribute__((always_inline)) {
    if constexpr (TA) return read_across(s + at_a + ((arow0 * 2 + 32 * i) ^ swz_a), 2 * BM);
    return Operand{*(const u32x4*)(s + at_a + 2048 * i), *(const u32x4*)(s + (at_a ^ 64) + 2048 * i)};
  };
  auto read_b = [&](const uint8_t* s, int i) __attribute__((always_inline)) {
    if constexpr (TB) return read_across(s + at_b + ((brow0 * 2 + 32 * i) ^ swz_b), 2 * BN);
    return Operand{*(const u32x4*)(s + at_b + 2048 * i), *(const u32x4*)(s + (at_b ^ 64) + 2048 * i)};
  };
  constexpr int RA = TA ? 4 : 2, RBN = TB ? 4 : 2;   // LDS reads of an operand tile

  // a zero that the compiler does not see as constant: it would split loop
  // variables that start at one into single registers
  f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  asm("" : "+v"(zero));
  f32x4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int n = 0; n < NI; ++n) acc[i][n] = zero;
  constexpr int HI = MI / 2, HJ = NI / 2;
  Operand x[2][HI], w[2][HJ];
  uint32_t id = 0;                                 // kSums: the pair that next_rows turns next
  auto fence = [] __attribute__((always_inline)) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&](f32x4& d, const Operand& b, const Operand& a) __attribute__((always_inline)) {
    d = mfma16(b.lo, a.lo, d);
    d = mfma16(b.hi, a.hi, d);
  };

  // one quarter: rows hx of A, hw of B (in register set set); read_one(i) reads
  // operand tile i for a later quarter (nr LDS reads in all), load(i) is load i
  auto quarter = [&](auto HX, auto HW, int set, auto read_one, int reads, int nr, auto load, int loads,
                     auto also) __attribute__((always_inline)) {
    constexpr int hx = decltype(HX)::value, hw = decltype(HW)::value;
#pragma unroll
    for (int i = 0; i < reads; ++i) read_one(i);
#pragma unroll
    for (int i = 0; i < loads; ++i) load(i);
    also();
#pragma unroll
    for (int q = 0; q < HI * HJ; ++q) {
      // the operand that arrives last goes slowest
      const int i = hx == 0 ? q % HI : q / HJ, n = hx == 0 ? q / HI : q % HJ;
      multiply(acc[hx * HI + i][hw * HJ + n], w[set][n], x[hx][i]);
    }
#pragma unroll
    for (int q = 0; q < 2 * HI * HJ; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);          // one MFMA
      if (q < nr) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);        // one LDS read
      if (q % 2 == 0 && q / 2 < loads) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);   // one load
    }
    fence();
  };
  using std::integral_constant;
  constexpr integral_constant<int, 0> lo{};
  constexpr integral_constant<int, 1> hi{};
  auto none = [](int) {};
  auto nothing = [] {};

  // one step on stage (sa, sb); (na, nb) is the next one's; the step's low
  // half of B is in set S
  auto body = [&](auto S, int step, uint8_t* sa, uint8_t* sb, uint8_t* na, uint8_t* nb)
      __attribute__((always_inline)) {
    constexpr int s = decltype(S)::value;
    constexpr int L2 = (XA + XB) * 3 / 8, L3 = (XA + XB) * 3 / 8;   // loads per quarter
    // read the rest of this stage; when everyone has, its buffer is free
    quarter(lo, lo, s,
            [&](int i) {
              if (i < HJ)
                w[1 - s][i] = read_b(sb, HJ + i);
              else
                x[1][i - HJ] = read_a(sa, HI + i - HJ);
            },
            HJ + HI, HJ * RBN + HI * RA, none, 0, nothing);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    fence();
    const uint32_t coming = load_id(step + 4);
    quarter(lo, hi, 1 - s, none, 0, 0, [&](int i) { load_one(i, step + 2, sa, sb); }, L2, nothing);
    // the next stage has landed; the loads just issued may be in flight, and the codes
    // of the step before, its last loads
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(EX + L2 + 2 * XC) : "memory");
    __builtin_amdgcn_s_barrier();
    fence();
    quarter(hi, hi, 1 - s, [&](int i) { x[0][i] = read_a(na, i); }, HI, HI * RA,
            [&](int i) { load_one(L2 + i, step + 2, sa, sb); }, L3, nothing);
    quarter(hi, lo, s, [&](int i) { w[1 - s][i] = read_b(nb, i); }, HJ, HJ * RBN,
            [&](int i) { load_one(L2 + L3 + i, step + 2, sa, sb); }, XA + XB - L2 - L3,
            [&] {
              put_codes(sb);
              next_rows(step + 3, id);
            });
    // behind the fence: the wait above counts these as the step's last loads
    load_codes(step + 3);
    fence();
    id = coming;
  };

  // the pairs of the first stages together, then the stages
  if constexpr (PARTS) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = load_id(first + i);
  }
  auto load_stage = [&](int i, uint8_t* sa, uint8_t* sb) __attribute__((always_inline)) {
    next_rows(first + i, f[i]);
    load_codes(first + i);
#pragma unroll
    for (int n = 0; n < XA + XB; ++n) load_one(n, first + i, sa, sb);
    put_codes(sb);
  };
  load_stage(0, as0, bs0);
  load_stage(1, as1, bs1);
  next_rows(first + 2, f[2]);
  id = f[3];
  fence();
  load_codes(first + 2);
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(C8 ? 2 * XC : XA + XB) : "memory");
  __builtin_amdgcn_s_barrier();
  fence();
#pragma unroll
  for (int i = 0; i < HI; ++i) x[0][i] = read_a(as0, i);
#pragma unroll
  for (int n = 0; n < HJ; ++n) w[0][n] = read_b(bs0, n);
  fence();
  for (int step = first; step < last; step += 2) {
    body(lo, step, as0, bs0, as1, bs1);
    body(hi, step + 1, as1, bs1, as0, bs0);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // loads past the end drained

  if constexpr (PARTS) {
    if (j.splits > 1) {
      // kRows: a row a pair, filled up to whole pieces of eight
      const int64_t width = G == kRows ? (j.N + 7) / 8 * 8 : j.N;
      float* const sums = j.part + ((G == kSums ? e : 0) * j.splits + split) * (G == kRows ? j.g.P : M) * width;
  #pragma unroll
      for (int i = 0; i < MI; ++i) {
        int64_t row = m0 + arow0 + r16 + 16 * i;
        bool ok = row < M;
        if constexpr (G == kRows) {
          row = ids[row];
          ok = (uint32_t)row < (uint32_t)j.g.P;
        }
  #pragma unroll
        for (int n = 0; n < NI; ++n) {
          const int64_t col = n0 + brow0 + 16 * n + 4 * h;
          if (ok && col < width) *(f32x4*)(sums + row * width + col) = acc[i][n];
        }
      }
      return;
    }
  }
  const bool vec = (j.N & 7) == 0 && ((uintptr_t)C & 15) == 0;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    int64_t row = m0 + arow0 + r16 + 16 * i;
    bool ok = row < M;
    if constexpr (G == kRows) {
      row = ids[row];
      ok = (uint32_t)row < (uint32_t)j.g.P;
    }
#pragma unroll
    for (int n = 0; n < NI; n += 2) {
      const u32x4 v = join_tiles(acc[i][n], acc[i][n + 1]);
      if (ok) store8(C + row * j.N, n0 + brow0 + 16 * n + 8 * h, j.N, v, vec);
    }
  }
}

// ---------------------------------------------------------------- short sums --
// Sums over few pairs write far more than they read and multiply, so that what a tile
// costs is its beginning (the search for the expert's pairs, their rows, the first
// loads: one load after the other) and its stores.  A workgroup therefore computes a
// run of 128 x 128 tiles side by side: it begins once, A's rows stay in LDS where they
// are one stage, and the loads of the next tile are under way below the products and
// the stores of this one.  Longer sums are right too, stage after stage.
// Measured (64 x 4 pairs over 32 of [1408, 2048]): 38 us, 63 in tiles of a workgroup
// each; 512 x 2 over 64 of [4096, 2048]: 252 and 438, 4.3 TB/s of stores, which bound it.
template <Group G, bool C8>
__global__ __launch_bounds__(256, 2) void k_bf16_short(Job j) {
  constexpr int BM = 128, BN = 128, MI = 4, NI = 4, RB = 256;
  constexpr int X = 4, XC = C8 ? 2 : 0;            // 1 KB loads per wave and operand; codes: 16 each
  constexpr int STORES = MI * NI / 2;
  __shared__ __attribute__((aligned(16))) uint8_t as0[BM * 128], as1[BM * 128];
  __shared__ __attribute__((aligned(16))) uint8_t bs0[BN * 128], bs1[BN * 128];
  __shared__ __attribute__((aligned(16))) u32x4 rows_[4][64];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) & 3);
  const int r16 = lane & 15, h = lane >> 4;
  const int M = (int)j.M, N = (int)j.N, runs = j.nt, tiles = j.mt * runs;
  const int at = blockIdx.x / 8, e = div_by((uint32_t)at, j.by_per);
  const int chunk = (blockIdx.x % 8 + 8 - (int)((uint32_t)e * (uint32_t)tiles % 8)) % 8;
  const int t = chunk * j.per + at - e * j.per;
  if (t >= tiles) return;
  const int band = div_by((uint32_t)t, j.by_band);
  const int m0 = band * BM, first = (t - band * runs) * j.run * BN, end = min(first + j.run * BN, N);

  int sum = (int)j.K;
  __amdgpu_buffer_rsrc_t ir = rsrc(nullptr, 0);
  auto load_id = [&](int step) __attribute__((always_inline)) {
    const int at = step * 64 + lane;
    return G == kSums ? (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(ir, at * 4, 0, 0) : (uint32_t)at;
  };
  uint32_t id;
  uint16_t* C = j.C;
  if constexpr (G == kSums) {
    const Blocks b = blocks_of(j, e);
    C += (int64_t)e * M * N;
    ir = rsrc(j.g.sorted_ids + b.first * j.g.B, (int64_t)(b.last - b.first) * j.g.B * 4);
    id = load_id(0);
    sum = b.last == b.first ? 0 : (b.last - 1 - b.first) * j.g.B + pairs_of_block(j.g, b.last - 1);
  } else {
    id = load_id(0);
  }
  const int steps = max((sum + 63) / 64, 1);       // none: one of zeros
  const int pairs = G == kSums ? (int)j.g.P : sum;
  const int64_t rows_a = div_by((uint32_t)pairs, j.by_a), rows_b = div_by((uint32_t)pairs, j.by_b);
  const int64_t ls = w8_cols(N);
  const __amdgpu_buffer_rsrc_t ar = rsrc(j.A, rows_a * M * 2), br = rsrc(j.B.p, rows_b * N * (C8 ? 1 : 2));
  const __amdgpu_buffer_rsrc_t sr = rsrc(j.B.scales, C8 ? rows_b * ls : 0);
  const __amdgpu_buffer_rsrc_t cr = rsrc(C, (int64_t)M * N * 2);

  // load i of an operand: lane's row of the stage and its column of the tile
  auto trow = [&](int i) { return 4 * (wave * X + i) + lane / 16; };
  auto tcol = [&](int i) {
    return 8 * ((((lane & 15) >> 1) ^ tr_swizzle<RB>(trow(i))) << 1 | (lane & 1));
  };
  auto crow = [&](int i) { return 32 * i + 8 * wave + lane / 8; };
  const int ccol = 16 * (lane & 7);
  uint32_t arow[X], brow[C8 ? XC : X], srow[C8 ? XC : 1];
  auto next_rows = [&](int step, uint32_t f) __attribute__((always_inline)) {
    u32x4* q = rows_[wave];                        // the wave's own
    const bool ok = step * 64 + lane < sum && f < (uint32_t)pairs;
    const uint32_t fb = (uint32_t)div_by(f, j.by_b);
    q[lane] = ok ? u32x4{(uint32_t)div_by(f, j.by_a) * (uint32_t)M * 2u, fb * (uint32_t)N * (C8 ? 1u : 2u),
                         C8 ? fb * (uint32_t)ls : 0u, 0u}
                 : u32x4{kOOB, kOOB, kOOB, 0u};
#pragma unroll
    for (int i = 0; i < X; ++i) {
      const u32x2 o = *(const u32x2*)&q[trow(i)];
      arow[i] = o.x;
      if constexpr (!C8) brow[i] = o.y;
    }
#pragma unroll
    for (int i = 0; i < XC; ++i) {
      const u32x4 o = q[crow(i)];
      brow[i] = o.y;
      srow[i] = o.z;
    }
  };
  u32x4 code[C8 ? XC : 1];
  uint32_t scale[C8 ? XC : 1];
  auto load_a = [&](uint8_t* s) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < X; ++i) {
      const int col = m0 + tcol(i);
      load_lds16(ar, s + (wave * X + i) * 1024, col < M ? arow[i] + 2 * col : kOOB, 0);
    }
  };
  auto load_b = [&](int n0, uint8_t* s) __attribute__((always_inline)) {
    if constexpr (!C8) {
#pragma unroll
      for (int i = 0; i < X; ++i) {
        const int col = n0 + tcol(i);
        load_lds16(br, s + (wave * X + i) * 1024, col < N ? brow[i] + 2 * col : kOOB, 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < XC; ++i) {
        const int col = n0 + ccol;
        code[i] = __builtin_amdgcn_raw_buffer_load_b128(br, col < N ? (int)(brow[i] + col) : (int)kOOB, 0, 0);
        scale[i] = __builtin_amdgcn_raw_buffer_load_b8(sr, col < N ? (int)(srow[i] + (col >> 7)) : (int)kOOB, 0, 0);
      }
    }
  };
  auto put_codes = [&](uint8_t* s) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < XC; ++i) {
      u32x4* d = (u32x4*)(s + crow(i) * RB + ((2 * ccol) ^ (32 * tr_swizzle<RB>(crow(i)))));
      const float f = __uint_as_float(scale[i] << 23);
      const u32x4 c = code[i];
      d[0] = u32x4{cvt2(c.x, f), cvt2h(c.x, f), cvt2(c.y, f), cvt2h(c.y, f)};
      d[1] = u32x4{cvt2(c.z, f), cvt2h(c.z, f), cvt2(c.w, f), cvt2h(c.w, f)};
    }
  };
  const int arow0 = (wave >> 1) * 16 * MI, brow0 = (wave & 1) * 16 * NI;
  const int from = (8 * h + (r16 >> 2)) * RB + (r16 & 3) * 8, swz = 32 * tr_swizzle<RB>(8 * h + (r16 >> 2));
  auto read = [&](const uint8_t* s, int col) __attribute__((always_inline)) {
    s += from + ((2 * col) ^ swz);
    const u32x2 a = read_tr(s), b = read_tr(s + 4 * RB), c = read_tr(s + 32 * RB), d = read_tr(s + 36 * RB);
    return Operand{u32x4{a.x, a.y, b.x, b.y}, u32x4{c.x, c.y, d.x, d.y}};
  };
  uint32_t row_at[MI];                             // of C
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int row = m0 + arow0 + r16 + 16 * i;
    row_at[i] = row < M ? (uint32_t)row * (uint32_t)N * 2u : kOOB;
  }

  f32x4 acc[MI][NI] = {};
  int n0 = first, step = 0;
  next_rows(0, id);
  load_a(as0);
  load_b(n0, bs0);
  id = steps > 1 ? load_id(1) : id;
  if constexpr (C8) put_codes(bs0);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  // one stage: its operands are (sa, sb), the next one's go into (na, nb).  Every wave's
  // loads have been waited for when it comes here, and its reads of (na, nb) are done.
  auto body = [&](const uint8_t* sa, const uint8_t* sb, uint8_t* na, uint8_t* nb)
      __attribute__((always_inline)) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const bool done = step + 1 == steps;
    const int next = done ? n0 + BN : n0;
    const bool more = next < end;
    step = done ? 0 : step + 1;
    if (more) {
      if (steps > 1) {
        next_rows(step, id);
        load_a(na);
        id = load_id(step + 1 == steps ? 0 : step + 1);
      }
      load_b(next, nb);
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    Operand x[MI], w[NI];
#pragma unroll
    for (int n = 0; n < NI; ++n) w[n] = read(sb, brow0 + 16 * n);
#pragma unroll
    for (int i = 0; i < MI; ++i) x[i] = read(sa, arow0 + 16 * i);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int n = 0; n < NI; ++n) {
        acc[i][n] = mfma16(w[n].lo, x[i].lo, acc[i][n]);
        acc[i][n] = mfma16(w[n].hi, x[i].hi, acc[i][n]);
      }
    if constexpr (C8) {
      if (more) put_codes(nb);
    }
    if (done) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int n = 0; n < NI; n += 2) {
          const int col = n0 + brow0 + 16 * n + 8 * h;
          const u32x4 v = join_tiles(acc[i][n], acc[i][n + 1]);
          __builtin_amdgcn_raw_buffer_store_b128(v, cr, col < N ? (int)(row_at[i] + 2 * col) : (int)kOOB, 0, 0);
          acc[i][n] = acc[i][n + 1] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
      // the next stage's loads came before these stores
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(STORES) : "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    n0 = next;
    return more;
  };
  if (steps == 1) {
    while (body(as0, bs0, as0, bs1) && body(as0, bs1, as0, bs0)) {}
  } else {
    while (body(as0, bs0, as1, bs1) && body(as1, bs1, as0, bs0)) {}
  }
}

// Partial sums joined in their order and rounded to bf16, eight columns a thread: of
// groups of `rows` rows, or (kRows) of the pairs that slots name.
template <Group G>
__global__ __launch_bounds__(256) void k_bf16_join(Job j, int64_t rows, int64_t pieces) {
  const int64_t width = (j.N + 7) / 8 * 8;
  const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (p >= pieces) return;
  int64_t row = p / (width / 8), group = 0;
  const int64_t col = (p - row * (width / 8)) * 8;
  if constexpr (G == kRows) {
    if (row >= j.g.ntpp[0]) return;
    row = j.g.sorted_ids[row];
    if ((uint32_t)row >= (uint32_t)j.g.P) return;
    const int e = j.g.expert_ids[(p / (width / 8)) / j.g.B];
    if (e < 0 || e >= j.g.E) return;
  } else {
    group = row / rows;
    row -= group * rows;
  }
  const float* q = j.part + (group * j.splits * rows + row) * width + col;
  f32x4 a = *(const f32x4*)q, b = *(const f32x4*)(q + 4);
  for (int s = 1; s < j.splits; ++s) {
    q += rows * width;
    a += *(const f32x4*)q;
    b += *(const f32x4*)(q + 4);
  }
  const u32x4 v = {pk_bf16(a.x, a.y), pk_bf16(a.z, a.w), pk_bf16(b.x, b.y), pk_bf16(b.z, b.w)};
  store8(j.C + (group * rows + row) * j.N, col, j.N, v, (j.N & 7) == 0 && ((uintptr_t)j.C & 15) == 0);
}

namespace {

int64_t moe_cap(int64_t P, int32_t E, int32_t B) {
  return (P + (int64_t)E * (B - 1) + B - 1) / B * B;
}

Div divisor(int32_t d) { return {(uint32_t)d, 0xFFFFFFFFu / (uint32_t)d}; }

int64_t tiles_of(int64_t M, int64_t N, int bm, int bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); }

// Buffer loads address an operand's rows with 32-bit byte offsets.
bool fits(int64_t elems) { return elems * 2 < (int64_t)kOOB; }

template <int MI, int NI, Group G, bool TA, bool TB, bool C8, bool WIDE = false>
hipError_t run_tile(Job j, hipStream_t st) {
  j.mt = (int)((j.M + 32 * MI - 1) / (32 * MI));
  j.nt = (int)((j.N + 32 * NI - 1) / (32 * NI));
  j.per = (int)(((int64_t)j.mt * j.nt + 7) / 8);
  j.by_band = divisor(8 * j.nt);
  j.by_per = divisor(j.per);
  j.by_splits = divisor(j.splits);
  int64_t mine;                                    // workgroups of an XCD
  if constexpr (G == kRows && workgroups_per_cu(MI, NI) == 1) {
    const Order o = order(j.mt, j.nt);
    mine = (int64_t)((o.groups + 7) / 8) * o.rows * o.cols;
  } else {
    mine = (int64_t)j.per * (G == kSums ? j.g.E : 1) * j.splits;
  }
  hipLaunchKernelGGL((k_bf16_tile<MI, NI, G, TA, TB, C8, WIDE>), dim3((unsigned)(8 * mine)), dim3(256), 0, st, j);
  return hipGetLastError();
}

template <Group G, bool C8>
hipError_t run_short(Job j, hipStream_t st) {
  const int tiles = (int)((j.N + 127) / 128);
  j.mt = (int)((j.M + 127) / 128);
  j.nt = (tiles + j.run - 1) / j.run;
  j.per = (int)(((int64_t)j.mt * j.nt + 7) / 8);
  j.by_band = divisor(j.nt);
  j.by_per = divisor(j.per);
  const int64_t mine = (int64_t)j.per * (G == kSums ? j.g.E : 1);
  hipLaunchKernelGGL((k_bf16_short<G, C8>), dim3((unsigned)(8 * mine)), dim3(256), 0, st, j);
  return hipGetLastError();
}

// The tiles and what they cost, in us: `fixed` and `step` (64 of the sum) for each
// tile of a CU that is kept busy, `latency` for tiles that have their CU to themselves;
// measured for products by rows (first) and for sums (second).  256 x 256 moves the
// least data and wins in long sums on full rounds of the CUs (4096 x 8 pairs over 64 of
// [4096, 2048]: 587 us, 801 in 128 x 128); 128 x 128 has two workgroups a CU, whose
// stores and first loads hide under each other's products (4096 x 5120 over 2050
// rows, 1.25 rounds of large tiles: 87 and 110; 512 x 4 pairs over 16 of [1024, 1024]:
// 14 and 28); the small ones are for few rows.
struct Kind {
  int bm, bn, occupancy;
  float fixed[2], step[2], latency[2], latency_step[2];
};
constexpr Kind kKinds[] = {
    {64, 64, 4, {1.1f, 1.2f}, {0.20f, 0.23f}, {2.2f, 2.3f}, {0.30f, 0.33f}},
    {64, 128, 3, {1.45f, 1.5f}, {0.33f, 0.38f}, {2.3f, 2.6f}, {0.33f, 0.37f}},
    {128, 128, 2, {2.3f, 2.1f}, {0.60f, 0.56f}, {3.6f, 3.8f}, {0.50f, 0.62f}},
    {256, 256, 1, {9.3f, 9.8f}, {1.45f, 1.58f}, {9.3f, 9.8f}, {1.45f, 1.58f}},
};
constexpr int kKindCount = 4;

// The estimates count the MI355X's compute units, whatever the current device has: a
// workspace is sized before the launch, perhaps with another device current, and both have
// to come to the same parts.
constexpr int64_t kCUs = 256;

float estimate(const Kind& t, int64_t tiles, float steps, bool sums) {
  const int64_t mine = (tiles + kCUs - 1) / kCUs;
  const int64_t waves = (mine + t.occupancy - 1) / t.occupancy;
  const float busy = (float)mine * (t.fixed[sums] + steps * t.step[sums]);
  const float alone = (float)waves * (t.latency[sums] + steps * t.latency_step[sums]);
  return 3.0f + std::max(busy, alone);
}

// k_bf16_short, in the same measure: a workgroup begins, then costs by tile and stage;
// a workgroup runs on when the others are done.  It wins below about 300 summed rows of
// large results (64 x [2816, 2048] over 256 pairs each: 396 us, 432 in 128 x 128 tiles;
// over 2050 x 6 pairs on 48 of [2808, 2064], the two are even and it loses 8%).
float estimate_short(int run, int64_t workgroups, float steps) {
  const int64_t mine = (workgroups + kCUs - 1) / kCUs, waves = (mine + 1) / 2;
  const float busy = ((float)mine + 0.25f) * (0.7f + (float)run * (1.1f + 0.65f * steps));
  const float alone = (float)waves * (3.2f + (float)run * (0.35f + 0.9f * steps));
  return 3.0f + std::max(busy, alone);
}

int64_t steps_of(int64_t sum) { return std::max((sum + 127) / 128 * 2, (int64_t)2); }

struct Choice {
  int kind, splits, run;   // run > 0: k_bf16_short, with that many tiles of a workgroup
};

// The kind that is done first, and in how many parts: few tiles of long sums are split
// between workgroups, whose fp32 sums a second launch joins (8192 rows into 64 x 64:
// 40 us whole, 15 in parts; one row of [4096, 4096]: 16 and 12).  groups sums of M x N
// results; B > 0: rows in blocks of B, the padding of an expert's last tile half full.
Choice choose(int64_t groups, int64_t M, int64_t N, int64_t sum, int32_t B, int32_t E, bool workspace) {
  Choice best = {0, 1, 0};
  float least = 0.0f;
  const int64_t steps = steps_of(sum);
  for (int splits = 1; splits <= (workspace ? 32 : 1); splits *= 2) {
    if (splits > 1 && steps < 4 * splits) break;
    const float join =
        splits == 1 ? 0.0f : 5.0f + (float)(groups * splits * M * N) * (8.0f / 4e6f);   // 4 TB/s
    for (int i = 0; i < kKindCount; ++i) {
      const Kind& t = kKinds[i];
      if ((B > 0 && B % t.bm != 0) || (splits > 1 && t.bm * t.bn > 128 * 128)) continue;
      int64_t high = (M + t.bm - 1) / t.bm;
      if (B > 0) {
        const int64_t used = std::min(M, (int64_t)E);
        high = std::max(used, high + used / 2);
      }
      const int64_t tiles = groups * splits * high * ((N + t.bn - 1) / t.bn);
      const int64_t part = (sum + splits - 1) / splits;
      const float mean = groups > 1 ? std::max((float)part / 64.0f + 1.0f, 2.0f) : (float)steps_of(part);
      const float us = join + estimate(t, tiles, mean, B == 0);
      if (least == 0.0f || us < least) {
        best = {i, splits, 0};
        least = us;
      }
    }
  }
  if (B == 0 && fits(M * N)) {
    const float stages = std::max(groups > 1 ? (float)sum / 64.0f + 0.5f : (float)((sum + 63) / 64), 1.0f);
    for (int run = 2; run <= 8; run *= 2) {
      const int64_t workgroups = groups * ((M + 127) / 128) * (((N + 127) / 128 + run - 1) / run);
      const float us = estimate_short(run, workgroups, stages);
      if (us < least) {
        best = {0, 1, run};
        least = us;
      }
    }
  }
  return best;
}

Choice choose_rows(const Bf16Plan& p, int64_t N, int64_t K, bool workspace) {
  return choose(1, p.P, N, K, p.B, p.E, workspace);
}
Choice choose_sums(int64_t groups, int64_t sum, int64_t M, int64_t N, bool workspace) {
  return choose(groups, M, N, sum, 0, 0, workspace);
}

// wide: operands of 2 GiB and more, whose tiles have 64-bit addresses (131142 x 8192
// by 1024 columns: rows 2680 us, weight gradient of 2 experts 2070, dense sums 2530; with
// 131000 rows, below 2 GiB: 1840 to 1970, 1760 and 2210).
template <Group G, bool TA, bool TB, bool C8 = false>
hipError_t run_kind(int kind, const Job& j, bool wide, hipStream_t st) {
  if (wide) {
    if (kind <= 1) return run_tile<2, 2, G, TA, TB, C8, true>(j, st);   // 64 x 128: few rows, not such operands
    return kind == 2 ? run_tile<4, 4, G, TA, TB, C8, true>(j, st) : run_tile<8, 8, G, TA, TB, C8, true>(j, st);
  }
  switch (kind) {
    case 0: return run_tile<2, 2, G, TA, TB, C8>(j, st);
    case 1: return run_tile<2, 4, G, TA, TB, C8>(j, st);
    case 2: return run_tile<4, 4, G, TA, TB, C8>(j, st);
    default: return run_tile<8, 8, G, TA, TB, C8>(j, st);
  }
}

Job job(const uint16_t* A, const Bf16Rows& B, uint16_t* C, int64_t M, int64_t N, int64_t K,
        const Bf16Plan& g, int32_t a_div, int32_t b_div, float* part) {
  Job j = {A, B, C, M, N, K, g, a_div, b_div, part, 1};
  j.by_a = divisor(a_div);
  j.by_b = divisor(b_div);
  j.by_block = divisor(std::max(g.B, 1));
  j.blocks = g.B == 0 ? 0 : (int)(moe_cap(g.P, g.E, g.B) / g.B);
  return j;
}

template <Group G>
hipError_t join(const Job& j, int64_t groups, int64_t rows, int64_t lines, hipStream_t st) {
  const int64_t pieces = groups * lines * ((j.N + 7) / 8);
  hipLaunchKernelGGL(k_bf16_join<G>, dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, st, j, rows,
                     pieces);
  return hipGetLastError();
}

template <Group G>
hipError_t run_sums(Job j, const Choice& c, int64_t rows_a, int64_t rows_b, hipStream_t st) {
  const bool wide = !fits(rows_a * j.M) || !fits(rows_b * j.N);
  const int kind = c.run > 0 ? 3 : c.kind;
  if (c.run > 0 && !wide) {
    j.run = c.run;
    return j.B.scales ? run_short<G, true>(j, st) : run_short<G, false>(j, st);
  }
  j.splits = c.splits;
  const hipError_t e = j.B.scales ? run_kind<G, true, true, true>(kind, j, wide, st)
                                  : run_kind<G, true, true>(kind, j, wide, st);
  return e != hipSuccess || j.splits == 1 ? e : join<G>(j, G == kSums ? j.g.E : 1, j.M, j.M, st);
}

}  // namespace

// (64 x 64 tiles are the most workgroups; parts are for few)
int64_t bf16_moe_threads(int64_t P, int32_t E, int64_t N, int64_t K, int32_t B) {
  return (tiles_of(moe_cap(P, E, B), N, 64, 64) + 8 * 32) * 256;
}
int64_t bf16_wgrad_threads(int32_t E, int64_t N, int64_t K) {
  return E * (tiles_of(N, K, 64, 64) + 8) * 256;
}

int64_t bf16_moe_workspace(int64_t P, int32_t E, int64_t N, int64_t K, int32_t B) {
  const int splits = choose(1, P, N, K, B, E, true).splits;
  return splits == 1 ? 0 : splits * P * ((N + 7) / 8 * 8);
}
int64_t bf16_sums_workspace(int64_t groups, int64_t sum, int64_t N, int64_t K) {
  const int splits = choose_sums(groups, sum, N, K, true).splits;
  return splits == 1 ? 0 : groups * splits * N * K;
}

namespace {
int32_t tile_of(const Choice& c) {
  return c.run > 0 ? 128 << 16 | 128 * c.run : kKinds[c.kind].bm << 16 | kKinds[c.kind].bn;
}
}  // namespace
int32_t bf16_moe_tile(int64_t P, int32_t E, int64_t N, int64_t K, int32_t B) {
  return tile_of(choose(1, P, N, K, B, E, true));
}
int32_t bf16_sums_tile(int64_t groups, int64_t sum, int64_t N, int64_t K) {
  return tile_of(choose_sums(groups, sum, N, K, true));
}

hipError_t launch_bf16_moe_gemm(const uint16_t* X, const uint16_t* W, uint16_t* Y,
                                const Bf16Plan& plan, int64_t N, int64_t K, int32_t div,
                                bool transposed, float* workspace, hipStream_t st) {
  Job j = job(X, {W, nullptr}, Y, moe_cap(plan.P, plan.E, plan.B), N, K, plan, div, 1, workspace);
  const bool wide = !fits(plan.P / div * K) || !fits(transposed ? N * K : std::min(N, (int64_t)256) * K);
  const Choice c = choose_rows(plan, N, K, workspace != nullptr);
  j.splits = c.splits;
  const hipError_t e = transposed ? run_kind<kRows, false, true>(c.kind, j, wide, st)
                                  : run_kind<kRows, false, false>(c.kind, j, wide, st);
  return e != hipSuccess || j.splits == 1 ? e : join<kRows>(j, 1, plan.P, j.M, st);
}

hipError_t launch_bf16_moe_wgrad(const uint16_t* dY, const Bf16Rows& X, uint16_t* dW,
                                 const Bf16Plan& plan, int64_t N, int64_t K, int32_t dy_div,
                                 int32_t x_div, float* workspace, hipStream_t st) {
  const Job j = job(dY, X, dW, N, K, 0, plan, dy_div, x_div, workspace);
  return run_sums<kSums>(j, choose_sums(plan.E, plan.P / plan.E, N, K, workspace != nullptr),
                         plan.P / dy_div, plan.P / x_div, st);
}

hipError_t launch_bf16_gemm_tn(const uint16_t* A, const Bf16Rows& B, uint16_t* C, int64_t M,
                               int64_t N, int64_t K, float* workspace, hipStream_t st) {
  const Job j = job(A, B, C, N, K, M, {}, 1, 1, workspace);
  return run_sums<kDense>(j, choose_sums(1, M, N, K, workspace != nullptr), M, M, st);
}

}  // namespace w4
