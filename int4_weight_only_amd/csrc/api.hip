// C ABI of libw4a16.so: argument validation and dispatch.
//
// Every entry point validates all of its arguments before enqueueing any
// work, so a nonzero status leaves the outputs untouched.  Nothing here
// allocates, synchronizes or reads device memory.
#include "w4a16.h"

#include "bf16.h"
#include "common.h"
#include "w8.h"

namespace {

thread_local int g_last_hip_error = 0;

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline int hip_status(hipError_t e) {
  if (e == hipSuccess) return W4_OK;
  g_last_hip_error = (int)e;
  return W4_ERR_HIP;
}

inline hipStream_t as_stream(void* s) { return (hipStream_t)s; }

constexpr int64_t kMaxI32 = 2147483647;

// The kernels address operands with 32-bit raw-buffer offsets and use
// offset 2^31 as "past the end" (reads zero): every buffer a kernel spans
// must stay below 2^31 bytes.
inline bool fits_buffer(int64_t bytes) { return bytes >= 0 && bytes < ((int64_t)1 << 31); }

// Decode path (M <= 32): per-workgroup weight buffers, X below 2^30 bytes.
inline bool use_decode(int64_t M, int64_t K) { return M <= 32 && K <= ((int64_t)1 << 24); }

// Tiled path: X [M, K] and the whole of Wq [N, K/8] in one buffer each,
// and a 1-D grid of tiles.
inline bool gemm_fits(int64_t M, int64_t N, int64_t K) {
  return fits_buffer(M * K * 2) && fits_buffer(N * (K / 2)) &&
         ((M + 127) / 128) * ((N + 255) / 256) < ((int64_t)1 << 31) - 8;
}

}  // namespace

namespace w4 {

// The launchers size their grids by it (decode tiles per workgroup, the
// bf16 product's tile shape).
int cu_count() {
  static int cus[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  if (cus[dev] == 0) {
    int v = 0;
    if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
        v <= 0)
      v = 256;
    cus[dev] = v;
  }
  return cus[dev];
}

}  // namespace w4

extern "C" {

const char* w4_status_string(int status) {
  switch (status) {
    case W4_OK: return "ok";
    case W4_ERR_NULL: return "null pointer";
    case W4_ERR_SHAPE: return "bad shape";
    case W4_ERR_MISALIGNED: return "misaligned pointer";
    case W4_ERR_UNSUPPORTED: return "unsupported arguments";
    case W4_ERR_HIP: return "HIP launch error";
    default: return "unknown status";
  }
}

int w4_last_hip_error(void) { return g_last_hip_error; }

const char* w4_version(void) { return "w4a16 gfx950 0.1"; }

int w4_quantize_pack(const uint16_t* W, int64_t N, int64_t K, int32_t* Wq, uint16_t* S,
                     void* stream) {
  if (N < 0 || K < 0 || K % 32 != 0) return W4_ERR_SHAPE;
  if (N == 0 || K == 0) return W4_OK;
  if (!W || !Wq || !S) return W4_ERR_NULL;
  if (!aligned(W, 16) || !aligned(Wq, 16) || !aligned(S, 2)) return W4_ERR_MISALIGNED;
  const int64_t words = N * (K / 8);
  if (words / (K / 8) != N || words > ((int64_t)1 << 38)) return W4_ERR_UNSUPPORTED;
  return hip_status(w4::launch_quantize(W, words, Wq, S, nullptr, nullptr, false, false,
                                        as_stream(stream)));
}

int w4_quantize_pack_asym(const uint16_t* W, int64_t N, int64_t K, int32_t* Wq, uint16_t* S,
                          uint8_t* Z, void* stream) {
  if (N < 0 || K < 0 || K % 32 != 0) return W4_ERR_SHAPE;
  if (N == 0 || K == 0) return W4_OK;
  if (!W || !Wq || !S || !Z) return W4_ERR_NULL;
  if (!aligned(W, 16) || !aligned(Wq, 16) || !aligned(S, 2)) return W4_ERR_MISALIGNED;
  const int64_t words = N * (K / 8);
  if (words / (K / 8) != N || words > ((int64_t)1 << 38)) return W4_ERR_UNSUPPORTED;
  return hip_status(w4::launch_quantize(W, words, Wq, S, Z, nullptr, false, true,
                                        as_stream(stream)));
}

int w4_fake_quant_asym(const uint16_t* W, int64_t N, int64_t K, uint16_t* W_fq, void* stream) {
  if (N < 0 || K < 0 || K % 32 != 0) return W4_ERR_SHAPE;
  if (N == 0 || K == 0) return W4_OK;
  if (!W || !W_fq) return W4_ERR_NULL;
  if (!aligned(W, 16) || !aligned(W_fq, 16)) return W4_ERR_MISALIGNED;
  const int64_t words = N * (K / 8);
  if (words / (K / 8) != N || words > ((int64_t)1 << 38)) return W4_ERR_UNSUPPORTED;
  const uintptr_t a = (uintptr_t)W, b = (uintptr_t)W_fq, len = (uintptr_t)(words * 16);
  if (a != b && a < b + len && b < a + len) return W4_ERR_UNSUPPORTED;
  return hip_status(w4::launch_quantize(W, words, nullptr, nullptr, nullptr, W_fq, true, true,
                                        as_stream(stream)));
}

int w4_fake_quant(const uint16_t* W, int64_t N, int64_t K, uint16_t* W_fq, void* stream) {
  if (N < 0 || K < 0 || K % 32 != 0) return W4_ERR_SHAPE;
  if (N == 0 || K == 0) return W4_OK;
  if (!W || !W_fq) return W4_ERR_NULL;
  if (!aligned(W, 16) || !aligned(W_fq, 16)) return W4_ERR_MISALIGNED;
  const int64_t words = N * (K / 8);
  if (words / (K / 8) != N || words > ((int64_t)1 << 38)) return W4_ERR_UNSUPPORTED;
  // in place is fine; partial overlap is not
  const uintptr_t a = (uintptr_t)W, b = (uintptr_t)W_fq, len = (uintptr_t)(words * 16);
  if (a != b && a < b + len && b < a + len) return W4_ERR_UNSUPPORTED;
  return hip_status(w4::launch_quantize(W, words, nullptr, nullptr, nullptr, W_fq, true, false,
                                        as_stream(stream)));
}

}  // extern "C"

namespace {

int dequant_checked(const int32_t* Wq, const uint16_t* S, const uint8_t* Z, bool asym, int64_t N,
                    int64_t K, uint16_t* W, void* stream) {
  if (N < 0 || K < 0 || K % 32 != 0) return W4_ERR_SHAPE;
  if (N == 0 || K == 0) return W4_OK;
  if (!Wq || !S || !W || (asym && !Z)) return W4_ERR_NULL;
  if (!aligned(Wq, 4) || !aligned(S, 2) || !aligned(W, 16)) return W4_ERR_MISALIGNED;
  const int64_t words = N * (K / 8);
  if (words / (K / 8) != N || words > ((int64_t)1 << 38)) return W4_ERR_UNSUPPORTED;
  return hip_status(w4::launch_dequant(Wq, S, asym ? Z : nullptr, W, words, as_stream(stream)));
}

}  // namespace

extern "C" {

int w4_dequant(const int32_t* Wq, const uint16_t* S, int64_t N, int64_t K, uint16_t* W,
               void* stream) {
  return dequant_checked(Wq, S, nullptr, false, N, K, W, stream);
}

int w4_dequant_asym(const int32_t* Wq, const uint16_t* S, const uint8_t* Z, int64_t N, int64_t K,
                    uint16_t* W, void* stream) {
  return dequant_checked(Wq, S, Z, true, N, K, W, stream);
}

int w4a16_gemm(const uint16_t* X, const int32_t* Wq, const uint16_t* S, uint16_t* Y, int64_t M,
               int64_t N, int64_t K, void* stream) {
  if (M < 0 || N < 0 || K < 0 || K % 32 != 0) return W4_ERR_SHAPE;
  if (M == 0 || N == 0) return W4_OK;
  if (!Y) return W4_ERR_NULL;
  if (!aligned(Y, 4)) return W4_ERR_MISALIGNED;
  if (M > kMaxI32 || N > kMaxI32 || K > kMaxI32 || M * N > ((int64_t)1 << 40) ||
      N * (K / 8) > ((int64_t)1 << 40))
    return W4_ERR_UNSUPPORTED;
  if (K == 0) return hip_status(w4::launch_zero_bf16(Y, M * N, as_stream(stream)));
  if (!X || !Wq || !S) return W4_ERR_NULL;
  if (!aligned(X, 16) || !aligned(Wq, 16) || !aligned(S, 2)) return W4_ERR_MISALIGNED;
  if (use_decode(M, K))
    return hip_status(w4::launch_gemv(X, Wq, S, Y, M, N, K, as_stream(stream)));
  if (!gemm_fits(M, N, K)) return W4_ERR_UNSUPPORTED;
  return hip_status(w4::launch_gemm(X, Wq, S, Y, M, N, K, as_stream(stream)));
}

int w4a16_gemm_asym(const uint16_t* X, const int32_t* Wq, const uint16_t* S, const uint8_t* Z,
                    uint16_t* Y, int64_t M, int64_t N, int64_t K, void* stream) {
  if (M < 0 || N < 0 || K < 0 || K % 32 != 0) return W4_ERR_SHAPE;
  if (M == 0 || N == 0) return W4_OK;
  if (!Y) return W4_ERR_NULL;
  if (!aligned(Y, 4)) return W4_ERR_MISALIGNED;
  if (M > kMaxI32 || N > kMaxI32 || K > kMaxI32 || M * N > ((int64_t)1 << 40) ||
      N * (K / 8) > ((int64_t)1 << 40))
    return W4_ERR_UNSUPPORTED;
  if (!use_decode(M, K) && !gemm_fits(M, N, K)) return W4_ERR_UNSUPPORTED;
  if (K == 0) return hip_status(w4::launch_zero_bf16(Y, M * N, as_stream(stream)));
  if (!X || !Wq || !S || !Z) return W4_ERR_NULL;
  if (!aligned(X, 16) || !aligned(Wq, 16) || !aligned(S, 2)) return W4_ERR_MISALIGNED;
  if (use_decode(M, K))
    return hip_status(w4::launch_gemv_zp(X, Wq, S, Z, Y, M, N, K, as_stream(stream)));
  return hip_status(w4::launch_gemm_zp(X, Wq, S, Z, Y, M, N, K, as_stream(stream)));
}

int64_t w4_repacked_words(int64_t N, int64_t K) {
  if (N < 0 || K < 0 || K % 32 != 0 || N > kMaxI32 || K > kMaxI32) return -1;
  return w4::tiled_words(N, K);
}

namespace {
int relayout_checked(const int32_t* src, int32_t* dst, int64_t E, int64_t N, int64_t K,
                     bool restore, void* stream) {
  if (E < 0 || N < 0 || K < 0 || K % 32 != 0) return W4_ERR_SHAPE;
  if (E == 0 || N == 0 || K == 0) return W4_OK;
  if (N > kMaxI32 || K > kMaxI32 || E * w4::tiled_words(N, K) > ((int64_t)1 << 40))
    return W4_ERR_UNSUPPORTED;
  if (!src || !dst) return W4_ERR_NULL;
  if (!aligned(src, 16) || !aligned(dst, 16)) return W4_ERR_MISALIGNED;
  // the two buffers must not overlap
  const uintptr_t a = (uintptr_t)src, b = (uintptr_t)dst;
  const uintptr_t la = (uintptr_t)(restore ? E * w4::tiled_words(N, K) : E * N * (K / 8)) * 4;
  const uintptr_t lb = (uintptr_t)(restore ? E * N * (K / 8) : E * w4::tiled_words(N, K)) * 4;
  if (a < b + lb && b < a + la) return W4_ERR_UNSUPPORTED;
  return hip_status(w4::launch_relayout(src, dst, E, N, K, restore, as_stream(stream)));
}
}  // namespace

int w4_repack(const int32_t* Wq, int64_t E, int64_t N, int64_t K, int32_t* Wt, void* stream) {
  return relayout_checked(Wq, Wt, E, N, K, false, stream);
}

int w4_restore(const int32_t* Wt, int64_t E, int64_t N, int64_t K, int32_t* Wq, void* stream) {
  return relayout_checked(Wt, Wq, E, N, K, true, stream);
}

int64_t w4_repacked_group_elems(int64_t N, int64_t K) {
  if (N < 0 || K < 0 || K % 32 != 0 || N > kMaxI32 || K > kMaxI32) return -1;
  return w4::tiled_group_elems(N, K);
}

namespace {
int relayout_groups_checked(const void* src, void* dst, int32_t elem_bytes, int64_t E, int64_t N,
                            int64_t K, bool restore, void* stream) {
  if (E < 0 || N < 0 || K < 0 || K % 32 != 0) return W4_ERR_SHAPE;
  if (elem_bytes != 1 && elem_bytes != 2) return W4_ERR_UNSUPPORTED;
  if (E == 0 || N == 0 || K == 0) return W4_OK;
  if (N > kMaxI32 || K > kMaxI32 || E * w4::tiled_group_elems(N, K) > ((int64_t)1 << 40))
    return W4_ERR_UNSUPPORTED;
  if (!src || !dst) return W4_ERR_NULL;
  if (!aligned(src, elem_bytes) || !aligned(dst, elem_bytes)) return W4_ERR_MISALIGNED;
  const uintptr_t a = (uintptr_t)src, b = (uintptr_t)dst;
  const int64_t tiled = E * w4::tiled_group_elems(N, K), canon = E * N * (K / 32);
  const uintptr_t la = (uintptr_t)(restore ? tiled : canon) * elem_bytes;
  const uintptr_t lb = (uintptr_t)(restore ? canon : tiled) * elem_bytes;
  if (a < b + lb && b < a + la) return W4_ERR_UNSUPPORTED;
  return hip_status(
      w4::launch_relayout_groups(src, dst, elem_bytes, E, N, K, restore, as_stream(stream)));
}
}  // namespace

int w4_repack_groups(const void* A, int32_t elem_bytes, int64_t E, int64_t N, int64_t K, void* At,
                     void* stream) {
  return relayout_groups_checked(A, At, elem_bytes, E, N, K, false, stream);
}

int w4_restore_groups(const void* At, int32_t elem_bytes, int64_t E, int64_t N, int64_t K, void* A,
                      void* stream) {
  return relayout_groups_checked(At, A, elem_bytes, E, N, K, true, stream);
}

int w4a16_gemm_tiled(const uint16_t* X, const int32_t* Wt, const uint16_t* S, const uint8_t* Z,
                     uint16_t* Y, int64_t M, int64_t N, int64_t K, void* stream) {
  if (M < 0 || N < 0 || K < 0 || K % 32 != 0) return W4_ERR_SHAPE;
  if (M == 0 || N == 0) return W4_OK;
  if (!Y) return W4_ERR_NULL;
  if (!aligned(Y, 4)) return W4_ERR_MISALIGNED;
  if (M > kMaxI32 || N > kMaxI32 || K > kMaxI32 || M * N > ((int64_t)1 << 40) ||
      N * (K / 8) > ((int64_t)1 << 40))
    return W4_ERR_UNSUPPORTED;
  const bool decode = use_decode(M, K);
  if (!decode && !(fits_buffer(M * K * 2) && fits_buffer(w4::tiled_words(N, K) * 4) &&
                   ((M + 127) / 128) * ((N + 255) / 256) < ((int64_t)1 << 31) - 8))
    return W4_ERR_UNSUPPORTED;
  if (K == 0) return hip_status(w4::launch_zero_bf16(Y, M * N, as_stream(stream)));
  if (!X || !Wt || !S) return W4_ERR_NULL;
  if (!aligned(X, 16) || !aligned(Wt, 16) || !aligned(S, 2)) return W4_ERR_MISALIGNED;
  if (decode)
    return hip_status(w4::launch_gemv_any(X, Wt, S, Z, Y, M, N, K, true, as_stream(stream)));
  return hip_status(w4::launch_gemm_any(X, Wt, S, Z, Y, M, N, K, true, as_stream(stream)));
}

int w4_dequant_t(const int32_t* Wq, const uint16_t* S, const uint8_t* Z, int64_t N, int64_t K,
                 uint16_t* WT, void* stream) {
  if (N < 0 || K < 0 || K % 32 != 0) return W4_ERR_SHAPE;
  if (N == 0 || K == 0) return W4_OK;
  if (!Wq || !S || !WT) return W4_ERR_NULL;
  if (!aligned(Wq, 4) || !aligned(S, 2) || !aligned(WT, 16)) return W4_ERR_MISALIGNED;
  if (N > kMaxI32 || K > kMaxI32 || N * K > ((int64_t)1 << 40) ||
      ((N + 63) / 64) * ((K + 127) / 128) >= kMaxI32)
    return W4_ERR_UNSUPPORTED;
  return hip_status(w4::launch_dequant_t(Wq, S, Z, WT, N, K, as_stream(stream)));
}

int w4_bf16_gemm_nt(const uint16_t* A, const uint16_t* B, uint16_t* C, int64_t M, int64_t N,
                    int64_t K, void* stream) {
  if (M < 0 || N < 0 || K < 0 || K % 8 != 0) return W4_ERR_SHAPE;
  if (M == 0 || N == 0) return W4_OK;
  if (!C) return W4_ERR_NULL;
  if (!aligned(C, 2)) return W4_ERR_MISALIGNED;
  if (((M + 127) / 128) * ((N + 127) / 128) >= kMaxI32 || M * N > ((int64_t)1 << 40))
    return W4_ERR_UNSUPPORTED;
  if (K == 0) return hip_status(w4::launch_zero_bf16(C, M * N, as_stream(stream)));
  // 256 rows of an operand are one buffer
  if (M > kMaxI32 - 256 || N > kMaxI32 - 256 || K > kMaxI32 - 256 ||
      !fits_buffer((M < 256 ? M : 256) * K * 2) || !fits_buffer((N < 256 ? N : 256) * K * 2))
    return W4_ERR_UNSUPPORTED;
  if (!A || !B) return W4_ERR_NULL;
  if (!aligned(A, 16) || !aligned(B, 16)) return W4_ERR_MISALIGNED;
  return hip_status(w4::launch_bf16_gemm_nt(A, B, C, M, N, K, as_stream(stream)));
}

int w4_bf16_transpose(const uint16_t* A, int64_t R, int64_t C, int64_t RP, uint16_t* AT,
                      void* stream) {
  if (R < 0 || C < 0 || RP < R) return W4_ERR_SHAPE;
  if (RP == 0 || C == 0) return W4_OK;
  if (!AT || (R > 0 && !A)) return W4_ERR_NULL;
  if (!aligned(A, 2) || !aligned(AT, 2)) return W4_ERR_MISALIGNED;
  if (R > ((int64_t)1 << 40) / (C > 0 ? C : 1) || RP > ((int64_t)1 << 40) / C ||
      ((RP + 63) / 64) * ((C + 63) / 64) >= kMaxI32)
    return W4_ERR_UNSUPPORTED;
  const uintptr_t a = (uintptr_t)A, b = (uintptr_t)AT;
  const uintptr_t la = (uintptr_t)(R * C) * 2u, lb = (uintptr_t)(RP * C) * 2u;
  if (R > 0 && a < b + lb && b < a + la) return W4_ERR_UNSUPPORTED;   // overlapping buffers
  return hip_status(w4::launch_transpose_bf16(A, AT, R, C, RP, as_stream(stream)));
}

int32_t w4_pick_block_size(int64_t T, int32_t k, int32_t E) {
  if (T < 0 || k < 1 || E < 1) return 0;
  const int64_t mean = (T * k + E - 1) / E;
  int64_t p = 1;
  while (p < mean) p *= 2;
  if (p < 16) p = 16;
  if (p > 64) p = 64;
  return (int32_t)p;
}

int64_t w4_moe_align_capacity(int64_t T, int32_t k, int32_t E, int32_t B) {
  if (T < 0 || k < 1 || E < 1 || B < 1) return -1;
  const int64_t n = T * k + (int64_t)E * (B - 1);
  return ((n + B - 1) / B) * B;
}

int moe_align_block_size(const int32_t* topk_ids, int64_t T, int32_t k, int32_t E, int32_t B,
                         int32_t* sorted_token_ids, int32_t* expert_ids,
                         int32_t* num_tokens_post_padded, void* stream) {
  if (T < 0 || k < 1 || E < 1 || B < 1) return W4_ERR_SHAPE;
  if (E > 1024 || B > 1024) return W4_ERR_UNSUPPORTED;
  if (T * k + (int64_t)E * B >= kMaxI32) return W4_ERR_UNSUPPORTED;
  if (!sorted_token_ids || !expert_ids || !num_tokens_post_padded) return W4_ERR_NULL;
  if (T > 0 && !topk_ids) return W4_ERR_NULL;
  if (!aligned(topk_ids, 4) || !aligned(sorted_token_ids, 4) || !aligned(expert_ids, 4) ||
      !aligned(num_tokens_post_padded, 4))
    return W4_ERR_MISALIGNED;
  const int64_t cap = w4_moe_align_capacity(T, k, E, B);
  return hip_status(w4::launch_align(topk_ids, T, k, E, B, cap, sorted_token_ids, expert_ids,
                                     num_tokens_post_padded, as_stream(stream)));
}

}  // extern "C"

namespace {

// Shared validation and dispatch of the grouped products (Z == nullptr:
// symmetric codes).  N is the weight rows per expert (2I with the SwiGLU).
// Checks shared by the grouped products; W4_OK, or -1 for a valid call with
// nothing to do (T == 0), or an error status.
int moe_gemm_validate(const uint16_t* X, const int32_t* Wq, const uint16_t* S, const uint8_t* Z,
                      bool asym, const int32_t* sorted_token_ids, const int32_t* expert_ids,
                      const int32_t* num_tokens_post_padded, const float* topk_weights,
                      uint16_t* Y, int64_t T, int32_t k, int32_t E, int64_t N, int64_t K,
                      int32_t B, int32_t x_row_div, bool swiglu, bool tiled) {
  if (T < 0 || k < 1 || E < 1 || N < 1 || K < 32 || K % 32 != 0 || B < 1) return W4_ERR_SHAPE;
  if (x_row_div != 1 && x_row_div != k) return W4_ERR_SHAPE;
  if (B > 1024 || E > 1024) return W4_ERR_UNSUPPORTED;
  if (T * k + (int64_t)E * B >= kMaxI32 || N > kMaxI32 || K > kMaxI32 ||
      (int64_t)E * N * (K / 8) > ((int64_t)1 << 40) || T * k * N > ((int64_t)1 << 40))
    return W4_ERR_UNSUPPORTED;
  // one buffer spans X's rows, one an expert's Wq
  if (!fits_buffer((T * k / x_row_div) * K * 2) ||
      !fits_buffer(tiled ? w4::tiled_words(N, K) * 4 : N * (K / 2)))
    return W4_ERR_UNSUPPORTED;
  if (T == 0) return -1;
  if (!X || !Wq || !S || !sorted_token_ids || !expert_ids || !num_tokens_post_padded || !Y ||
      (asym && !Z))
    return W4_ERR_NULL;
  if (!aligned(X, 16) || !aligned(Wq, 16) || !aligned(S, 2) || !aligned(Y, 4) ||
      !aligned(sorted_token_ids, 4) || !aligned(expert_ids, 4) ||
      !aligned(num_tokens_post_padded, 4) || !aligned(topk_weights, 4))
    return W4_ERR_MISALIGNED;
  if (w4::moe_gemm_workgroups(T, k, E, N, B, swiglu) >= kMaxI32) return W4_ERR_UNSUPPORTED;
  return W4_OK;
}

// Shared validation and dispatch of the grouped products (Z == nullptr:
// symmetric codes).  N is the weight rows per expert (2I with the SwiGLU).
int moe_gemm_checked(const uint16_t* X, const int32_t* Wq, const uint16_t* S, const uint8_t* Z,
                     bool asym, const int32_t* sorted_token_ids, const int32_t* expert_ids,
                     const int32_t* num_tokens_post_padded, const float* topk_weights,
                     uint16_t* Y, int64_t T, int32_t k, int32_t E, int64_t N, int64_t K,
                     int32_t B, int32_t x_row_div, bool swiglu, bool tiled, void* stream) {
  const int v = moe_gemm_validate(X, Wq, S, Z, asym, sorted_token_ids, expert_ids,
                                  num_tokens_post_padded, topk_weights, Y, T, k, E, N, K, B,
                                  x_row_div, swiglu, tiled);
  if (v != W4_OK) return v < 0 ? W4_OK : v;
  if (swiglu)
    return hip_status(w4::launch_moe_gemm_swiglu(X, Wq, S, asym ? Z : nullptr, sorted_token_ids,
                                                 expert_ids, num_tokens_post_padded, Y, T, k, E,
                                                 N / 2, K, B, x_row_div, tiled,
                                                 as_stream(stream)));
  return hip_status(w4::launch_moe_gemm(X, Wq, S, asym ? Z : nullptr, sorted_token_ids,
                                        expert_ids, num_tokens_post_padded, topk_weights, Y, T,
                                        k, E, N, K, B, x_row_div, tiled, as_stream(stream)));
}

}  // namespace

extern "C" {

int w4a16_moe_gemm(const uint16_t* X, const int32_t* Wq, const uint16_t* S,
                   const int32_t* sorted_token_ids, const int32_t* expert_ids,
                   const int32_t* num_tokens_post_padded, const float* topk_weights, uint16_t* Y,
                   int64_t T, int32_t k, int32_t E, int64_t N, int64_t K, int32_t B,
                   int32_t x_row_div, void* stream) {
  return moe_gemm_checked(X, Wq, S, nullptr, false, sorted_token_ids, expert_ids,
                          num_tokens_post_padded, topk_weights, Y, T, k, E, N, K, B, x_row_div,
                          false, false, stream);
}

int w4a16_moe_gemm_asym(const uint16_t* X, const int32_t* Wq, const uint16_t* S, const uint8_t* Z,
                        const int32_t* sorted_token_ids, const int32_t* expert_ids,
                        const int32_t* num_tokens_post_padded, const float* topk_weights,
                        uint16_t* Y, int64_t T, int32_t k, int32_t E, int64_t N, int64_t K,
                        int32_t B, int32_t x_row_div, void* stream) {
  return moe_gemm_checked(X, Wq, S, Z, true, sorted_token_ids, expert_ids,
                          num_tokens_post_padded, topk_weights, Y, T, k, E, N, K, B, x_row_div,
                          false, false, stream);
}

int w4a16_moe_gemm_swiglu(const uint16_t* X, const int32_t* Wq, const uint16_t* S,
                          const int32_t* sorted_token_ids, const int32_t* expert_ids,
                          const int32_t* num_tokens_post_padded, uint16_t* A, int64_t T,
                          int32_t k, int32_t E, int64_t I, int64_t K, int32_t B,
                          int32_t x_row_div, void* stream) {
  if (I < 1) return W4_ERR_SHAPE;
  const int64_t N = I > kMaxI32 ? kMaxI32 + 1 : 2 * I;   // past the limit: unsupported
  return moe_gemm_checked(X, Wq, S, nullptr, false, sorted_token_ids, expert_ids,
                          num_tokens_post_padded, nullptr, A, T, k, E, N, K, B, x_row_div,
                          true, false, stream);
}

int w4a16_moe_gemm_swiglu_asym(const uint16_t* X, const int32_t* Wq, const uint16_t* S,
                               const uint8_t* Z, const int32_t* sorted_token_ids,
                               const int32_t* expert_ids, const int32_t* num_tokens_post_padded,
                               uint16_t* A, int64_t T, int32_t k, int32_t E, int64_t I, int64_t K,
                               int32_t B, int32_t x_row_div, void* stream) {
  if (I < 1) return W4_ERR_SHAPE;
  const int64_t N = I > kMaxI32 ? kMaxI32 + 1 : 2 * I;   // past the limit: unsupported
  return moe_gemm_checked(X, Wq, S, Z, true, sorted_token_ids, expert_ids,
                          num_tokens_post_padded, nullptr, A, T, k, E, N, K, B, x_row_div,
                          true, false, stream);
}

int w4a16_moe_gemm_tiled(const uint16_t* X, const int32_t* Wt, const uint16_t* S,
                         const uint8_t* Z, const int32_t* sorted_token_ids,
                         const int32_t* expert_ids, const int32_t* num_tokens_post_padded,
                         const float* topk_weights, uint16_t* Y, int64_t T, int32_t k, int32_t E,
                         int64_t N, int64_t K, int32_t B, int32_t x_row_div, void* stream) {
  return moe_gemm_checked(X, Wt, S, Z, Z != nullptr, sorted_token_ids, expert_ids,
                          num_tokens_post_padded, topk_weights, Y, T, k, E, N, K, B, x_row_div,
                          false, true, stream);
}

int w4a16_moe_gemm_swiglu_tiled(const uint16_t* X, const int32_t* Wt, const uint16_t* S,
                                const uint8_t* Z, const int32_t* sorted_token_ids,
                                const int32_t* expert_ids,
                                const int32_t* num_tokens_post_padded, uint16_t* A, int64_t T,
                                int32_t k, int32_t E, int64_t I, int64_t K, int32_t B,
                                int32_t x_row_div, void* stream) {
  if (I < 1) return W4_ERR_SHAPE;
  const int64_t N = I > kMaxI32 ? kMaxI32 + 1 : 2 * I;   // past the limit: unsupported
  return moe_gemm_checked(X, Wt, S, Z, Z != nullptr, sorted_token_ids, expert_ids,
                          num_tokens_post_padded, nullptr, A, T, k, E, N, K, B, x_row_div,
                          true, true, stream);
}

int w4_silu_mul(const uint16_t* H1, uint16_t* A, int64_t R, int64_t I, void* stream) {
  if (R < 0 || I < 0 || I % 2 != 0) return W4_ERR_SHAPE;
  if (R == 0 || I == 0) return W4_OK;
  if (!H1 || !A) return W4_ERR_NULL;
  if (!aligned(H1, 4) || !aligned(A, 4)) return W4_ERR_MISALIGNED;
  return hip_status(w4::launch_silu_mul(H1, A, R, I, as_stream(stream)));
}

int w4_moe_sum(const uint16_t* H2, const float* topk_weights, uint16_t* Out, int64_t T, int32_t k,
               int64_t H, void* stream) {
  if (T < 0 || k < 1 || H < 0 || H % 2 != 0) return W4_ERR_SHAPE;
  if (T == 0 || H == 0) return W4_OK;
  if (!H2 || !Out) return W4_ERR_NULL;
  if (!aligned(H2, 4) || !aligned(Out, 4) || !aligned(topk_weights, 4)) return W4_ERR_MISALIGNED;
  return hip_status(w4::launch_moe_sum(H2, topk_weights, Out, T, k, H, as_stream(stream)));
}

int w4_moe_route(const float* logits, int64_t T, int32_t E, int32_t k, int32_t* topk_ids,
                 float* topk_weights, void* stream) {
  if (T < 0 || E < 1 || k < 1) return W4_ERR_SHAPE;
  if (E > 1024 || k > 16 || k > E || T > kMaxI32) return W4_ERR_UNSUPPORTED;
  if (T == 0) return W4_OK;
  if (!logits || !topk_ids || !topk_weights) return W4_ERR_NULL;
  if (!aligned(logits, 4) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4))
    return W4_ERR_MISALIGNED;
  return hip_status(w4::launch_route(logits, T, E, k, topk_ids, topk_weights, as_stream(stream)));
}

int64_t w4_moe_combine_workspace_words(int64_t T, int32_t k, int32_t E, int64_t N, int32_t B) {
  if (T < 0 || k < 1 || E < 1 || N < 1 || B < 1) return -1;
  return w4::moe_combine_counters(T, k, E, N, B);
}

}  // extern "C"

namespace {

// Checks of the fused combine's operands other than the counters: W4_OK,
// -1 for a valid call with nothing to do (T == 0), or an error status.
int combine_validate(const uint16_t* A, const int32_t* Wq, const uint16_t* S,
                     const int32_t* sorted_token_ids, const int32_t* expert_ids,
                     const int32_t* num_tokens_post_padded, const int32_t* topk_ids,
                     const float* topk_weights, uint16_t* H2, uint16_t* Out, int64_t T,
                     int32_t k, int32_t E, int64_t N, int64_t K, int32_t B, int32_t tiled) {
  const int v = moe_gemm_validate(A, Wq, S, nullptr, false, sorted_token_ids, expert_ids,
                                  num_tokens_post_padded, topk_weights, H2, T, k, E, N, K, B, 1,
                                  false, tiled != 0);
  if (v != W4_OK) return v;
  if (T * N >= ((int64_t)1 << 40) || k > 16) return W4_ERR_UNSUPPORTED;
  if (!topk_ids || !topk_weights || !Out) return W4_ERR_NULL;
  if (!aligned(topk_ids, 4) || !aligned(Out, 2)) return W4_ERR_MISALIGNED;
  return W4_OK;
}

}  // namespace

extern "C" {

int w4a16_moe_gemm_combine(const uint16_t* A, const int32_t* Wq, const uint16_t* S,
                           const int32_t* sorted_token_ids, const int32_t* expert_ids,
                           const int32_t* num_tokens_post_padded, const int32_t* topk_ids,
                           const float* topk_weights, uint16_t* H2, uint16_t* Out, int64_t T,
                           int32_t k, int32_t E, int64_t N, int64_t K, int32_t B, int32_t tiled,
                           int32_t* workspace, void* stream) {
  const int v = combine_validate(A, Wq, S, sorted_token_ids, expert_ids, num_tokens_post_padded,
                                 topk_ids, topk_weights, H2, Out, T, k, E, N, K, B, tiled);
  if (v < 0) return W4_OK;
  if (v != W4_OK) return v;
  if (!workspace) return W4_ERR_NULL;
  if (!aligned(workspace, 4)) return W4_ERR_MISALIGNED;
  return hip_status(w4::launch_moe_gemm_combine(A, Wq, S, sorted_token_ids, expert_ids,
                                                num_tokens_post_padded, topk_ids, topk_weights,
                                                H2, Out, workspace, T, k, E, N, K, B, tiled != 0,
                                                as_stream(stream)));
}

int w4a16_moe_gemm_combine_noalloc(const uint16_t* A, const int32_t* Wq, const uint16_t* S,
                                   const int32_t* sorted_token_ids, const int32_t* expert_ids,
                                   const int32_t* num_tokens_post_padded,
                                   const int32_t* topk_ids, const float* topk_weights,
                                   uint16_t* H2, uint16_t* Out, int64_t T, int32_t k, int32_t E,
                                   int64_t N, int64_t K, int32_t B, int32_t tiled,
                                   void* stream) {
  const int v = combine_validate(A, Wq, S, sorted_token_ids, expert_ids, num_tokens_post_padded,
                                 topk_ids, topk_weights, H2, Out, T, k, E, N, K, B, tiled);
  if (v < 0) return W4_OK;
  if (v != W4_OK) return v;
  if (w4::moe_combine_counters(T, k, E, N, B) > w4::kCombineScratchWords)
    return W4_ERR_UNSUPPORTED;
  int32_t* words = nullptr;
  const hipError_t e = w4::combine_scratch(&words);
  if (e != hipSuccess) return hip_status(e);
  return hip_status(w4::launch_moe_gemm_combine(A, Wq, S, sorted_token_ids, expert_ids,
                                                num_tokens_post_padded, topk_ids, topk_weights,
                                                H2, Out, words, T, k, E, N, K, B, tiled != 0,
                                                as_stream(stream)));
}

}  // extern "C"

// ------------------------------------------------ W8A8 and the scored router --

namespace {

constexpr int64_t kMaxElems = (int64_t)1 << 40;
constexpr int64_t kMaxGrid = (int64_t)1 << 32;      // threads of one launch

constexpr int64_t kMaxTokens = (int64_t)1 << 25;    // one wave each

// Sizes of an e4m3 operand [R, K]: K in whole 16-byte pieces.
int w8_shape(int64_t R, int64_t K) {
  if (R < 0 || K < 0 || K % 16 != 0) return W4_ERR_SHAPE;
  if (K > w4::kW8MaxK || R > kMaxI32 || R * K > kMaxElems) return W4_ERR_UNSUPPORTED;
  return W4_OK;
}

// Checks shared by the grouped products (Y: their output, of that alignment);
// W4_OK, -1 for a valid call with nothing to do (T == 0), or an error status.
int w8_moe_validate(const uint8_t* X8, const uint8_t* SX, const uint8_t* W8, const uint8_t* SW,
                    const int32_t* sorted_token_ids, const int32_t* expert_ids,
                    const int32_t* num_tokens_post_padded, const void* Y, uintptr_t align,
                    int64_t T, int32_t k, int32_t E, int64_t N, int64_t K, int32_t B,
                    int32_t x_row_div) {
  if (T < 0 || k < 1 || E < 1 || N < 1 || K < 16 || K % 16 != 0 || B < 16 || B % 16 != 0)
    return W4_ERR_SHAPE;
  if (x_row_div != 1 && x_row_div != k) return W4_ERR_SHAPE;
  if (B > 1024 || E > 1024 || T > kMaxI32 || N > kMaxI32 || K > w4::kW8MaxK ||
      T * k + (int64_t)E * B >= kMaxI32 || T * k * N > kMaxElems || N * K > kMaxElems ||
      E * (N * K) > kMaxElems)
    return W4_ERR_UNSUPPORTED;
  if (w4::w8_moe_threads(T, k, E, N, K, B, x_row_div) >= kMaxGrid) return W4_ERR_UNSUPPORTED;
  if (T == 0) return -1;
  if (!X8 || !SX || !W8 || !SW || !sorted_token_ids || !expert_ids || !num_tokens_post_padded || !Y)
    return W4_ERR_NULL;
  if (!aligned(X8, 16) || !aligned(W8, 16) || !aligned(SX, 4) || !aligned(SW, 4) ||
      !aligned(Y, align) || !aligned(sorted_token_ids, 4) || !aligned(expert_ids, 4) ||
      !aligned(num_tokens_post_padded, 4))
    return W4_ERR_MISALIGNED;
  return W4_OK;
}

int route_rule(int32_t E, int32_t k, int32_t groups, int32_t topk_groups, int32_t group_top) {
  if (E < 1 || k < 1 || groups < 1 || topk_groups < 1 || topk_groups > groups || E % groups != 0)
    return W4_ERR_SHAPE;
  if (group_top != 1 && group_top != 2) return W4_ERR_SHAPE;
  if (E > 1024 || k > 16 || k > E || groups > 64 || (int64_t)topk_groups * (E / groups) < k)
    return W4_ERR_UNSUPPORTED;
  return W4_OK;
}

}  // namespace

extern "C" {

int64_t w8_scale_cols(int64_t K) { return K < 0 ? -1 : w4::w8_cols(K); }

int w8_quantize_rows(const uint16_t* X, int64_t M, int64_t K, uint8_t* X8, uint8_t* SX,
                     void* stream) {
  const int v = w8_shape(M, K);
  if (v != W4_OK) return v;
  if (M == 0 || K == 0) return W4_OK;
  if (!X || !X8 || !SX) return W4_ERR_NULL;
  if (!aligned(X, 16) || !aligned(X8, 16) || !aligned(SX, 4)) return W4_ERR_MISALIGNED;
  return hip_status(w4::launch_w8_quantize_rows(X, M, K, X8, SX, as_stream(stream)));
}

int w8_quantize_blocks(const uint16_t* W, int64_t N, int64_t K, uint8_t* W8, uint8_t* SW,
                       uint8_t* WT8, uint8_t* ST, void* stream) {
  const int v = w8_shape(N, K);
  if (v != W4_OK) return v;
  if (N == 0 || K == 0) return W4_OK;
  if (!W || !W8 || !SW || (WT8 != nullptr) != (ST != nullptr)) return W4_ERR_NULL;
  if (WT8) {
    const int u = w8_shape(K, N);
    if (u != W4_OK) return u;
  }
  if (w4::w8_cols(K) * (w4::w8_blocks(N) + 3) * 256 >= kMaxGrid) return W4_ERR_UNSUPPORTED;
  if (!aligned(W, 16) || !aligned(W8, 16) || !aligned(SW, 4) || !aligned(WT8, 16) ||
      !aligned(ST, 4))
    return W4_ERR_MISALIGNED;
  return hip_status(w4::launch_w8_quantize_blocks(W, N, K, W8, SW, WT8, ST, as_stream(stream)));
}

int w8_silu_mul_quantize(const uint16_t* H1, int64_t R, int64_t I, uint8_t* A8, uint8_t* SA,
                         void* stream) {
  const int v = w8_shape(R, I);
  if (v != W4_OK) return v;
  if (R == 0 || I == 0) return W4_OK;
  if (!H1 || !A8 || !SA) return W4_ERR_NULL;
  if (!aligned(H1, 16) || !aligned(A8, 16) || !aligned(SA, 4)) return W4_ERR_MISALIGNED;
  return hip_status(w4::launch_w8_silu_mul_quantize(H1, R, I, A8, SA, as_stream(stream)));
}

int w8a8_gemm(const uint8_t* X8, const uint8_t* SX, const uint8_t* W8, const uint8_t* SW,
              uint16_t* Y, int64_t M, int64_t N, int64_t K, void* stream) {
  if (M < 0 || N < 0) return W4_ERR_SHAPE;
  int v = w8_shape(M, K);
  if (v == W4_OK) v = w8_shape(N, K);
  if (v != W4_OK) return v;
  if (M * N > kMaxElems || w4::w8_gemm_threads(M, N, K) >= kMaxGrid) return W4_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return W4_OK;
  if (!Y) return W4_ERR_NULL;
  if (!aligned(Y, 2)) return W4_ERR_MISALIGNED;
  if (K == 0) return hip_status(w4::launch_zero_bf16(Y, M * N, as_stream(stream)));
  if (!X8 || !SX || !W8 || !SW) return W4_ERR_NULL;
  if (!aligned(X8, 16) || !aligned(W8, 16) || !aligned(SX, 4) || !aligned(SW, 4))
    return W4_ERR_MISALIGNED;
  return hip_status(w4::launch_w8_gemm(X8, SX, W8, SW, Y, M, N, K, as_stream(stream)));
}

// Blocks that hold most experts' rows whole, so that an expert's weights are
// read once: 2048 x 8 pairs over 32 experts of [4096, 4096] take 332 us in
// blocks of 256, 410 of 128 and 581 of 64; 1024 x 8 over 128 of them (64 rows
// each) 442 us in 128 and 513 in 64; 512 x 8 over 128 of [2048, 4096] 230 us in
// 64 and 450 in 16.  Up to 8 rows the 16-row tiles read the weights fastest (64 x
// 8 pairs over 128 of [4096, 4096]: 341 us, 370 in blocks of 64).
int32_t w8_pick_block_size(int64_t T, int32_t k, int32_t E) {
  if (T < 0 || k < 1 || E < 1) return 0;
  if (T > ((int64_t)1 << 40)) return 256;
  const int64_t pairs = T * k;
  if (pairs <= 8 * (int64_t)E) return 16;
  int32_t B = 64;
  while (B < 256 && 2 * (int64_t)B * E < 3 * pairs) B *= 2;
  return B;
}

int w8a8_moe_gemm(const uint8_t* X8, const uint8_t* SX, const uint8_t* W8, const uint8_t* SW,
                  const int32_t* sorted_token_ids, const int32_t* expert_ids,
                  const int32_t* num_tokens_post_padded, uint16_t* Y, int64_t T, int32_t k,
                  int32_t E, int64_t N, int64_t K, int32_t B, int32_t x_row_div, void* stream) {
  const int v = w8_moe_validate(X8, SX, W8, SW, sorted_token_ids, expert_ids,
                                num_tokens_post_padded, Y, 2, T, k, E, N, K, B, x_row_div);
  if (v != W4_OK) return v < 0 ? W4_OK : v;
  return hip_status(w4::launch_w8_moe_gemm(X8, SX, W8, SW, sorted_token_ids, expert_ids,
                                           num_tokens_post_padded, Y, T, k, E, N, K, B, x_row_div,
                                           as_stream(stream)));
}

int w8a8_moe_gemm_swiglu(const uint8_t* X8, const uint8_t* SX, const uint8_t* W8,
                         const uint8_t* SW, const int32_t* sorted_token_ids,
                         const int32_t* expert_ids, const int32_t* num_tokens_post_padded,
                         uint8_t* A8, uint8_t* SA, int64_t T, int32_t k, int32_t E, int64_t I,
                         int64_t K, int32_t B, int32_t x_row_div, void* stream) {
  if (I < 1 || I % 16 != 0) return W4_ERR_SHAPE;
  const int64_t N = I > kMaxI32 / 2 ? kMaxI32 + 1 : 2 * I;   // past the limit: unsupported
  const int v = w8_moe_validate(X8, SX, W8, SW, sorted_token_ids, expert_ids,
                                num_tokens_post_padded, A8, 16, T, k, E, N, K, B, x_row_div);
  if (v > 0) return v;
  if (!w4::w8_moe_swiglu_fits(T * k / x_row_div, I, K, B)) return W4_ERR_UNSUPPORTED;
  if (v < 0) return W4_OK;
  if (!SA) return W4_ERR_NULL;
  if (!aligned(SA, 4)) return W4_ERR_MISALIGNED;
  return hip_status(w4::launch_w8_moe_gemm_swiglu(X8, SX, W8, SW, sorted_token_ids, expert_ids,
                                                  num_tokens_post_padded, A8, SA, T, k, E, I, K, B,
                                                  x_row_div, as_stream(stream)));
}

int w4_moe_route_scored(const float* logits, const float* bias, int64_t T, int32_t E, int32_t k,
                        int32_t sigmoid, int32_t groups, int32_t topk_groups, int32_t group_top,
                        int32_t renorm, float scale, int32_t* topk_ids, float* topk_weights,
                        void* stream) {
  if (T < 0) return W4_ERR_SHAPE;
  const int v = route_rule(E, k, groups, topk_groups, group_top);
  if (v != W4_OK) return v;
  if (T > kMaxTokens) return W4_ERR_UNSUPPORTED;
  if (T == 0) return W4_OK;
  if (!logits || !topk_ids || !topk_weights) return W4_ERR_NULL;
  if (!aligned(logits, 4) || !aligned(bias, 4) || !aligned(topk_ids, 4) ||
      !aligned(topk_weights, 4))
    return W4_ERR_MISALIGNED;
  const w4::RouteRule r = {sigmoid != 0, groups, topk_groups, group_top, renorm != 0, scale};
  return hip_status(w4::launch_route_scored(logits, bias, T, E, k, r, topk_ids, topk_weights,
                                            as_stream(stream)));
}

int w4_moe_route_scored_bwd(const float* logits, const int32_t* topk_ids,
                            const float* topk_weights, const float* grad_weights, int64_t T,
                            int32_t E, int32_t k, int32_t sigmoid, int32_t renorm, float scale,
                            float* grad_logits, void* stream) {
  if (T < 0) return W4_ERR_SHAPE;
  const int v = route_rule(E, k, 1, 1, 1);
  if (v != W4_OK) return v;
  if (T > kMaxTokens) return W4_ERR_UNSUPPORTED;
  if (T == 0) return W4_OK;
  if (!logits || !topk_ids || !topk_weights || !grad_weights || !grad_logits) return W4_ERR_NULL;
  if (!aligned(logits, 4) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4) ||
      !aligned(grad_weights, 4) || !aligned(grad_logits, 4))
    return W4_ERR_MISALIGNED;
  const w4::RouteRule r = {sigmoid != 0, 1, 1, 1, renorm != 0, scale};
  return hip_status(w4::launch_route_scored_bwd(logits, topk_ids, topk_weights, grad_weights, T, E,
                                                k, r, grad_logits, as_stream(stream)));
}

}  // extern "C"

// ------------------------------------------- training the routed experts --

namespace {

constexpr int64_t kBf16MaxCols = (int64_t)1 << 22;
// slots of an expert's pairs that the sums reach with 32-bit byte offsets
constexpr int64_t kBf16MaxSumSlots = (int64_t)1 << 28;
// rows that the products gather, addressed in units of 16 bytes: 32 GiB of bf16, and of
// a checkpoint's scales, addressed in bytes
bool bf16_in_reach(int64_t rows, int64_t cols, bool codes) {
  return rows * cols < (int64_t)1 << 34 && (!codes || rows * w4::w8_cols(cols) < kMaxI32);
}

// Sizes and alignment arrays shared by the grouped bf16 products; W4_OK or an
// error status.
int bf16_moe_validate(const int32_t* sorted_token_ids, const int32_t* expert_ids,
                      const int32_t* num_tokens_post_padded, int64_t T, int32_t k, int32_t E,
                      int64_t N, int64_t K, int32_t B) {
  if (T < 0 || k < 1 || E < 1 || N < 1 || K < 1 || K % 8 != 0 || B < 64 || B % 64 != 0)
    return W4_ERR_SHAPE;
  if (B > 1024 || E > 1024 || T > kMaxI32 || N > kBf16MaxCols || K > kBf16MaxCols ||
      T * k + (int64_t)E * B >= kMaxI32 || T * k * N > kMaxElems || T * k * K > kMaxElems ||
      E * (N * K) > kMaxElems)
    return W4_ERR_UNSUPPORTED;
  if (!sorted_token_ids || !expert_ids || !num_tokens_post_padded) return W4_ERR_NULL;
  if (!aligned(sorted_token_ids, 4) || !aligned(expert_ids, 4) ||
      !aligned(num_tokens_post_padded, 4))
    return W4_ERR_MISALIGNED;
  return W4_OK;
}

}  // namespace

extern "C" {

int32_t w4_bf16_pick_block_size(int64_t T, int32_t k, int32_t E) {
  if (T < 0 || k < 1 || E < 1) return 0;
  if (T > ((int64_t)1 << 40) / k) return 256;
  int32_t B = 64;
  while (B < 256 && 2 * (int64_t)B * E < 3 * T * k) B *= 2;
  return B;
}

int64_t w4_bf16_moe_gemm_workspace(int64_t T, int32_t k, int32_t E, int64_t N, int64_t K, int32_t B) {
  if (T < 0 || k < 1 || E < 1 || N < 1 || K < 1 || B < 64 || B % 64 != 0 || T > kMaxI32 ||
      N > kBf16MaxCols || K > kBf16MaxCols || E > 1024 || B > 1024 ||
      T * k + (int64_t)E * B >= kMaxI32)
    return -1;
  return T == 0 ? 0 : w4::bf16_moe_workspace(T * k, E, N, K, B);
}

int32_t w4_bf16_moe_gemm_tile(int64_t T, int32_t k, int32_t E, int64_t N, int64_t K, int32_t B) {
  if (w4_bf16_moe_gemm_workspace(T, k, E, N, K, B) < 0) return -1;
  return T == 0 ? 0 : w4::bf16_moe_tile(T * k, E, N, K, B);
}

int w4_bf16_moe_gemm(const uint16_t* X, const uint16_t* W, const int32_t* sorted_token_ids,
                     const int32_t* expert_ids, const int32_t* num_tokens_post_padded,
                     uint16_t* Y, int64_t T, int32_t k, int32_t E, int64_t N, int64_t K,
                     int32_t B, int32_t x_row_div, int32_t transposed, float* workspace,
                     void* stream) {
  const int v = bf16_moe_validate(sorted_token_ids, expert_ids, num_tokens_post_padded, T, k, E, N,
                                  K, B);
  if (v == W4_ERR_SHAPE) return v;
  if ((x_row_div != 1 && x_row_div != k) || (transposed && N % 8 != 0)) return W4_ERR_SHAPE;
  if (v == W4_ERR_UNSUPPORTED || !bf16_in_reach(T * k / x_row_div, K, false) ||
      (transposed && !bf16_in_reach(K, N, false)) ||
      w4::bf16_moe_threads(T * k, E, N, K, B) >= kMaxGrid)
    return W4_ERR_UNSUPPORTED;
  if (T == 0) return W4_OK;
  if (v != W4_OK) return v;
  if (!X || !W || !Y) return W4_ERR_NULL;
  if (!aligned(X, 16) || !aligned(W, 16) || !aligned(Y, 2) || !aligned(workspace, 16))
    return W4_ERR_MISALIGNED;
  const w4::Bf16Plan plan = {sorted_token_ids, expert_ids, num_tokens_post_padded, T * k, E, B};
  return hip_status(w4::launch_bf16_moe_gemm(X, W, Y, plan, N, K, x_row_div, transposed != 0,
                                             workspace, as_stream(stream)));
}

int w4_bf16_moe_wgrad(const uint16_t* dY, const void* X, const uint8_t* SX,
                      const int32_t* sorted_token_ids, const int32_t* expert_ids,
                      const int32_t* num_tokens_post_padded, uint16_t* dW, int64_t T, int32_t k,
                      int32_t E, int64_t N, int64_t K, int32_t B, int32_t dy_row_div,
                      int32_t x_row_div, float* workspace, void* stream) {
  const int v = bf16_moe_validate(sorted_token_ids, expert_ids, num_tokens_post_padded, T, k, E, N,
                                  K, B);
  if (v == W4_ERR_SHAPE) return v;
  if ((dy_row_div != 1 && dy_row_div != k) || (x_row_div != 1 && x_row_div != k) || N % 8 != 0 ||
      (SX && K % 16 != 0))
    return W4_ERR_SHAPE;
  if (v == W4_ERR_UNSUPPORTED || T * k + (int64_t)E * B > kBf16MaxSumSlots ||
      !bf16_in_reach(T * k / dy_row_div, N, false) || !bf16_in_reach(T * k / x_row_div, K, SX != nullptr) ||
      w4::bf16_wgrad_threads(E, N, K) >= kMaxGrid)
    return W4_ERR_UNSUPPORTED;
  if (v != W4_OK) return v;
  if (!dW || (T > 0 && (!dY || !X))) return W4_ERR_NULL;
  if (!aligned(dY, 16) || !aligned(X, 16) || !aligned(SX, 4) || !aligned(dW, 16) ||
      !aligned(workspace, 16))
    return W4_ERR_MISALIGNED;
  const w4::Bf16Plan plan = {sorted_token_ids, expert_ids, num_tokens_post_padded, T * k, E, B};
  return hip_status(w4::launch_bf16_moe_wgrad(dY, {X, SX}, dW, plan, N, K, dy_row_div, x_row_div,
                                              workspace, as_stream(stream)));
}

int64_t w4_bf16_moe_wgrad_workspace(int64_t T, int32_t k, int32_t E, int64_t N, int64_t K) {
  if (T < 0 || k < 1 || E < 1 || N < 1 || K < 1 || T > kMaxI32 || N > kBf16MaxCols ||
      K > kBf16MaxCols || E > 1024 || T * k > kBf16MaxSumSlots || E * (N * K) > kMaxElems)
    return -1;
  return w4::bf16_sums_workspace(E, T * k / E, N, K);
}

int32_t w4_bf16_moe_wgrad_tile(int64_t T, int32_t k, int32_t E, int64_t N, int64_t K) {
  if (w4_bf16_moe_wgrad_workspace(T, k, E, N, K) < 0) return -1;
  return w4::bf16_sums_tile(E, T * k / E, N, K);
}

int64_t w4_bf16_gemm_tn_workspace(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0 || M > kMaxI32 || N > kBf16MaxCols || K > kBf16MaxCols ||
      N * K > kMaxElems)
    return -1;
  return N == 0 || K == 0 ? 0 : w4::bf16_sums_workspace(1, M, N, K);
}

int w4_bf16_gemm_tn(const uint16_t* A, const void* B, const uint8_t* SB, uint16_t* C, int64_t M,
                    int64_t N, int64_t K, float* workspace, void* stream) {
  if (M < 0 || N < 0 || K < 0 || N % 8 != 0 || K % 8 != 0 || (SB && K % 16 != 0))
    return W4_ERR_SHAPE;
  if (M > (int64_t)1 << 30 || N > kBf16MaxCols || K > kBf16MaxCols || !bf16_in_reach(M, N, false) ||
      !bf16_in_reach(M, K, SB != nullptr) || N * K > kMaxElems ||
      w4::bf16_wgrad_threads(1, N, K) >= kMaxGrid)
    return W4_ERR_UNSUPPORTED;
  if (N == 0 || K == 0) return W4_OK;
  if (!C || (M > 0 && (!A || !B))) return W4_ERR_NULL;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(SB, 4) || !aligned(C, 16) ||
      !aligned(workspace, 16))
    return W4_ERR_MISALIGNED;
  if (M == 0) return hip_status(w4::launch_zero_bf16(C, N * K, as_stream(stream)));
  return hip_status(w4::launch_bf16_gemm_tn(A, {B, SB}, C, M, N, K, workspace, as_stream(stream)));
}

int w4_silu_mul_bwd(const void* H1, const uint8_t* SH, const uint16_t* dA, const float* weights,
                    int64_t R, int64_t I, uint16_t* dH1, uint16_t* A, float* dw, void* stream) {
  if (R < 0 || I < 0 || I % 8 != 0) return W4_ERR_SHAPE;
  if (R > kMaxI32 || I > kBf16MaxCols || R * I > kMaxElems) return W4_ERR_UNSUPPORTED;
  if (R == 0 || (I == 0 && !dw)) return W4_OK;
  if (I > 0 && (!H1 || !dA || !dH1)) return W4_ERR_NULL;
  if (!aligned(H1, 16) || !aligned(SH, 4) || !aligned(dA, 16) || !aligned(weights, 4) ||
      !aligned(dH1, 16) || !aligned(A, 16) || !aligned(dw, 4))
    return W4_ERR_MISALIGNED;
  return hip_status(w4::launch_silu_mul_bwd({H1, SH}, dA, weights, R, I, dH1, A, dw,
                                            as_stream(stream)));
}

}  // extern "C"
