// Host side of the int8 entry points (include/tsm_gemm.h): argument checks,
// kernel selection and launch on the caller's stream.  As in gemm_api.hip,
// every check runs before any HIP call.
#include <stdlib.h>
#include <string.h>

#include "elems.hpp"
#include "gemm_internal.hpp"
#include "host_checks.hpp"
#include "i8_common.hpp"
#include "tsm_gemm.h"

namespace tsm {
namespace {

const char *i8_name(I8Kernel k) {
  switch (k) {
    case I8Kernel::Block128:
      return "i8_block_128x128x128";
    case I8Kernel::Block64:
      return "i8_block_64x64x128";
    case I8Kernel::Tile:
      return "i8_tile_256x256x128";
    case I8Kernel::Stream:
      return "i8_stream";
    case I8Kernel::Skinny:
      return "i8_skinny";
    default:
      return nullptr;
  }
}

int i8_plan(int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda, int64_t strideA, const float *scale_a,
            int64_t stride_sa, const int8_t *B, int64_t ldb, int64_t strideB, const float *scale_b, int64_t stride_sb,
            void *C, int64_t ldc, int64_t strideC, int64_t batch, const int32_t *rows, bool grouped, int out_dtype,
            int act, float slope, I8Args *p, I8Kernel *kernel, bool *forced) {
  g_detail[0] = '\0';
  *kernel = I8Kernel::None;
  *forced = false;
  if (out_dtype != TSM_F32 && out_dtype != TSM_F16 && out_dtype != TSM_BF16)
    return fail(TSM_ERROR_INVALID_VALUE, "unknown out_dtype %d", out_dtype);
  if (act != TSM_ACT_NONE && act != TSM_ACT_RELU && act != TSM_ACT_LEAKY_RELU)
    return fail(TSM_ERROR_INVALID_VALUE, "unknown activation %d", act);
  if (act == TSM_ACT_LEAKY_RELU && !__builtin_isfinite(slope))
    return fail(TSM_ERROR_INVALID_VALUE, "leaky ReLU slope is not finite");
  if (M < 0 || N < 0 || K < 0)
    return fail(TSM_ERROR_INVALID_VALUE, "negative size M=%lld N=%lld K=%lld", (long long)M, (long long)N, (long long)K);
  if (batch < 0) return fail(TSM_ERROR_INVALID_VALUE, "negative batch %lld", (long long)batch);
  if (M == 0 || N == 0 || batch == 0) return TSM_SUCCESS;  // nothing to compute
  if (grouped) {
    if (!rows) return fail(TSM_ERROR_INVALID_VALUE, "rows is NULL");
    if ((uintptr_t)rows % 4) return fail(TSM_ERROR_INVALID_VALUE, "rows not 4-byte aligned");
  }
  if (M > 0x7fffffffLL || N > 0x7fffffffLL) return fail(TSM_ERROR_NOT_SUPPORTED, "a dimension exceeds 2^31-1");
  if (K > kI8MaxK)
    return fail(TSM_ERROR_NOT_SUPPORTED, "K=%lld exceeds %lld: the int32 sums could overflow", (long long)K,
                (long long)kI8MaxK);
  const int64_t es = fmt_bytes(out_dtype);
  if (!C) return fail(TSM_ERROR_INVALID_VALUE, "C is NULL");
  if ((uintptr_t)C % (uintptr_t)es) return fail(TSM_ERROR_INVALID_VALUE, "C not %lld-byte aligned", (long long)es);
  if (ldc < N) return fail(TSM_ERROR_INVALID_VALUE, "ldc=%lld < N=%lld", (long long)ldc, (long long)N);
  if (batch == 1) strideA = strideB = strideC = stride_sa = stride_sb = 0;
  if (strideA < 0 || strideB < 0 || strideC < 0 || stride_sa < 0 || stride_sb < 0)
    return fail(TSM_ERROR_INVALID_VALUE, "negative stride");
  int64_t span, c_elems, c_bytes;
  if (!extent(1, 0, M, ldc, N, &span) || !extent(batch, strideC, M, ldc, N, &c_elems) || !mul_ok(c_elems, es, &c_bytes))
    return fail(TSM_ERROR_NOT_SUPPORTED, "C extent overflows int64");
  if (batch > 1 && strideC < span)
    return fail(TSM_ERROR_INVALID_VALUE, "strideC=%lld makes the outputs overlap (needs >= %lld)", (long long)strideC,
                (long long)span);
  if (K > 0) {
    if (!A) return fail(TSM_ERROR_INVALID_VALUE, "A is NULL");
    if (!B) return fail(TSM_ERROR_INVALID_VALUE, "B is NULL");
    if (lda < K) return fail(TSM_ERROR_INVALID_VALUE, "lda=%lld < K=%lld", (long long)lda, (long long)K);
    if (ldb < K) return fail(TSM_ERROR_INVALID_VALUE, "ldb=%lld < K=%lld", (long long)ldb, (long long)K);
    int64_t a_bytes, b_bytes;
    if (!extent(batch, strideA, M, lda, K, &a_bytes) || !extent(batch, strideB, N, ldb, K, &b_bytes))
      return fail(TSM_ERROR_NOT_SUPPORTED, "operand extent overflows int64");
    if (ranges_overlap(C, c_bytes, A, a_bytes)) return fail(TSM_ERROR_INVALID_VALUE, "C overlaps A");
    if (ranges_overlap(C, c_bytes, B, b_bytes)) return fail(TSM_ERROR_INVALID_VALUE, "C overlaps B");
  }
  const float *sc[2] = {scale_a, scale_b};
  const int64_t sn[2] = {M, N}, ss[2] = {stride_sa, stride_sb};
  for (int i = 0; i < 2; ++i) {
    if (!sc[i]) continue;
    if ((uintptr_t)sc[i] % 4) return fail(TSM_ERROR_INVALID_VALUE, "scale_%c not 4-byte aligned", 'a' + i);
    int64_t n, bytes;
    if (!extent(batch, ss[i], 1, 0, sn[i], &n) || !mul_ok(n, 4, &bytes))
      return fail(TSM_ERROR_NOT_SUPPORTED, "scale extent overflows int64");
    if (ranges_overlap(C, c_bytes, sc[i], bytes)) return fail(TSM_ERROR_INVALID_VALUE, "C overlaps scale_%c", 'a' + i);
  }

  *p = I8Args{};
  p->A = A;
  p->B = B;
  p->sa = scale_a;
  p->sb = scale_b;
  p->C = C;
  p->M = M;
  p->N = N;
  p->K = K;
  p->lda = lda;
  p->ldb = ldb;
  p->ldc = ldc;
  p->strideA = strideA;
  p->strideB = strideB;
  p->strideC = strideC;
  p->stride_sa = stride_sa;
  p->stride_sb = stride_sb;
  p->batch = batch;
  p->rows = rows;
  p->fmt = out_dtype;
  p->act = act;
  p->slope = act == TSM_ACT_LEAKY_RELU ? slope : 0.f;
  p->vec_store = (uintptr_t)C % (uintptr_t)(4 * es) == 0 && ldc % 4 == 0 && strideC % 4 == 0;

  // 64-tiles up to 128 of 128 x 128 (512 x 4096 x 4096, 128 tiles: 24.6 us
  // against 26.3; 640 x 4096 x 2048, 160: 19.0 against 15.5) and up to 64 rows
  // (48 x 28672 x 4096 31.6 against 34.5), 256-tiles from 72
  // (2304 x 2304 x 1024, 81: 19.4 against 21.1; 2048 x 2048 x 2048, 64: 27.7
  // against 17.3) unless rows fill half of them at most and 128-tiles take one
  // round (128 x 32768 x 8192, 256 of those: 88 us against 69; 128 x 128256 x
  // 4096, 1002: 123 against 141; 16 batches of 100 x 2048 x 4096: 55 against 40);
  // up to 64 rows see i8_skinny_plan.
  const int64_t tiles128 = ((M + 127) / 128) * ((N + 127) / 128), tiles64 = ((M + 63) / 64) * ((N + 63) / 64);
  const bool small = tiles128 * batch <= 128 || (M <= 64 && tiles64 * 512 <= 0xffffffffLL);
  *kernel = small ? I8Kernel::Block64 : I8Kernel::Block128;
  if ((*kernel == I8Kernel::Block64 ? tiles64 : tiles128) * 512 > 0xffffffffLL)
    return fail(TSM_ERROR_NOT_SUPPORTED, "tile grid too large");
  const bool half = M <= 128 && tiles128 * batch <= 256;  // 256-tiles half empty, and a round of 128-tiles does it
  const int64_t tiles256 = ((M + 255) / 256) * ((N + 255) / 256) * batch;
  if (M > 64 && !half && tiles256 >= kFewTiles && i8_tile_supports(*p)) *kernel = I8Kernel::Tile;
  const I8Skinny sk = i8_skinny_plan(*p);
  if (sk.kernel != I8Kernel::None) *kernel = sk.kernel;
  // TSM_GEMM_KERNEL=<name> forces a variant (tests and tuning); names of other
  // families are left alone, a variant that cannot run the problem is an error.
  const char *force = getenv("TSM_GEMM_KERNEL");
  if (force && strncmp(force, "i8_", 3) == 0) {
    I8Kernel want = I8Kernel::None;
    for (I8Kernel k : {I8Kernel::Block128, I8Kernel::Block64, I8Kernel::Tile, I8Kernel::Stream, I8Kernel::Skinny})
      if (strcmp(force, i8_name(k)) == 0) want = k;
    if (want == I8Kernel::None) return fail(TSM_ERROR_INVALID_VALUE, "TSM_GEMM_KERNEL=%s names no kernel", force);
    // (128-tiles fit: they are fewer, and what is checked above where the rule takes them)
    if ((want == I8Kernel::Block64 && tiles64 * 512 > 0xffffffffLL) ||
        (want == I8Kernel::Tile && !i8_tile_supports(*p)) || (want == I8Kernel::Stream && !sk.can_stream) ||
        (want == I8Kernel::Skinny && !sk.can_skinny))
      return fail(TSM_ERROR_NOT_SUPPORTED, "TSM_GEMM_KERNEL=%s cannot run this problem", force);
    *kernel = want;
    *forced = true;
  }
  return TSM_SUCCESS;
}

int i8_run(const I8Args &p, I8Kernel k, bool forced, void *stream) {
  const hipStream_t s = (hipStream_t)stream;
  hipError_t e = hipSuccess;
  switch (k) {
    case I8Kernel::None:
      break;
    case I8Kernel::Block128:
      e = launch_i8_block(p, 128, s);
      break;
    case I8Kernel::Block64:
      e = launch_i8_block(p, 64, s);
      break;
    case I8Kernel::Tile:
      e = launch_i8_tile(p, !forced, s);
      break;
    case I8Kernel::Stream:
      e = launch_i8_stream(p, s);
      break;
    case I8Kernel::Skinny:
      e = launch_i8_skinny(p, s);
      break;
  }
  if (e != hipSuccess) return fail(TSM_ERROR_LAUNCH, "launch failed: %s", hipGetErrorString(e));
  return TSM_SUCCESS;
}

}  // namespace
}  // namespace tsm

extern "C" {

int gemm_i8_strided_batched(int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda, int64_t strideA,
                            const float *scale_a, int64_t stride_sa, const int8_t *B, int64_t ldb, int64_t strideB,
                            const float *scale_b, int64_t stride_sb, void *C, int64_t ldc, int64_t strideC,
                            int64_t batch, int out_dtype, int activation, float slope, void *stream) {
  tsm::I8Args p;
  tsm::I8Kernel k;
  bool forced;
  const int st = tsm::i8_plan(M, N, K, A, lda, strideA, scale_a, stride_sa, B, ldb, strideB, scale_b, stride_sb, C, ldc,
                              strideC, batch, nullptr, false, out_dtype, activation, slope, &p, &k, &forced);
  return st == TSM_SUCCESS ? tsm::i8_run(p, k, forced, stream) : st;
}

int gemm_i8(int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda, const float *scale_a, const int8_t *B,
            int64_t ldb, const float *scale_b, void *C, int64_t ldc, int out_dtype, void *stream) {
  return gemm_i8_strided_batched(M, N, K, A, lda, 0, scale_a, 0, B, ldb, 0, scale_b, 0, C, ldc, 0, 1, out_dtype,
                                 TSM_ACT_NONE, 0.f, stream);
}

int gemm_i8_grouped(int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda, int64_t strideA,
                    const float *scale_a, int64_t stride_sa, const int8_t *B, int64_t ldb, int64_t strideB,
                    const float *scale_b, int64_t stride_sb, void *C, int64_t ldc, int64_t strideC,
                    const int32_t *rows, int64_t groups, int out_dtype, int activation, float slope, void *stream) {
  tsm::I8Args p;
  tsm::I8Kernel k;
  bool forced;
  const int st = tsm::i8_plan(M, N, K, A, lda, strideA, scale_a, stride_sa, B, ldb, strideB, scale_b, stride_sb, C, ldc,
                              strideC, groups, rows, true, out_dtype, activation, slope, &p, &k, &forced);
  return st == TSM_SUCCESS ? tsm::i8_run(p, k, forced, stream) : st;
}

const char *tsm_gemm_i8_kernel_name(int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda, int64_t strideA,
                                    const int8_t *B, int64_t ldb, int64_t strideB, void *C, int64_t ldc,
                                    int64_t strideC, int64_t batch, const int32_t *rows, int out_dtype) {
  tsm::I8Args p;
  tsm::I8Kernel k;
  bool forced;
  if (tsm::i8_plan(M, N, K, A, lda, strideA, nullptr, 0, B, ldb, strideB, nullptr, 0, C, ldc, strideC, batch, rows,
                   rows != nullptr, out_dtype, TSM_ACT_NONE, 0.f, &p, &k, &forced) != TSM_SUCCESS)
    return nullptr;
  return tsm::i8_name(k);
}

int quantize_i8(int64_t R, int64_t C, const void *X, int64_t ldx, int64_t strideX, int xdtype, int8_t *Q, int64_t ldq,
                int64_t strideQ, float *scale, int64_t stride_scale, const int32_t *rows, int64_t groups,
                void *stream) {
  using namespace tsm;
  g_detail[0] = '\0';
  if (xdtype != TSM_F32 && xdtype != TSM_F16 && xdtype != TSM_BF16)
    return fail(TSM_ERROR_INVALID_VALUE, "unknown xdtype %d", xdtype);
  if (R < 0 || C < 0) return fail(TSM_ERROR_INVALID_VALUE, "negative size R=%lld C=%lld", (long long)R, (long long)C);
  if (groups < 0) return fail(TSM_ERROR_INVALID_VALUE, "negative groups %lld", (long long)groups);
  if (R == 0 || groups == 0) return TSM_SUCCESS;
  if (R > 0x7fffffffLL || C > 0x7fffffffLL) return fail(TSM_ERROR_NOT_SUPPORTED, "a dimension exceeds 2^31-1");
  if ((uintptr_t)rows % 4) return fail(TSM_ERROR_INVALID_VALUE, "rows not 4-byte aligned");
  if (!scale) return fail(TSM_ERROR_INVALID_VALUE, "scale is NULL");
  if ((uintptr_t)scale % 4) return fail(TSM_ERROR_INVALID_VALUE, "scale not 4-byte aligned");
  if (groups == 1) strideX = strideQ = stride_scale = 0;
  if (strideX < 0 || strideQ < 0 || stride_scale < 0) return fail(TSM_ERROR_INVALID_VALUE, "negative stride");
  if (groups > 1 && stride_scale < R)
    return fail(TSM_ERROR_INVALID_VALUE, "stride_scale=%lld makes the scales overlap (needs >= %lld)",
                (long long)stride_scale, (long long)R);
  int64_t n, total, s_bytes;
  if (!extent(groups, stride_scale, 1, 0, R, &n) || !mul_ok(n, 4, &s_bytes) || !mul_ok(groups, R, &total))
    return fail(TSM_ERROR_NOT_SUPPORTED, "scale extent overflows int64");
  if (C > 0) {
    const int64_t es = fmt_bytes(xdtype);
    if (!X) return fail(TSM_ERROR_INVALID_VALUE, "X is NULL");
    if (!Q) return fail(TSM_ERROR_INVALID_VALUE, "Q is NULL");
    if ((uintptr_t)X % (uintptr_t)es) return fail(TSM_ERROR_INVALID_VALUE, "X not %lld-byte aligned", (long long)es);
    if (ldx < 0) return fail(TSM_ERROR_INVALID_VALUE, "negative ldx");
    if (ldq < C) return fail(TSM_ERROR_INVALID_VALUE, "ldq=%lld < C=%lld", (long long)ldq, (long long)C);
    int64_t span, q_bytes, x_elems, x_bytes;
    if (!extent(1, 0, R, ldq, C, &span) || !extent(groups, strideQ, R, ldq, C, &q_bytes) ||
        !extent(groups, strideX, R, ldx, C, &x_elems) || !mul_ok(x_elems, es, &x_bytes))
      return fail(TSM_ERROR_NOT_SUPPORTED, "operand extent overflows int64");
    if (groups > 1 && strideQ < span)
      return fail(TSM_ERROR_INVALID_VALUE, "strideQ=%lld makes the codes overlap (needs >= %lld)", (long long)strideQ,
                  (long long)span);
    if (ranges_overlap(Q, q_bytes, X, x_bytes)) return fail(TSM_ERROR_INVALID_VALUE, "Q overlaps X");
    if (ranges_overlap(scale, s_bytes, X, x_bytes)) return fail(TSM_ERROR_INVALID_VALUE, "scale overlaps X");
    if (ranges_overlap(scale, s_bytes, Q, q_bytes)) return fail(TSM_ERROR_INVALID_VALUE, "scale overlaps Q");
  }
  const QuantArgs a{X, Q, scale, R, C, ldx, ldq, strideX, strideQ, stride_scale, groups, rows, xdtype, 0};
  const hipError_t e = launch_quantize(a, (hipStream_t)stream);
  if (e != hipSuccess) return fail(TSM_ERROR_LAUNCH, "launch failed: %s", hipGetErrorString(e));
  return TSM_SUCCESS;
}

}  // extern "C"
