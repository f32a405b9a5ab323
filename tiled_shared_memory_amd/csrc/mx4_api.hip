// Host side of the microscaled 4-bit entry points (include/tsm_gemm.h): argument
// checks, kernel selection and launch on the caller's stream.  Every check runs
// before any HIP call.
#include <stdlib.h>
#include <string.h>

#include "elems.hpp"
#include "gemm_internal.hpp"
#include "host_checks.hpp"
#include "mx4_common.hpp"
#include "tsm_gemm.h"

namespace tsm {
namespace {

const char *mx4_name(Mx4Kernel k) {
  switch (k) {
    case Mx4Kernel::Block128:
      return "mx4_block_128x128x256";
    case Mx4Kernel::Block64:
      return "mx4_block_64x64x256";
    case Mx4Kernel::Tile:
      return "mx4_tile_256x256x256";
    case Mx4Kernel::Ring128:
      return "mx4_ring_128x128x256";
    case Mx4Kernel::Ring64:
      return "mx4_ring_64x64x256";
    case Mx4Kernel::Stream:
      return "mx4_stream";
    default:
      return nullptr;
  }
}

bool float_format(int f) { return f == TSM_F32 || f == TSM_F16 || f == TSM_BF16; }

// Codes and scales of an operand of `rows` rows of K elements, `batch` of them; their extents in bytes.
int operand_check(char name, int64_t rows, int64_t K, const uint8_t *codes, int64_t ld, int64_t stride,
                  const uint8_t *scale, int64_t lds, int64_t stride_scale, int64_t batch, int64_t *bytes,
                  int64_t *scale_bytes) {
  const int64_t kb = mx4_code_bytes(K), nb = mx4_blocks(K);
  if (!codes) return fail(TSM_ERROR_INVALID_VALUE, "%c is NULL", name);
  if (!scale) return fail(TSM_ERROR_INVALID_VALUE, "scale_%c is NULL", name - 'A' + 'a');
  if (ld < kb)
    return fail(TSM_ERROR_INVALID_VALUE, "ld%c=%lld < %lld bytes of a row's codes", name - 'A' + 'a', (long long)ld,
                (long long)kb);
  if (lds < nb)
    return fail(TSM_ERROR_INVALID_VALUE, "ld_s%c=%lld < %lld scales of a row", name - 'A' + 'a', (long long)lds,
                (long long)nb);
  if (!extent(batch, stride, rows, ld, kb, bytes) || !extent(batch, stride_scale, rows, lds, nb, scale_bytes))
    return fail(TSM_ERROR_NOT_SUPPORTED, "operand extent overflows int64");
  return TSM_SUCCESS;
}

struct Call {
  Mx4Args p;
  Mx4Kernel kernel;
  bool forced;
};

// What the products of every form check of their sizes and of C.  false in *work: nothing to compute.
int result_check(int64_t M, int64_t N, int64_t K, void *C, int64_t ldc, int64_t *strideC, int64_t batch,
                 const int32_t *rows, bool grouped, int out_dtype, int act, float slope, int64_t *c_bytes, bool *work) {
  g_detail[0] = '\0';
  *work = false;
  if (!float_format(out_dtype)) return fail(TSM_ERROR_INVALID_VALUE, "unknown out_dtype %d", out_dtype);
  if (act != TSM_ACT_NONE && act != TSM_ACT_RELU && act != TSM_ACT_LEAKY_RELU)
    return fail(TSM_ERROR_INVALID_VALUE, "unknown activation %d", act);
  if (act == TSM_ACT_LEAKY_RELU && !__builtin_isfinite(slope))
    return fail(TSM_ERROR_INVALID_VALUE, "leaky ReLU slope is not finite");
  if (M < 0 || N < 0 || K < 0)
    return fail(TSM_ERROR_INVALID_VALUE, "negative size M=%lld N=%lld K=%lld", (long long)M, (long long)N, (long long)K);
  if (batch < 0) return fail(TSM_ERROR_INVALID_VALUE, "negative batch %lld", (long long)batch);
  if (M == 0 || N == 0 || batch == 0) return TSM_SUCCESS;
  if (grouped && !rows) return fail(TSM_ERROR_INVALID_VALUE, "rows is NULL");
  if ((uintptr_t)rows % 4) return fail(TSM_ERROR_INVALID_VALUE, "rows not 4-byte aligned");
  if (M > 0x7fffffffLL || N > 0x7fffffffLL || K > 0x7fffffffLL)
    return fail(TSM_ERROR_NOT_SUPPORTED, "a dimension exceeds 2^31-1");
  const int64_t es = fmt_bytes(out_dtype);
  if (!C) return fail(TSM_ERROR_INVALID_VALUE, "C is NULL");
  if ((uintptr_t)C % (uintptr_t)es) return fail(TSM_ERROR_INVALID_VALUE, "C not %lld-byte aligned", (long long)es);
  if (ldc < N) return fail(TSM_ERROR_INVALID_VALUE, "ldc=%lld < N=%lld", (long long)ldc, (long long)N);
  if (batch == 1) *strideC = 0;
  if (*strideC < 0) return fail(TSM_ERROR_INVALID_VALUE, "negative stride");
  int64_t span, c_elems;
  if (!extent(1, 0, M, ldc, N, &span) || !extent(batch, *strideC, M, ldc, N, &c_elems) || !mul_ok(c_elems, es, c_bytes))
    return fail(TSM_ERROR_NOT_SUPPORTED, "C extent overflows int64");
  if (batch > 1 && *strideC < span)
    return fail(TSM_ERROR_INVALID_VALUE, "strideC=%lld makes the outputs overlap (needs >= %lld)", (long long)*strideC,
                (long long)span);
  *work = true;
  return TSM_SUCCESS;
}

int mx4_plan(int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda, int64_t strideA, const uint8_t *scale_a,
             int64_t ld_sa, int64_t stride_sa, const uint8_t *B, int64_t ldb, int64_t strideB, const uint8_t *scale_b,
             int64_t ld_sb, int64_t stride_sb, void *C, int64_t ldc, int64_t strideC, int64_t batch,
             const int32_t *rows, bool grouped, int out_dtype, int act, float slope, Call *call) {
  call->kernel = Mx4Kernel::None;
  call->forced = false;
  int64_t c_bytes = 0;
  bool work;
  int st = result_check(M, N, K, C, ldc, &strideC, batch, rows, grouped, out_dtype, act, slope, &c_bytes, &work);
  if (st != TSM_SUCCESS || !work) return st;
  if (batch == 1) strideA = strideB = stride_sa = stride_sb = 0;
  if (strideA < 0 || strideB < 0 || stride_sa < 0 || stride_sb < 0)
    return fail(TSM_ERROR_INVALID_VALUE, "negative stride");
  if (K > 0) {
    int64_t bytes[4];
    if ((st = operand_check('A', M, K, A, lda, strideA, scale_a, ld_sa, stride_sa, batch, bytes, bytes + 1)) != TSM_SUCCESS)
      return st;
    if ((st = operand_check('B', N, K, B, ldb, strideB, scale_b, ld_sb, stride_sb, batch, bytes + 2, bytes + 3)) != TSM_SUCCESS)
      return st;
    const void *in[4] = {A, scale_a, B, scale_b};
    const char *const names[4] = {"A", "scale_a", "B", "scale_b"};
    for (int i = 0; i < 4; ++i)
      if (ranges_overlap(C, c_bytes, in[i], bytes[i])) return fail(TSM_ERROR_INVALID_VALUE, "C overlaps %s", names[i]);
  }
  // Problems that share B and whose rows follow each other in A and C are one of all rows: B is read for all of them at
  // once (64 of 16 x 4096 x 4096: 18 us, one by one 76).  (Not of more rows than one grid of 128-tiles holds, below.)
  if (batch > 1 && !rows && strideB == 0 && stride_sb == 0 && K > 0 && batch <= 0x7fffffffLL / M &&
      (M * batch + 127) / 128 * ((N + 127) / 128) * 512 <= 0xffffffffLL) {
    const int64_t kb = mx4_code_bytes(K), nb = mx4_blocks(K);
    const bool one = M == 1;
    if ((one ? strideA >= kb : strideA == M * lda) && (one ? stride_sa >= nb : stride_sa == M * ld_sa) &&
        (one || strideC == M * ldc)) {
      if (one) lda = strideA, ld_sa = stride_sa, ldc = strideC;
      M *= batch;
      batch = 1;
      strideA = stride_sa = strideC = 0;
    }
  }
  const int64_t es = fmt_bytes(out_dtype);
  Mx4Args &p = call->p;
  p = Mx4Args{};
  p.A = (const int8_t *)A;
  p.B = (const int8_t *)B;
  p.SA = scale_a;
  p.SB = scale_b;
  p.C = C;
  p.M = M;
  p.N = N;
  p.K = K;
  p.kb = mx4_code_bytes(K);
  p.nb = mx4_blocks(K);
  p.lda = lda;
  p.ldb = ldb;
  p.ldsa = ld_sa;
  p.ldsb = ld_sb;
  p.ldc = ldc;
  p.strideA = strideA;
  p.strideB = strideB;
  p.strideSA = stride_sa;
  p.strideSB = stride_sb;
  p.strideC = strideC;
  p.batch = batch;
  p.rows = rows;
  p.fmt = out_dtype;
  p.act = act;
  p.slope = act == TSM_ACT_LEAKY_RELU ? slope : 0.f;
  p.vec_store = (uintptr_t)C % (uintptr_t)(4 * es) == 0 && ldc % 4 == 0 && strideC % 4 == 0;

  // 64-tiles while there are at most 128 of 128 x 128, those while one round of the CUs does them, then 256-tiles; the
  // first two with direct copies where the operands are aligned, else through registers (us, general 64 | 128 | direct 64 |
  // 128 | 256):
  //    512 x 4096 x 4096   16.1 |      | 13.7 | 15.8              256 x 8192 x 8192   33.7 |      | 30.3 | 34.0 | 50
  //   1024 x 2048 x 4096   15.8 | 18.9 | 13.9 | 16.1 | 25.2      1024 x 2560 x 4096        |      | 21.3 | 16.4 | 25
  //   2048 x 2048 x 4096   27.7 | 19.6 | 24.4 | 17.9 | 25.5      2048 x 2304 x 4096   32.8 | 35.6 | 32.5 | 29.9 | 25.2
  //   256 x 16384 x 4096   35   | 24.7 | 32.6 | 22.0 | 29.6      2000 x 2000 x 2001   27   | 17.9
  // and for up to 64 rows: 64 x 16384 x 8192   25.0 | 35.3 | 22.5 | 33.0.
  const int64_t tiles128 = ((M + 127) / 128) * ((N + 127) / 128), tiles64 = ((M + 63) / 64) * ((N + 63) / 64);
  const int64_t all128 = tiles128 > ((int64_t)1 << 40) / batch ? (int64_t)1 << 40 : tiles128 * batch;
  const bool small = all128 <= 128 || (M <= 64 && tiles64 * 512 <= 0xffffffffLL), direct = mx4_tile_supports(p);
  call->kernel = direct ? (small ? Mx4Kernel::Ring64 : Mx4Kernel::Ring128)
                        : (small ? Mx4Kernel::Block64 : Mx4Kernel::Block128);
  if ((small ? tiles64 : tiles128) * 512 > 0xffffffffLL) return fail(TSM_ERROR_NOT_SUPPORTED, "tile grid too large");
  if (M > 64 && all128 > 256 && direct) call->kernel = Mx4Kernel::Tile;
  const Mx4Few few = mx4_few_plan(p);
  if (few.use_stream) call->kernel = Mx4Kernel::Stream;
  // TSM_GEMM_KERNEL=<name> forces a variant (tests and tuning); names of other
  // families are left alone, a variant that cannot run the problem is an error.
  const char *force = getenv("TSM_GEMM_KERNEL");
  if (force && strncmp(force, "mx4_", 4) == 0) {
    Mx4Kernel want = Mx4Kernel::None;
    for (Mx4Kernel k : {Mx4Kernel::Block128, Mx4Kernel::Block64, Mx4Kernel::Ring128, Mx4Kernel::Ring64, Mx4Kernel::Tile,
                        Mx4Kernel::Stream})
      if (strcmp(force, mx4_name(k)) == 0) want = k;
    if (want == Mx4Kernel::None) return fail(TSM_ERROR_INVALID_VALUE, "TSM_GEMM_KERNEL=%s names no kernel", force);
    if (((want == Mx4Kernel::Block64 || want == Mx4Kernel::Ring64) && tiles64 * 512 > 0xffffffffLL) ||
        ((want == Mx4Kernel::Tile || want == Mx4Kernel::Ring128 || want == Mx4Kernel::Ring64) && !direct) || (want == Mx4Kernel::Stream && !few.can_stream))
      return fail(TSM_ERROR_NOT_SUPPORTED, "TSM_GEMM_KERNEL=%s cannot run this problem", force);
    call->kernel = want;
    call->forced = true;
  }
  return TSM_SUCCESS;
}

int launched(hipError_t e) {
  if (e != hipSuccess) return fail(TSM_ERROR_LAUNCH, "launch failed: %s", hipGetErrorString(e));
  return TSM_SUCCESS;
}

int mx4_run(const Call &c, void *stream) {
  const hipStream_t s = (hipStream_t)stream;
  switch (c.kernel) {
    case Mx4Kernel::Block128:
      return launched(launch_mx4_block(c.p, 128, s));
    case Mx4Kernel::Block64:
      return launched(launch_mx4_block(c.p, 64, s));
    case Mx4Kernel::Ring128:
      return launched(launch_mx4_ring(c.p, 128, s));
    case Mx4Kernel::Ring64:
      return launched(launch_mx4_ring(c.p, 64, s));
    case Mx4Kernel::Tile:
      return launched(launch_mx4_tile(c.p, !c.forced, s));
    case Mx4Kernel::Stream:
      return launched(launch_mx4_stream(c.p, s));
    default:
      return TSM_SUCCESS;
  }
}

// Codes and scales of M x K activations in a workspace: rows of 16-byte multiples, then the scales, of 4.
struct Room {
  int64_t ld, lds, codes, bytes;
};
bool room_of(int64_t M, int64_t K, int64_t batch, Room *r) {
  r->ld = (mx4_code_bytes(K) + 15) / 16 * 16;
  r->lds = (mx4_blocks(K) + 3) / 4 * 4;
  int64_t rows, s;
  return mul_ok(M, batch, &rows) && mul_ok(rows, r->ld, &r->codes) && mul_ok(rows, r->lds, &s) &&
         add_ok(r->codes, s, &r->bytes);
}

// The matrix of values X of a quantisation, its extent in bytes.
int values_check(const void *X, int64_t R, int64_t C, int64_t ld, int layout, int64_t stride, int64_t groups, int dtype,
                 int64_t *bytes) {
  const int64_t es = fmt_bytes(dtype);
  if (!X) return fail(TSM_ERROR_INVALID_VALUE, "X is NULL");
  if ((uintptr_t)X % (uintptr_t)es) return fail(TSM_ERROR_INVALID_VALUE, "X not %lld-byte aligned", (long long)es);
  if (ld < 0) return fail(TSM_ERROR_INVALID_VALUE, "negative ldx");
  int64_t n;
  const bool ok = layout == TSM_ROW ? extent(groups, stride, R, ld, C, &n) : extent(groups, stride, C, ld, R, &n);
  if (!ok || !mul_ok(n, es, bytes)) return fail(TSM_ERROR_NOT_SUPPORTED, "X extent overflows int64");
  return TSM_SUCCESS;
}

// Codes and scales of a quantisation and back, their extents in bytes; as outputs their groups may not overlap.
int codes_check(const uint8_t *Q, int64_t ldq, int64_t strideQ, const uint8_t *scale, int64_t lds, int64_t strideS,
                int64_t R, int64_t C, int64_t groups, bool out, int64_t *q_bytes, int64_t *s_bytes) {
  const int64_t kb = mx4_code_bytes(C), nb = mx4_blocks(C);
  if (!Q) return fail(TSM_ERROR_INVALID_VALUE, "Q is NULL");
  if (!scale) return fail(TSM_ERROR_INVALID_VALUE, "scale is NULL");
  if (ldq < kb)
    return fail(TSM_ERROR_INVALID_VALUE, "ldq=%lld < %lld bytes of a row's codes", (long long)ldq, (long long)kb);
  if (lds < nb)
    return fail(TSM_ERROR_INVALID_VALUE, "ld_scale=%lld < %lld scales of a row", (long long)lds, (long long)nb);
  int64_t span, sspan;
  if (!extent(1, 0, R, ldq, kb, &span) || !extent(1, 0, R, lds, nb, &sspan) ||
      !extent(groups, strideQ, R, ldq, kb, q_bytes) || !extent(groups, strideS, R, lds, nb, s_bytes))
    return fail(TSM_ERROR_NOT_SUPPORTED, "codes' extent overflows int64");
  if (out && groups > 1 && strideQ < span)
    return fail(TSM_ERROR_INVALID_VALUE, "strideQ=%lld makes the codes overlap (needs >= %lld)", (long long)strideQ,
                (long long)span);
  if (out && groups > 1 && strideS < sspan)
    return fail(TSM_ERROR_INVALID_VALUE, "stride_scale=%lld makes the scales overlap (needs >= %lld)",
                (long long)strideS, (long long)sspan);
  return TSM_SUCCESS;
}

// Sizes and strides of a quantisation and back.  false in *work: nothing to do.
int quant_sizes(int64_t R, int64_t C, int dtype, const char *dtype_name, const int32_t *rows, int64_t groups,
                int64_t *s0, int64_t *s1, int64_t *s2, bool *work) {
  g_detail[0] = '\0';
  *work = false;
  if (!float_format(dtype)) return fail(TSM_ERROR_INVALID_VALUE, "unknown %s %d", dtype_name, dtype);
  if (R < 0 || C < 0) return fail(TSM_ERROR_INVALID_VALUE, "negative size R=%lld C=%lld", (long long)R, (long long)C);
  if (groups < 0) return fail(TSM_ERROR_INVALID_VALUE, "negative groups %lld", (long long)groups);
  if (R == 0 || C == 0 || groups == 0) return TSM_SUCCESS;
  if (R > 0x7fffffffLL || C > 0x7fffffffLL) return fail(TSM_ERROR_NOT_SUPPORTED, "a dimension exceeds 2^31-1");
  if ((uintptr_t)rows % 4) return fail(TSM_ERROR_INVALID_VALUE, "rows not 4-byte aligned");
  if (groups == 1) *s0 = *s1 = *s2 = 0;
  if (*s0 < 0 || *s1 < 0 || *s2 < 0) return fail(TSM_ERROR_INVALID_VALUE, "negative stride");
  int64_t total;
  if (!mul_ok(groups, R, &total)) return fail(TSM_ERROR_NOT_SUPPORTED, "groups * R overflows int64");
  *work = true;
  return TSM_SUCCESS;
}

}  // namespace
}  // namespace tsm

extern "C" {

int gemm_mx4_strided_batched(int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda, int64_t strideA,
                             const uint8_t *scale_a, int64_t ld_sa, int64_t stride_sa, const uint8_t *B, int64_t ldb,
                             int64_t strideB, const uint8_t *scale_b, int64_t ld_sb, int64_t stride_sb, void *C,
                             int64_t ldc, int64_t strideC, int64_t batch, int out_dtype, int activation, float slope,
                             void *stream) {
  tsm::Call c;
  const int st = tsm::mx4_plan(M, N, K, A, lda, strideA, scale_a, ld_sa, stride_sa, B, ldb, strideB, scale_b, ld_sb,
                               stride_sb, C, ldc, strideC, batch, nullptr, false, out_dtype, activation, slope, &c);
  return st == TSM_SUCCESS ? tsm::mx4_run(c, stream) : st;
}

int gemm_mx4(int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda, const uint8_t *scale_a, int64_t ld_sa,
             const uint8_t *B, int64_t ldb, const uint8_t *scale_b, int64_t ld_sb, void *C, int64_t ldc, int out_dtype,
             void *stream) {
  return gemm_mx4_strided_batched(M, N, K, A, lda, 0, scale_a, ld_sa, 0, B, ldb, 0, scale_b, ld_sb, 0, C, ldc, 0, 1,
                                  out_dtype, TSM_ACT_NONE, 0.f, stream);
}

int gemm_mx4_grouped(int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda, int64_t strideA,
                     const uint8_t *scale_a, int64_t ld_sa, int64_t stride_sa, const uint8_t *B, int64_t ldb,
                     int64_t strideB, const uint8_t *scale_b, int64_t ld_sb, int64_t stride_sb, void *C, int64_t ldc,
                     int64_t strideC, const int32_t *rows, int64_t groups, int out_dtype, int activation, float slope,
                     void *stream) {
  tsm::Call c;
  const int st = tsm::mx4_plan(M, N, K, A, lda, strideA, scale_a, ld_sa, stride_sa, B, ldb, strideB, scale_b, ld_sb,
                               stride_sb, C, ldc, strideC, groups, rows, true, out_dtype, activation, slope, &c);
  return st == TSM_SUCCESS ? tsm::mx4_run(c, stream) : st;
}

const char *tsm_gemm_mx4_kernel_name(int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda, int64_t strideA,
                                     const uint8_t *scale_a, int64_t ld_sa, int64_t stride_sa, const uint8_t *B,
                                     int64_t ldb, int64_t strideB, const uint8_t *scale_b, int64_t ld_sb,
                                     int64_t stride_sb, void *C, int64_t ldc, int64_t strideC, int64_t batch,
                                     const int32_t *rows, int out_dtype) {
  tsm::Call c;
  if (tsm::mx4_plan(M, N, K, A, lda, strideA, scale_a, ld_sa, stride_sa, B, ldb, strideB, scale_b, ld_sb, stride_sb, C,
                    ldc, strideC, batch, rows, rows != nullptr, out_dtype, TSM_ACT_NONE, 0.f, &c) != TSM_SUCCESS)
    return nullptr;
  return tsm::mx4_name(c.kernel);
}

int64_t gemm_mx4_float_a_workspace_bytes(int64_t M, int64_t K, int64_t batch) {
  tsm::Room r;
  return M > 0 && K > 0 && batch > 0 && M <= 0x7fffffffLL && K <= 0x7fffffffLL && tsm::room_of(M, K, batch, &r) ? r.bytes
                                                                                                             : 0;
}

int gemm_mx4_float_a(int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx, int64_t strideX, int xdtype,
                     const uint8_t *B, int64_t ldb, int64_t strideB, const uint8_t *scale_b, int64_t ld_sb,
                     int64_t stride_sb, void *C, int64_t ldc, int64_t strideC, int64_t batch, const int32_t *rows,
                     int out_dtype, int activation, float slope, void *workspace, int64_t workspace_bytes,
                     void *stream) {
  using namespace tsm;
  g_detail[0] = '\0';
  if (!float_format(xdtype)) return fail(TSM_ERROR_INVALID_VALUE, "unknown xdtype %d", xdtype);
  if (workspace_bytes < 0) return fail(TSM_ERROR_INVALID_VALUE, "negative workspace_bytes");
  int64_t c_bytes = 0;
  bool work;
  int st = result_check(M, N, K, C, ldc, &strideC, batch, rows, false, out_dtype, activation, slope, &c_bytes, &work);
  if (st != TSM_SUCCESS || !work) return st;
  if (batch == 1) strideX = 0;
  if (strideX < 0) return fail(TSM_ERROR_INVALID_VALUE, "negative stride");
  // activations that every problem shares are quantised once
  const int64_t groups = strideX == 0 ? 1 : batch;
  Room room{};
  const uint8_t *codes = (const uint8_t *)workspace, *scales = codes;
  if (K > 0) {
    int64_t x_bytes;
    if ((st = values_check(X, M, K, ldx, TSM_ROW, strideX, groups, xdtype, &x_bytes)) != TSM_SUCCESS) return st;
    if (!room_of(M, K, groups, &room)) return fail(TSM_ERROR_NOT_SUPPORTED, "workspace size overflows int64");
    if (!workspace) return fail(TSM_ERROR_INVALID_VALUE, "workspace is NULL");
    if ((uintptr_t)workspace & 15) return fail(TSM_ERROR_INVALID_VALUE, "workspace not 16-byte aligned");
    if (workspace_bytes < room.bytes)
      return fail(TSM_ERROR_INVALID_VALUE, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes,
                  (long long)room.bytes);
    if (ranges_overlap(workspace, room.bytes, X, x_bytes)) return fail(TSM_ERROR_INVALID_VALUE, "workspace overlaps X");
    if (ranges_overlap(C, c_bytes, X, x_bytes)) return fail(TSM_ERROR_INVALID_VALUE, "C overlaps X");
    if (ranges_overlap(workspace, room.bytes, C, c_bytes)) return fail(TSM_ERROR_INVALID_VALUE, "workspace overlaps C");
    scales = codes + room.codes;
    if (B && scale_b && ldb >= mx4_code_bytes(K) && ld_sb >= mx4_blocks(K)) {  // (else refused below)
      int64_t b, s;
      if (extent(batch, batch == 1 ? 0 : strideB, N, ldb, mx4_code_bytes(K), &b) &&
          extent(batch, batch == 1 ? 0 : stride_sb, N, ld_sb, mx4_blocks(K), &s)) {
        if (ranges_overlap(workspace, room.bytes, B, b)) return fail(TSM_ERROR_INVALID_VALUE, "workspace overlaps B");
        if (ranges_overlap(workspace, room.bytes, scale_b, s))
          return fail(TSM_ERROR_INVALID_VALUE, "workspace overlaps scale_b");
      }
    }
  }
  Call c;
  st = mx4_plan(M, N, K, codes, room.ld, groups > 1 ? M * room.ld : 0, scales, room.lds, groups > 1 ? M * room.lds : 0,
                B, ldb, strideB, scale_b, ld_sb, stride_sb, C, ldc, strideC, batch, rows, false, out_dtype, activation,
                slope, &c);
  if (st != TSM_SUCCESS) return st;
  // (problems that mx4_plan made one have to lie so in X too)
  const bool alike = c.p.M == M || (M == 1 ? strideX > 0 : strideX == M * ldx);
  if (c.kernel == Mx4Kernel::Stream && !c.forced && alike && mx4_rows_supports(c.p)) {
    c.p.X = X;
    c.p.ldx = c.p.M != M && M == 1 ? strideX : ldx;
    return launched(launch_mx4_rows(c.p, xdtype, (hipStream_t)stream));
  }
  if (K > 0) {
    const Mx4QuantArgs q{X, (uint8_t *)codes, (uint8_t *)scales, M, K, ldx, room.ld, room.lds, strideX, M * room.ld,
                         M * room.lds, groups, groups > 1 || batch == 1 ? rows : nullptr, xdtype, 0, 0};
    if ((st = launched(launch_quantize_mx4(q, false, (hipStream_t)stream))) != TSM_SUCCESS) return st;
  }
  return mx4_run(c, stream);
}

int mx4_quantize(int64_t R, int64_t C, const void *X, int64_t ldx, int layout, int64_t strideX, int xdtype, uint8_t *Q,
                 int64_t ldq, int64_t strideQ, uint8_t *scale, int64_t ld_scale, int64_t stride_scale,
                 const int32_t *rows, int64_t groups, void *stream) {
  using namespace tsm;
  bool work;
  int st = quant_sizes(R, C, xdtype, "xdtype", rows, groups, &strideX, &strideQ, &stride_scale, &work);
  if (st != TSM_SUCCESS) return st;
  if (layout != TSM_ROW && layout != TSM_COL) return fail(TSM_ERROR_INVALID_VALUE, "unknown layout %d", layout);
  if (!work) return TSM_SUCCESS;
  int64_t x_bytes, q_bytes, s_bytes;
  if ((st = values_check(X, R, C, ldx, layout, strideX, groups, xdtype, &x_bytes)) != TSM_SUCCESS) return st;
  if ((st = codes_check(Q, ldq, strideQ, scale, ld_scale, stride_scale, R, C, groups, true, &q_bytes, &s_bytes)) != TSM_SUCCESS)
    return st;
  if (ranges_overlap(Q, q_bytes, X, x_bytes)) return fail(TSM_ERROR_INVALID_VALUE, "Q overlaps X");
  if (ranges_overlap(scale, s_bytes, X, x_bytes)) return fail(TSM_ERROR_INVALID_VALUE, "scale overlaps X");
  if (ranges_overlap(scale, s_bytes, Q, q_bytes)) return fail(TSM_ERROR_INVALID_VALUE, "scale overlaps Q");
  const Mx4QuantArgs a{X, Q, scale, R, C, ldx, ldq, ld_scale, strideX, strideQ, stride_scale, groups, rows, xdtype, 0, 0};
  return launched(launch_quantize_mx4(a, layout == TSM_COL, (hipStream_t)stream));
}

int mx4_dequantize(int64_t R, int64_t C, const uint8_t *Q, int64_t ldq, int64_t strideQ, const uint8_t *scale,
                   int64_t ld_scale, int64_t stride_scale, void *Y, int64_t ldy, int64_t strideY, int ydtype,
                   const int32_t *rows, int64_t groups, void *stream) {
  using namespace tsm;
  bool work;
  int st = quant_sizes(R, C, ydtype, "ydtype", rows, groups, &strideY, &strideQ, &stride_scale, &work);
  if (st != TSM_SUCCESS || !work) return st;
  int64_t y_elems, y_bytes, span, q_bytes, s_bytes;
  if ((st = codes_check(Q, ldq, strideQ, scale, ld_scale, stride_scale, R, C, groups, false, &q_bytes, &s_bytes)) != TSM_SUCCESS)
    return st;
  const int64_t es = fmt_bytes(ydtype);
  if (!Y) return fail(TSM_ERROR_INVALID_VALUE, "Y is NULL");
  if ((uintptr_t)Y % (uintptr_t)es) return fail(TSM_ERROR_INVALID_VALUE, "Y not %lld-byte aligned", (long long)es);
  if (ldy < C) return fail(TSM_ERROR_INVALID_VALUE, "ldy=%lld < C=%lld", (long long)ldy, (long long)C);
  if (!extent(1, 0, R, ldy, C, &span) || !extent(groups, strideY, R, ldy, C, &y_elems) || !mul_ok(y_elems, es, &y_bytes))
    return fail(TSM_ERROR_NOT_SUPPORTED, "Y extent overflows int64");
  if (groups > 1 && strideY < span)
    return fail(TSM_ERROR_INVALID_VALUE, "strideY=%lld makes the results overlap (needs >= %lld)", (long long)strideY,
                (long long)span);
  if (ranges_overlap(Y, y_bytes, Q, q_bytes)) return fail(TSM_ERROR_INVALID_VALUE, "Y overlaps Q");
  if (ranges_overlap(Y, y_bytes, scale, s_bytes)) return fail(TSM_ERROR_INVALID_VALUE, "Y overlaps scale");
  const Mx4QuantArgs a{Y, (uint8_t *)Q, (uint8_t *)scale, R, C, ldy, ldq, ld_scale, strideY, strideQ, stride_scale, groups, rows, ydtype, 0, 0};
  return launched(launch_dequantize_mx4(a, (hipStream_t)stream));
}

}  // extern "C"
