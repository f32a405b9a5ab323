// Host side of the expert-routing entry points (include/tsm_gemm.h): argument
// checks and launch on the caller's stream.  Every check runs before any HIP call.
#include "elems.hpp"
#include "host_checks.hpp"
#include "moe_internal.hpp"
#include "tsm_gemm.h"

namespace tsm {
namespace {

// A matrix operand of the row operators: non-null, aligned, its extent in bytes.
int matrix_check(const char *name, const void *p, int64_t rows, int64_t ld, int64_t cols, int64_t es, int64_t *bytes) {
  if (!p) return fail(TSM_ERROR_INVALID_VALUE, "%s is NULL", name);
  if ((uintptr_t)p % (uintptr_t)es) return fail(TSM_ERROR_INVALID_VALUE, "%s not %lld-byte aligned", name, (long long)es);
  if (ld < cols)
    return fail(TSM_ERROR_INVALID_VALUE, "%s: leading dimension %lld < %lld", name, (long long)ld, (long long)cols);
  int64_t n;
  if (!extent(1, 0, rows, ld, cols, &n) || !mul_ok(n, es, bytes))
    return fail(TSM_ERROR_NOT_SUPPORTED, "%s extent overflows int64", name);
  return TSM_SUCCESS;
}

int array_check(const char *name, const void *p) {
  if (!p) return fail(TSM_ERROR_INVALID_VALUE, "%s is NULL", name);
  if ((uintptr_t)p % 4) return fail(TSM_ERROR_INVALID_VALUE, "%s not 4-byte aligned", name);
  return TSM_SUCCESS;
}

struct Range {
  const char *name;
  const void *p;
  int64_t bytes;
};

// No output may overlap an input or another output.
template <int NO, int NI>
int disjoint(const Range (&out)[NO], const Range (&in)[NI]) {
  for (int i = 0; i < NO; ++i) {
    if (!out[i].p) continue;
    for (int j = 0; j < NI; ++j)
      if (in[j].p && ranges_overlap(out[i].p, out[i].bytes, in[j].p, in[j].bytes))
        return fail(TSM_ERROR_INVALID_VALUE, "%s overlaps %s", out[i].name, in[j].name);
    for (int j = 0; j < i; ++j)
      if (out[j].p && ranges_overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
        return fail(TSM_ERROR_INVALID_VALUE, "%s overlaps %s", out[i].name, out[j].name);
  }
  return TSM_SUCCESS;
}

// Sizes shared by the row operators; *entries = tokens * topk.
int sizes_check(int64_t tokens, int64_t topk, int64_t hidden, int64_t slots, int64_t *entries) {
  g_detail[0] = '\0';
  if (tokens < 0 || topk < 0 || hidden < 0 || slots < 0)
    return fail(TSM_ERROR_INVALID_VALUE, "negative size tokens=%lld topk=%lld hidden=%lld slots=%lld",
                (long long)tokens, (long long)topk, (long long)hidden, (long long)slots);
  if (tokens > 0x7fffffffLL || topk > 0x7fffffffLL || hidden > 0x7fffffffLL || slots > 0x7fffffffLL)
    return fail(TSM_ERROR_NOT_SUPPORTED, "a size exceeds 2^31-1");
  *entries = tokens * topk;  // below 2^62
  if (*entries > 0x7fffffffLL) return fail(TSM_ERROR_NOT_SUPPORTED, "tokens * topk exceeds 2^31-1");
  return TSM_SUCCESS;
}

int launched(hipError_t e) {
  if (e != hipSuccess) return fail(TSM_ERROR_LAUNCH, "launch failed: %s", hipGetErrorString(e));
  return TSM_SUCCESS;
}

}  // namespace
}  // namespace tsm

extern "C" {

int64_t moe_sort_workspace_bytes(int64_t tokens, int64_t topk, int64_t experts) {
  int64_t n;
  if (tokens <= 0 || topk <= 0 || experts <= 0 || !tsm::mul_ok(tokens, topk, &n) || n > 0x7fffffffLL ||
      experts > tsm::SortInfo::kMaxExperts)
    return 0;
  const int64_t blocks = tsm::sort_blocks(n);
  return blocks > 1 ? blocks * tsm::sort_pitch(experts) * 4 : 0;
}

int moe_sort(int64_t tokens, int64_t topk, const void *ids, int64_t ld_ids, int idtype, int64_t experts,
             int64_t capacity, int32_t *positions, int32_t *counts, void *workspace, int64_t workspace_bytes,
             void *stream) {
  using namespace tsm;
  g_detail[0] = '\0';
  if (idtype != TSM_I32 && idtype != TSM_I64) return fail(TSM_ERROR_INVALID_VALUE, "unknown idtype %d", idtype);
  if (tokens < 0 || topk < 0 || experts < 0 || capacity < 0)
    return fail(TSM_ERROR_INVALID_VALUE, "negative size tokens=%lld topk=%lld experts=%lld capacity=%lld",
                (long long)tokens, (long long)topk, (long long)experts, (long long)capacity);
  if (workspace_bytes < 0) return fail(TSM_ERROR_INVALID_VALUE, "negative workspace_bytes");
  if (experts > SortInfo::kMaxExperts)
    return fail(TSM_ERROR_NOT_SUPPORTED, "experts=%lld exceeds %d", (long long)experts, SortInfo::kMaxExperts);
  int64_t n, slots;
  if (!mul_ok(tokens, topk, &n) || n > 0x7fffffffLL)
    return fail(TSM_ERROR_NOT_SUPPORTED, "tokens * topk exceeds 2^31-1");
  if (!mul_ok(experts, capacity, &slots) || slots > 0x7fffffffLL)
    return fail(TSM_ERROR_NOT_SUPPORTED, "experts * capacity exceeds 2^31-1");
  int st;
  if (experts > 0 && (st = array_check("counts", counts)) != TSM_SUCCESS) return st;
  const int64_t es = idtype == TSM_I64 ? 8 : 4;
  int64_t id_bytes = 0;
  if (n > 0) {
    if ((st = matrix_check("ids", ids, tokens, ld_ids, topk, es, &id_bytes)) != TSM_SUCCESS) return st;
    if ((st = array_check("positions", positions)) != TSM_SUCCESS) return st;
  }
  const int64_t need = moe_sort_workspace_bytes(tokens, topk, experts);
  if (need) {
    if (!workspace) return fail(TSM_ERROR_INVALID_VALUE, "workspace is NULL");
    if ((uintptr_t)workspace & 15) return fail(TSM_ERROR_INVALID_VALUE, "workspace not 16-byte aligned");
    if (workspace_bytes < need)
      return fail(TSM_ERROR_INVALID_VALUE, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes,
                  (long long)need);
  }
  const Range out[3] = {{"positions", n ? positions : nullptr, n * 4},
                        {"counts", experts ? counts : nullptr, experts * 4},
                        {"workspace", need ? workspace : nullptr, need}};
  const Range in[1] = {{"ids", n ? ids : nullptr, id_bytes}};
  if ((st = disjoint(out, in)) != TSM_SUCCESS) return st;
  if (n == 0 && experts == 0) return TSM_SUCCESS;
  const SortArgs a{ids,      tokens, topk ? ld_ids : 0, (int32_t)topk, (int32_t)experts, capacity, idtype == TSM_I64,
                   positions, counts, need ? (int32_t *)workspace : nullptr, false};
  return launched(launch_sort(a, (hipStream_t)stream));
}

int moe_dispatch(int64_t tokens, int64_t topk, int64_t hidden, const void *X, int64_t ldx, int dtype,
                 const float *scale, const int32_t *positions, int64_t slots, void *slabs, int64_t ld_slabs,
                 float *slab_scale, void *stream) {
  using namespace tsm;
  int64_t n;
  int st = sizes_check(tokens, topk, hidden, slots, &n);
  if (st != TSM_SUCCESS) return st;
  if (dtype < TSM_F32 || dtype > TSM_I8) return fail(TSM_ERROR_INVALID_VALUE, "unknown dtype %d", dtype);
  if (!scale != !slab_scale) return fail(TSM_ERROR_INVALID_VALUE, "scale and slab_scale come together");
  if (n == 0 || slots == 0 || (hidden == 0 && !scale)) return TSM_SUCCESS;
  int64_t xb = 0, sb = 0;
  if (hidden > 0) {
    if ((st = matrix_check("X", X, tokens, ldx, hidden, fmt_bytes(dtype), &xb)) != TSM_SUCCESS) return st;
    if ((st = matrix_check("slabs", slabs, slots, ld_slabs, hidden, fmt_bytes(dtype), &sb)) != TSM_SUCCESS) return st;
  }
  if ((st = array_check("positions", positions)) != TSM_SUCCESS) return st;
  if (scale && ((st = array_check("scale", scale)) != TSM_SUCCESS ||
                (st = array_check("slab_scale", slab_scale)) != TSM_SUCCESS))
    return st;
  const Range out[2] = {{"slabs", hidden ? slabs : nullptr, sb}, {"slab_scale", slab_scale, slots * 4}};
  const Range in[3] = {{"X", hidden ? X : nullptr, xb}, {"positions", positions, n * 4}, {"scale", scale, tokens * 4}};
  if ((st = disjoint(out, in)) != TSM_SUCCESS) return st;
  MoveArgs a{};
  a.X = X;
  a.Y = slabs;
  a.ldx = ldx;
  a.ldy = ld_slabs;
  a.tokens = tokens;
  a.hidden = hidden;
  a.slots = slots;
  a.topk = (int32_t)topk;
  a.fmt = dtype;
  a.positions = positions;
  a.scale = scale;
  a.slab_scale = slab_scale;
  return launched(launch_dispatch(a, (hipStream_t)stream));
}

int moe_combine(int64_t tokens, int64_t topk, int64_t hidden, const void *slabs, int64_t ld_slabs, int64_t slots,
                int dtype, const int32_t *positions, const float *weights, void *Y, int64_t ldy, void *stream) {
  using namespace tsm;
  int64_t n;
  int st = sizes_check(tokens, topk, hidden, slots, &n);
  if (st != TSM_SUCCESS) return st;
  if (dtype < TSM_F32 || dtype > TSM_BF16) return fail(TSM_ERROR_INVALID_VALUE, "unknown dtype %d", dtype);
  if (tokens == 0 || hidden == 0) return TSM_SUCCESS;
  int64_t yb = 0, sb = 0;
  if ((st = matrix_check("Y", Y, tokens, ldy, hidden, fmt_bytes(dtype), &yb)) != TSM_SUCCESS) return st;
  if (slots > 0 && (st = matrix_check("slabs", slabs, slots, ld_slabs, hidden, fmt_bytes(dtype), &sb)) != TSM_SUCCESS)
    return st;
  if (n > 0 && (st = array_check("positions", positions)) != TSM_SUCCESS) return st;
  if ((uintptr_t)weights % 4) return fail(TSM_ERROR_INVALID_VALUE, "weights not 4-byte aligned");
  const Range out[1] = {{"Y", Y, yb}};
  const Range in[3] = {{"slabs", slots ? slabs : nullptr, sb}, {"positions", n ? positions : nullptr, n * 4},
                       {"weights", n ? weights : nullptr, n * 4}};
  if ((st = disjoint(out, in)) != TSM_SUCCESS) return st;
  MoveArgs a{};
  a.X = slabs;
  a.Y = Y;
  a.ldx = ld_slabs;
  a.ldy = ldy;
  a.tokens = tokens;
  a.hidden = hidden;
  a.slots = slots;
  a.topk = slots ? (int32_t)topk : 0;  // no slabs: zeros
  a.fmt = dtype;
  a.positions = positions;
  a.weights = weights;
  return launched(launch_combine(a, (hipStream_t)stream));
}

int moe_combine_backward(int64_t tokens, int64_t topk, int64_t hidden, const void *dY, int64_t lddy, const void *slabs,
                         int64_t ld_slabs, int64_t slots, int dtype, const int32_t *positions, const float *weights,
                         void *dslabs, int64_t ld_dslabs, float *dweights, void *stream) {
  using namespace tsm;
  int64_t n;
  int st = sizes_check(tokens, topk, hidden, slots, &n);
  if (st != TSM_SUCCESS) return st;
  if (dtype < TSM_F32 || dtype > TSM_BF16) return fail(TSM_ERROR_INVALID_VALUE, "unknown dtype %d", dtype);
  if (n == 0) return TSM_SUCCESS;
  const int64_t es = fmt_bytes(dtype);
  int64_t gb = 0, sb = 0, db = 0;
  if (hidden > 0 && slots > 0) {
    if ((st = matrix_check("dY", dY, tokens, lddy, hidden, es, &gb)) != TSM_SUCCESS) return st;
    if ((st = matrix_check("slabs", slabs, slots, ld_slabs, hidden, es, &sb)) != TSM_SUCCESS) return st;
    if ((st = matrix_check("dslabs", dslabs, slots, ld_dslabs, hidden, es, &db)) != TSM_SUCCESS) return st;
  }
  if ((st = array_check("positions", positions)) != TSM_SUCCESS) return st;
  if ((st = array_check("dweights", dweights)) != TSM_SUCCESS) return st;
  if ((uintptr_t)weights % 4) return fail(TSM_ERROR_INVALID_VALUE, "weights not 4-byte aligned");
  const Range out[2] = {{"dslabs", db ? dslabs : nullptr, db}, {"dweights", dweights, n * 4}};
  const Range in[4] = {{"dY", gb ? dY : nullptr, gb}, {"slabs", sb ? slabs : nullptr, sb},
                       {"positions", positions, n * 4}, {"weights", weights, n * 4}};
  if ((st = disjoint(out, in)) != TSM_SUCCESS) return st;
  MoveArgs a{};
  a.X = dY;
  a.Y = dslabs;
  a.S = slabs;
  a.ldx = lddy;
  a.ldy = ld_dslabs;
  a.lds = ld_slabs;
  a.tokens = tokens;
  a.hidden = slots ? hidden : 0;
  a.slots = slots;
  a.topk = (int32_t)topk;
  a.fmt = dtype;
  a.positions = positions;
  a.weights = weights;
  a.dweights = dweights;
  return launched(launch_combine_backward(a, (hipStream_t)stream));
}

}  // extern "C"
