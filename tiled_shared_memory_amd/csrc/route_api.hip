// Host side of the expert router's entry points (include/tsm_gemm.h): argument
// checks and launch on the caller's stream.  Every check runs before any HIP call.
#include "elems.hpp"
#include "host_checks.hpp"
#include "route_internal.hpp"
#include "tsm_gemm.h"

namespace tsm {
namespace {

struct Range {
  const char *name;
  const void *p;
  int64_t align, bytes;
};

int range_check(const Range &r) {
  if (!r.p) return fail(TSM_ERROR_INVALID_VALUE, "%s is NULL", r.name);
  if ((uintptr_t)r.p % (uintptr_t)r.align)
    return fail(TSM_ERROR_INVALID_VALUE, "%s not %lld-byte aligned", r.name, (long long)r.align);
  return TSM_SUCCESS;
}

// Sizes and formats of both directions; *work: there is something to do.
int route_sizes(int64_t tokens, int64_t experts, int64_t topk, int dtype, int scores, bool *work) {
  g_detail[0] = '\0';
  *work = false;
  if (dtype != TSM_F32 && dtype != TSM_F16 && dtype != TSM_BF16)
    return fail(TSM_ERROR_INVALID_VALUE, "unknown dtype %d", dtype);
  if (scores != TSM_SCORE_SOFTMAX && scores != TSM_SCORE_SIGMOID)
    return fail(TSM_ERROR_INVALID_VALUE, "unknown scores %d", scores);
  if (tokens < 0 || experts < 0 || topk < 0)
    return fail(TSM_ERROR_INVALID_VALUE, "negative size tokens=%lld experts=%lld topk=%lld", (long long)tokens,
                (long long)experts, (long long)topk);
  if (tokens > 0x7fffffffLL) return fail(TSM_ERROR_NOT_SUPPORTED, "tokens exceeds 2^31-1");
  if (experts > RouteInfo::kMaxExperts)
    return fail(TSM_ERROR_NOT_SUPPORTED, "experts=%lld exceeds %d", (long long)experts, RouteInfo::kMaxExperts);
  if (topk > RouteInfo::kMaxTopk)
    return fail(TSM_ERROR_NOT_SUPPORTED, "topk=%lld exceeds %d", (long long)topk, RouteInfo::kMaxTopk);
  if (topk > experts)
    return fail(TSM_ERROR_INVALID_VALUE, "topk=%lld of %lld experts", (long long)topk, (long long)experts);
  *work = tokens > 0 && experts > 0;
  return TSM_SUCCESS;
}

int matrix_range(const char *name, const void *p, int64_t rows, int64_t ld, int64_t cols, int dtype, Range *r) {
  const int64_t es = fmt_bytes(dtype);
  *r = Range{name, p, es, 0};
  if (ld < cols)
    return fail(TSM_ERROR_INVALID_VALUE, "%s: leading dimension %lld < %lld", name, (long long)ld, (long long)cols);
  int64_t n;
  if (!extent(1, 0, rows, ld, cols, &n) || !mul_ok(n, es, &r->bytes))
    return fail(TSM_ERROR_NOT_SUPPORTED, "%s extent overflows int64", name);
  return range_check(*r);
}

// No output may overlap an input or another output.
int disjoint(const Range *out, int no, const Range *in, int ni) {
  for (int i = 0; i < no; ++i) {
    for (int j = 0; j < ni; ++j)
      if (in[j].p && ranges_overlap(out[i].p, out[i].bytes, in[j].p, in[j].bytes))
        return fail(TSM_ERROR_INVALID_VALUE, "%s overlaps %s", out[i].name, in[j].name);
    for (int j = 0; j < i; ++j)
      if (ranges_overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
        return fail(TSM_ERROR_INVALID_VALUE, "%s overlaps %s", out[i].name, out[j].name);
  }
  return TSM_SUCCESS;
}

int launched(hipError_t e) {
  if (e != hipSuccess) return fail(TSM_ERROR_LAUNCH, "launch failed: %s", hipGetErrorString(e));
  return TSM_SUCCESS;
}

}  // namespace
}  // namespace tsm

extern "C" {

int moe_route(int64_t tokens, int64_t experts, int64_t topk, const void *logits, int64_t ld_logits, int dtype,
              int scores, const float *bias, int64_t groups, int64_t top_groups, int group_best, int renormalize,
              float factor, int32_t *ids, float *weights, void *stream) {
  using namespace tsm;
  bool work;
  int st = route_sizes(tokens, experts, topk, dtype, scores, &work);
  if (st != TSM_SUCCESS) return st;
  if (groups < 1 || (experts > 0 && (groups > experts || experts % groups)))
    return fail(TSM_ERROR_INVALID_VALUE, "%lld experts in %lld groups", (long long)experts, (long long)groups);
  if (top_groups < 1 || top_groups > groups)
    return fail(TSM_ERROR_INVALID_VALUE, "top_groups=%lld of %lld groups", (long long)top_groups, (long long)groups);
  if (groups > RouteInfo::kMaxGroups && top_groups < groups)
    return fail(TSM_ERROR_NOT_SUPPORTED, "groups=%lld exceeds %d", (long long)groups, RouteInfo::kMaxGroups);
  if (group_best != 1 && group_best != 2) return fail(TSM_ERROR_INVALID_VALUE, "group_best=%d", group_best);
  if (topk > experts / groups * top_groups)
    return fail(TSM_ERROR_INVALID_VALUE, "topk=%lld of the %lld experts of %lld groups", (long long)topk,
                (long long)(experts / groups * top_groups), (long long)top_groups);
  if (!__builtin_isfinite(factor)) return fail(TSM_ERROR_INVALID_VALUE, "factor is not finite");
  if (!work || topk == 0) return TSM_SUCCESS;
  Range in[2], out[2] = {{"ids", ids, 4, 4 * tokens * topk}, {"weights", weights, 4, 4 * tokens * topk}};
  if ((st = matrix_range("logits", logits, tokens, ld_logits, experts, dtype, &in[0])) != TSM_SUCCESS) return st;
  in[1] = Range{"bias", bias, 4, 4 * experts};
  if (bias && (st = range_check(in[1])) != TSM_SUCCESS) return st;
  for (const Range &r : out)
    if ((st = range_check(r)) != TSM_SUCCESS) return st;
  if ((st = disjoint(out, 2, in, 2)) != TSM_SUCCESS) return st;
  RouteArgs a{};
  a.logits = logits;
  a.tokens = tokens;
  a.ld = ld_logits;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  a.fmt = dtype;
  a.experts = (int32_t)experts;
  a.topk = (int32_t)topk;
  a.groups = (int32_t)groups;
  a.top_groups = (int32_t)top_groups;
  a.best = group_best;
  a.sigmoid = scores == TSM_SCORE_SIGMOID;
  a.renormalize = renormalize != 0;
  a.factor = factor;
  return launched(launch_route(a, (hipStream_t)stream));
}

int moe_route_backward(int64_t tokens, int64_t experts, int64_t topk, const float *dweights, const void *logits,
                       int64_t ld_logits, int dtype, const int32_t *ids, int scores, int renormalize, float factor,
                       void *dlogits, int64_t ld_dlogits, void *stream) {
  using namespace tsm;
  bool work;
  int st = route_sizes(tokens, experts, topk, dtype, scores, &work);
  if (st != TSM_SUCCESS) return st;
  if (!__builtin_isfinite(factor)) return fail(TSM_ERROR_INVALID_VALUE, "factor is not finite");
  if (!work) return TSM_SUCCESS;
  Range in[3] = {{}, {"ids", ids, 4, 4 * tokens * topk}, {"dweights", dweights, 4, 4 * tokens * topk}}, out[1];
  if ((st = matrix_range("logits", logits, tokens, ld_logits, experts, dtype, &in[0])) != TSM_SUCCESS) return st;
  for (int i = 1; i < 3 && topk > 0; ++i)
    if ((st = range_check(in[i])) != TSM_SUCCESS) return st;
  if ((st = matrix_range("dlogits", dlogits, tokens, ld_dlogits, experts, dtype, &out[0])) != TSM_SUCCESS) return st;
  if ((st = disjoint(out, 1, in, 3)) != TSM_SUCCESS) return st;
  RouteArgs a{};
  a.logits = logits;
  a.dlogits = dlogits;
  a.tokens = tokens;
  a.ld = ld_logits;
  a.ldd = ld_dlogits;
  a.ids = const_cast<int32_t *>(ids);
  a.weights = const_cast<float *>(dweights);
  a.fmt = dtype;
  a.experts = (int32_t)experts;
  a.topk = (int32_t)topk;
  a.groups = a.top_groups = 1;
  a.sigmoid = scores == TSM_SCORE_SIGMOID;
  a.renormalize = renormalize != 0;
  a.factor = factor;
  return launched(launch_route_backward(a, (hipStream_t)stream));
}

}  // extern "C"
