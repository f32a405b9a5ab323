// Interface between the expert router's API (route_api.hip) and its kernels (route.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tsm {

struct RouteInfo {
  static constexpr int kMaxExperts = 512;  // as the sort's
  static constexpr int kMaxTopk = 64;
  static constexpr int kMaxGroups = 64;
};

struct RouteArgs {
  const void *logits;  // [tokens][ld]
  void *dlogits;       // backward: [tokens][ldd]
  int64_t tokens, ld, ldd;
  const float *bias;   // [experts], or null
  int32_t *ids;        // [tokens][topk]
  float *weights;      // [tokens][topk]; backward: their gradients
  int32_t fmt;
  int32_t experts, topk;
  int32_t groups, top_groups, best;  // groups == top_groups: no choice of groups
  int32_t sigmoid, renormalize;
  float factor;
  int64_t t0;          // first token of this launch
  int32_t size, shift, per;  // route8_kernel: 2^shift lanes hold `size` experts, `per` each
};
hipError_t launch_route(const RouteArgs &a, hipStream_t stream);
hipError_t launch_route_backward(const RouteArgs &a, hipStream_t stream);

}  // namespace tsm
