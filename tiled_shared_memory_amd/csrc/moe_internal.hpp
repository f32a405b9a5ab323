// Interface between the expert-routing API (moe_api.hip) and its kernels (moe.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tsm {

struct SortArgs {
  const void *ids;  // [tokens][ld], int32 or int64
  int64_t tokens, ld;
  int32_t topk, experts;
  int64_t capacity;
  bool id64;
  int32_t *positions;  // [tokens][topk]
  int32_t *counts;     // [experts]
  int32_t *hist;       // [blocks][sort_pitch(experts)], 16-byte aligned (null: one block)
  bool scanned;        // hist holds sums of the blocks before (set by the launch)
};
struct SortInfo {
  static constexpr int kMaxExperts = 512;
  static constexpr int64_t kOneBlock = 8192;  // entries one workgroup sorts by itself
  static constexpr int64_t kTile = 4096;      // entries per workgroup otherwise
  static constexpr int64_t kScanBlocks = 256; // workgroups from which their counts are summed in a launch of their own
};
inline int64_t sort_blocks(int64_t n) { return n <= SortInfo::kOneBlock ? 1 : (n + SortInfo::kTile - 1) / SortInfo::kTile; }
__host__ __device__ inline int64_t sort_pitch(int64_t experts) { return (experts + 3) / 4 * 4; }
hipError_t launch_sort(const SortArgs &a, hipStream_t stream);

// Rows between a token-major matrix and the experts' slabs.
struct MoveArgs {
  const void *X;   // dispatch: token rows; combine: slab rows; backward: dY
  void *Y;         // dispatch: slab rows; combine: token rows; backward: the slabs' gradient
  const void *S;   // backward: slab rows
  int64_t ldx, ldy, lds;  // elements
  int64_t tokens, hidden, slots;
  int64_t t0;      // first token of this launch
  int32_t topk;
  int32_t fmt;
  int32_t segs;    // workgroups per row
  const int32_t *positions;
  const float *weights;  // [tokens][topk], or null (ones)
  const float *scale;    // dispatch: a float per token, or null
  float *slab_scale;     // dispatch: a float per slab row
  float *dweights;       // backward: [tokens][topk]
};
hipError_t launch_dispatch(const MoveArgs &a, hipStream_t stream);
hipError_t launch_combine(const MoveArgs &a, hipStream_t stream);
hipError_t launch_combine_backward(const MoveArgs &a, hipStream_t stream);

}  // namespace tsm
