// Interface between the microscaled 4-bit API (mx4_api.hip) and its kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tsm {

constexpr int kMxBlock = 32;  // elements per scale
inline int64_t mx4_code_bytes(int64_t C) { return (C + 1) / 2; }
inline int64_t mx4_blocks(int64_t C) { return (C + kMxBlock - 1) / kMxBlock; }

// C[i][j] = act(sum_k A[i][k] B[j][k]), both operands contiguous along k: codes of 4 bits, two to a byte, and a scale
// byte per 32 of them.
struct Mx4Args {
  const int8_t *A, *B;      // codes
  const uint8_t *SA, *SB;   // scale bytes
  void *C;
  const void *X;            // few rows: activations to quantise, in A's place
  int64_t ldx;
  int64_t M, N, K;          // K in elements
  int64_t kb, nb;           // bytes of codes and of scales per row
  int64_t lda, ldb, ldsa, ldsb, ldc;  // bytes; of C elements
  int64_t strideA, strideB, strideSA, strideSB, strideC;
  int64_t batch;
  const int32_t *rows;  // grouped: row counts in device memory
  int32_t fmt;          // output format (TSM_F32, TSM_F16, TSM_BF16)
  int32_t act;
  float slope;
  int32_t vec_store;    // C's rows take stores of 4 elements
  // set by the launch
  int32_t tiles_m, tiles_n;
  int64_t z0;       // first problem of this launch
  int32_t nz;       // problems of this launch
  int32_t cus;      // 256 x 256 tiles: CUs, one tile each per round (0: no second launch)
};

// tile: 64 or 128; for operands that mx4_tile_supports takes.
hipError_t launch_mx4_ring(const Mx4Args &p, int tile, hipStream_t stream);
// 256 x 256 tiles: see mx4_tile_supports for what they need.
bool mx4_tile_supports(const Mx4Args &p);
// whole_only: tiles left over from whole rounds of the CUs go to launch_mx4_rest.
hipError_t launch_mx4_tile(const Mx4Args &p, bool whole_only, hipStream_t stream);
// The 256 x 256 tiles that whole_rounds leaves of a launch (tiles_m, tiles_n, z0 and nz set), at most `tiles`, in
// smaller ones.
hipError_t launch_mx4_rest(const Mx4Args &a, int64_t tiles, hipStream_t stream);
// CUs of the current device (gemm_api.hip).
int device_cus();

enum class Mx4Kernel { None, Block128, Block64, Ring128, Ring64, Tile, Stream };
// Few rows (up to 64): what the problem allows, and the rule's choice.
struct Mx4Few {
  bool can_stream = false, use_stream = false;
  int rows = 0, nb = 0, waves = 0;  // streaming: rows by 16 nb columns per workgroup of `waves` waves
};
Mx4Few mx4_few_plan(const Mx4Args &p);
hipError_t launch_mx4_stream(const Mx4Args &p, hipStream_t stream);
// Activations X of format xfmt in A's place, quantised within the launch.
bool mx4_rows_supports(const Mx4Args &p);
hipError_t launch_mx4_rows(const Mx4Args &p, int xfmt, hipStream_t stream);
hipError_t launch_mx4_block(const Mx4Args &p, int tile, hipStream_t stream);

struct Mx4QuantArgs {
  const void *X;  // quantisation: the values; back: the result
  uint8_t *Q, *S;
  int64_t R, C, ldx, ldq, lds, strideX, strideQ, strideS, groups;
  const int32_t *rows;
  int32_t fmt;
  int32_t segs;    // workgroups per row
  int64_t r0;      // first (group, row) pair of this launch, or its first (group, row tile)
};
hipError_t launch_quantize_mx4(const Mx4QuantArgs &a, bool columns, hipStream_t stream);
hipError_t launch_dequantize_mx4(const Mx4QuantArgs &a, hipStream_t stream);

}  // namespace tsm
