// Interface between the int8 API (i8_api.hip) and its kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tsm {

// C[i][j] = act(sa[i] * sb[j] * sum_k A[i][k] B[j][k]): A row-major, B column-major (both contiguous along k).
struct I8Args {
  const int8_t *A, *B;
  const float *sa, *sb;  // null: ones
  void *C;
  int64_t M, N, K;
  int64_t lda, ldb, ldc;
  int64_t strideA, strideB, strideC, stride_sa, stride_sb;
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

// |sum| <= K * 128 * 128 stays below 2^31
constexpr int64_t kI8MaxK = 131071;

// 256 x 256 tiles: see i8_tile_supports for what they need.
bool i8_tile_supports(const I8Args &p);
// whole_only: tiles left over from whole rounds of the CUs go to launch_i8_rest.
hipError_t launch_i8_tile(const I8Args &p, bool whole_only, hipStream_t stream);
// The 256 x 256 tiles that whole_rounds leaves of a launch (tiles_m, tiles_n, z0 and nz set), as 128 x 128 ones.
hipError_t launch_i8_rest(const I8Args &a, hipStream_t stream);
// CUs of the current device (gemm_api.hip).
int device_cus();

enum class I8Kernel { None, Block128, Block64, Tile, Stream, Skinny };
// Few rows (up to 64).
struct I8Skinny {
  I8Kernel kernel = I8Kernel::None;  // the rule's choice; None: the general kernel
  bool can_skinny = false, can_stream = false;  // what the problem allows
  int rows = 0, nb = 0, waves = 0;  // streaming: rows by 16 nb columns per workgroup of `waves` waves
};
I8Skinny i8_skinny_plan(const I8Args &p);
hipError_t launch_i8_stream(const I8Args &p, hipStream_t stream);
hipError_t launch_i8_skinny(const I8Args &p, hipStream_t stream);
hipError_t launch_i8_block(const I8Args &p, int tile, hipStream_t stream);

struct QuantArgs {
  const void *X;
  int8_t *Q;
  float *scale;
  int64_t R, C, ldx, ldq, strideX, strideQ, strideS, groups;
  const int32_t *rows;
  int32_t fmt;
  int64_t r0;  // first (group, row) pair of this launch
};
hipError_t launch_quantize(const QuantArgs &a, hipStream_t stream);

}  // namespace tsm
