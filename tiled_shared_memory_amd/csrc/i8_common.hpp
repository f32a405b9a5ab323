// Pieces shared by the int8 product kernels.
#pragma once

#include "codes.hpp"
#include "i8_internal.hpp"

namespace tsm {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// v_mfma_i32_16x16x64_i8: D(16x16) += A(16x64) * B(64x16), 16 codes per lane and
// operand: row (column) lane % 16, k = 16 * (lane / 16) + 0..15 in both, so any
// order of k that both operands share gives the same sum.  D as for the
// 16x16x32 forms (mfma.hpp).
__device__ __forceinline__ i32x4 mfma_i8(u32x4 a, u32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// Four results of one row of C, columns n .. n+3 (n < N): each sum to float32
// once, times the token's scale, times the channel's, then the activation and
// the output's rounding.
template <int FMT>
__device__ __forceinline__ void store_i8(const I8Args &p, const Epilogue &ep, char *row, int64_t n, float sa,
                                         const float (&sb)[4], i32x4 acc) {
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = act_codes(ep, (float)acc[i] * sa * sb[i]);
  if (p.vec_store && n + 4 <= p.N) {
    if constexpr (FMT == FMT_F32) {
      *reinterpret_cast<f32x4 *>(row + n * 4) = f32x4{v[0], v[1], v[2], v[3]};
    } else {
      *reinterpret_cast<u32x2 *>(row + n * 2) = u32x2{f32_elem<FMT>(v[0]) | (f32_elem<FMT>(v[1]) << 16),
                                                      f32_elem<FMT>(v[2]) | (f32_elem<FMT>(v[3]) << 16)};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < p.N) put_bits<FMT>(row, n + i, f32_elem<FMT>(v[i]));
  }
}

// Scales of channels n .. n+3 of problem z (past N the last one's, for results that are not stored).
__device__ __forceinline__ void channel_scales(const I8Args &p, int64_t z, int64_t n, float (&c)[4]) {
  if (!p.sb) {  // uniform
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = 1.f;
    return;
  }
  const float *sb = p.sb + z * p.stride_sb;
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = sb[n + i < p.N ? n + i : p.N - 1];
}

}  // namespace tsm
