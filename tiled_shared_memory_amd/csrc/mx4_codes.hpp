// Microscaled 4-bit codes and scale bytes of eight elements at a time (quantize_mx4.hip has the rule).
#pragma once

#include "chunk.hpp"
#include "elems.hpp"

namespace tsm {

// Scale byte of a block from the bits of its largest magnitude (a NaN's are above infinity's).
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const uint32_t f = top >> 23;
  return top >= 0x7f800000u ? 255u : f > 2 ? f - 2 : 0u;
}
// The power of two of a scale byte below 255.
__device__ __forceinline__ float scale_of(uint32_t e) { return __builtin_bit_cast(float, e ? e << 23 : 0x00400000u); }

// Eight codes of a chunk, the first in the lowest bits.
template <int FMT>
__device__ __forceinline__ uint32_t codes_of(const Chunk<FMT> &ch, float scale) {
  uint32_t q = 0;
  if constexpr (FMT == FMT_F32) {
    float v[8];
    ch.values(v);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], scale, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], scale, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], scale, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], scale, 3);
  } else if constexpr (FMT == FMT_F16) {
    typedef _Float16 pair __attribute__((ext_vector_type(2)));
    const uint32_t *d = ch.raw[0].d;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(pair, d[0]), scale, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(pair, d[1]), scale, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(pair, d[2]), scale, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(pair, d[3]), scale, 3);
  } else {
    typedef __bf16 pair __attribute__((ext_vector_type(2)));
    const uint32_t *d = ch.raw[0].d;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(pair, d[0]), scale, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(pair, d[1]), scale, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(pair, d[2]), scale, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(pair, d[3]), scale, 3);
  }
  return q;
}

// Largest of the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  const uint32_t a = __builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true);  // lanes 1 0 3 2
  v = a > v ? a : v;
  const uint32_t b = __builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true);  // lanes 2 3 0 1
  return b > v ? b : v;
}

}  // namespace tsm
