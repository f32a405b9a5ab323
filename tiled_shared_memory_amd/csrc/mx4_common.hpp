// Pieces shared by the microscaled 4-bit product kernels.
#pragma once

#include "codes.hpp"
#include "mx4_internal.hpp"

namespace tsm {

// v_mfma_scale_f32_16x16x128_f8f6f4 on 4-bit codes (format 4): D(16x16) += A(16x128) * B(128x16), 32 codes per lane
// and operand: row (column) lane % 16, block lane / 16, whose scale is byte O of the lane's scale register.  Which
// block of K a lane's codes are does not matter as long as both operands and their scales agree.  D as for the
// 16x16x32 forms (mfma.hpp).  A scale byte of 255 makes the row NaN, with codes of 0 too.
template <int OA, int OB>
__device__ __forceinline__ f32x4 mfma_mx4(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x4 c) {
  typedef int i32x8 __attribute__((ext_vector_type(8)));
  const i32x8 va = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 vb = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, c, 4, 4, OA, (int)sa, OB, (int)sb);
}

// v_mfma_scale_f32_32x32x64_f8f6f4: D(32x32) += A(32x64) * B(64x32), row (column) lane % 32, block lane / 32, byte O of
// both scale registers.  D as for the 32x32x16 forms.
template <int O>
__device__ __forceinline__ f32x16 mfma_mx4_32(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x16 c) {
  typedef int i32x8 __attribute__((ext_vector_type(8)));
  const i32x8 va = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 vb = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(va, vb, c, 4, 4, O, (int)sa, O, (int)sb);
}

// Fewer than this many 256-tiles left over from whole rounds of the CUs run as 64-tiles in a second launch (whole
// products, in us, two launches | another round: 4112 x 4096 x 4096, 16 tiles left, 51 | 59; 4608 rows, 32 left, 56.5 |
// 59.5; 5120 rows, 64 left, 71 | 59.9).
constexpr int kFewMx4Tiles = 33;

// f(0) .. f(N - 1) with constants.
template <int I>
struct Const {
  static constexpr int value = I;
  constexpr operator int() const { return I; }
};
template <int N, int I = 0, class F>
__device__ __forceinline__ void unrolled(F &&f) {
  if constexpr (I < N) {
    f(Const<I>{});
    unrolled<N, I + 1>(f);
  }
}

// Codes of a vector of 16 bytes from byte `at` of a row of K elements: an odd K's last byte holds one code, and what
// is in its high half must not count.
__device__ __forceinline__ u32x4 without_odd(u32x4 v, int64_t at, int64_t K) {
  const int64_t i = K / 2 - at;
  if ((K & 1) && i >= 0 && i < 16) {
#pragma unroll
    for (int d = 0; d < 4; ++d)
      if (i / 4 == d) v[d] &= ~(0xf0u << (8 * (i & 3)));
  }
  return v;
}

// Two float32 values to 16-bit ones side by side, to nearest even (bf16: one instruction for both).
template <int FMT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  if constexpr (FMT == FMT_BF16) {
    typedef __bf16 pair __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), pair));
  } else {
    typedef _Float16 pair __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), pair));
  }
}

// The kernel's arguments, read again for each tile: held in scalar registers through the loop they would spill.
__device__ __forceinline__ Mx4Args args_again() {
  typedef const __attribute__((address_space(4))) Mx4Args *At;
  At p = (At)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const Mx4Args *)p;
}

// Four results of one row of C, columns n .. n+3 (n < N): activation, rounding, store.
template <int FMT>
__device__ __forceinline__ void store_mx4(const Mx4Args &p, const Epilogue &ep, char *row, int64_t n, f32x4 acc) {
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = act_codes(ep, acc[i]);
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

}  // namespace tsm
