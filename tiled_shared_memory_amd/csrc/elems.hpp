// Elements of the row operators (quantisation, expert routing): formats, and
// vectors of 16 bytes read and written at any alignment of the element.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tsm {

// Element formats, the numbers of TSM_F32 .. TSM_I8.
enum Fmt { FMT_F32 = 0, FMT_F16 = 1, FMT_BF16 = 2, FMT_I8 = 3 };

constexpr int fmt_bytes(int f) { return f == FMT_F32 ? 4 : f == FMT_I8 ? 1 : 2; }

// 16 bytes at any address: gfx950 global memory takes vector accesses at any
// byte alignment, so odd leading dimensions need no path of their own.
struct __attribute__((packed, aligned(1))) Raw16 {
  uint32_t d[4];
};
static_assert(sizeof(Raw16) == 16, "");

// The same past the caches (read or written once).
__device__ __forceinline__ Raw16 load_once(const char *p) {
  typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(1)));
  const vec v = __builtin_nontemporal_load((const vec *)p);
  return Raw16{{v[0], v[1], v[2], v[3]}};
}
__device__ __forceinline__ void store_once(char *p, const Raw16 &r) {
  typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(1)));
  __builtin_nontemporal_store(vec{r.d[0], r.d[1], r.d[2], r.d[3]}, (vec *)p);
}

template <bool ONCE>
__device__ __forceinline__ Raw16 load_vec(const char *p) {
  if constexpr (ONCE) return load_once(p);
  return *(const Raw16 *)p;
}
template <bool ONCE>
__device__ __forceinline__ void store_vec(char *p, const Raw16 &r) {
  if constexpr (ONCE)
    store_once(p, r);
  else
    *(Raw16 *)p = r;
}

template <int FMT>
__device__ __forceinline__ float elem_f32(uint32_t bits) {
  if constexpr (FMT == FMT_F32) return __builtin_bit_cast(float, bits);
  if constexpr (FMT == FMT_F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  return __builtin_bit_cast(float, bits << 16);
}

// float32 -> element bits, to nearest even.
template <int FMT>
__device__ __forceinline__ uint32_t f32_elem(float v) {
  if constexpr (FMT == FMT_F32) return __builtin_bit_cast(uint32_t, v);
  if constexpr (FMT == FMT_F16) return __builtin_bit_cast(uint16_t, (_Float16)v);
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// Elements of a 16-byte vector as float32, and back.
template <int FMT>
struct Vec {
  static constexpr int N = 16 / fmt_bytes(FMT);
  float v[N];
  __device__ __forceinline__ void unpack(const Raw16 &r) {
    if constexpr (FMT == FMT_F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = elem_f32<FMT>(r.d[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = elem_f32<FMT>(r.d[i] & 0xffffu);
        v[2 * i + 1] = elem_f32<FMT>(r.d[i] >> 16);
      }
    }
  }
  __device__ __forceinline__ Raw16 pack() const {
    Raw16 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (FMT == FMT_F32)
        r.d[i] = f32_elem<FMT>(v[i]);
      else
        r.d[i] = f32_elem<FMT>(v[2 * i]) | (f32_elem<FMT>(v[2 * i + 1]) << 16);
    }
    return r;
  }
};

// Bits of element i of an array of the format.
template <int FMT>
__device__ __forceinline__ uint32_t elem_bits(const void *p, int64_t i) {
  if constexpr (fmt_bytes(FMT) == 4) return ((const uint32_t *)p)[i];
  if constexpr (fmt_bytes(FMT) == 2) return ((const uint16_t *)p)[i];
  return ((const uint8_t *)p)[i];
}
template <int FMT>
__device__ __forceinline__ void put_bits(void *p, int64_t i, uint32_t bits) {
  if constexpr (fmt_bytes(FMT) == 4)
    ((uint32_t *)p)[i] = bits;
  else if constexpr (fmt_bytes(FMT) == 2)
    ((uint16_t *)p)[i] = (uint16_t)bits;
  else
    ((uint8_t *)p)[i] = (uint8_t)bits;
}

// Butterfly over the 64 lanes of a wave, a fixed order: every lane ends with the sum.
__device__ __forceinline__ float wave_add(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

}  // namespace tsm
