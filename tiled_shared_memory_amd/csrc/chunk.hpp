// Eight elements of a row, as the quantisations read them.
#pragma once

#include "elems.hpp"

namespace tsm {

// A chunk is 8 elements (16 bytes, or two vectors of float32), kept as loaded; its codes are 8 bytes.
template <int FMT>
struct Chunk {
  static constexpr int V = FMT == FMT_F32 ? 2 : 1;
  Raw16 raw[V];
  __device__ __forceinline__ void load(const char *x, int64_t c) {
#pragma unroll
    for (int i = 0; i < V; ++i) raw[i] = *(const Raw16 *)(x + (c * V + i) * 16);
  }
  // the same of what is read once (non-temporal)
  __device__ __forceinline__ void load_once(const char *x, int64_t c) {
    typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const u32x4_any v = __builtin_nontemporal_load((const u32x4_any *)(x + (c * V + i) * 16));
      raw[i] = Raw16{{v[0], v[1], v[2], v[3]}};
    }
  }
  // the first n elements at x, zeros behind them
  __device__ __forceinline__ void load_part(const char *x, int64_t c, int n) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = i < n ? elem_bits<FMT>(x, c * 8 + i) : 0u;
#pragma unroll
    for (int i = 0; i < 4 * V; ++i)
      raw[i / 4].d[i % 4] = FMT == FMT_F32 ? w[i] : w[(2 * i) % 8] | (w[(2 * i + 1) % 8] << 16);
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      Vec<FMT> u;
      u.unpack(raw[i]);
#pragma unroll
      for (int j = 0; j < Vec<FMT>::N; ++j) v[i * Vec<FMT>::N + j] = u.v[j];
    }
  }
  // bits of the largest magnitude as float32 (magnitudes of every format order like their bits)
  __device__ __forceinline__ uint32_t top() const {
    if constexpr (FMT == FMT_F32) {
      uint32_t t = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) t = max(t, raw[i / 4].d[i % 4] & 0x7fffffffu);
      return t;
    } else {
      uint32_t lo = 0, hi = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo = max(lo, raw[0].d[i] & 0x7fffu);
        hi = max(hi, raw[0].d[i] & 0x7fff0000u);
      }
      return __builtin_bit_cast(uint32_t, elem_f32<FMT>(max(lo, hi >> 16)));
    }
  }
};

struct __attribute__((packed, aligned(1))) Raw8 {
  uint32_t d[2];
};
struct __attribute__((packed, aligned(1))) Raw4 {
  uint32_t d;
};

}  // namespace tsm
