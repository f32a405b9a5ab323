// Rows to int8 codes with one float32 scale each, for gemm_i8:
//   m = max_c |X[r][c]|,  scale[r] = m / 127,  Q[r][c] = nearest(127 X[r][c] / m), ties to even.
//
// The codes are those of the exact quotient t = 127 x / m.  With inv = 127 / m
// rounded once, x * inv is off by at most t * 2^-24 < 2^-17, so its nearest whole
// number is the right one unless it lies that close to a half:
//  * 16-bit x: t - (n + 1/2) is (254 x - (2n + 1) m) / (2 m).  With x = X 2^a and
//    m = M 2^b, a <= b, X and M whole and below 2^11, that is 0 or at least
//    2^(a-b) / (2 M), i.e. t / (254 X) > t * 2^-19: within t * 2^-21 of a half it
//    is a tie and takes the even neighbour (x = m / 2 is 63.5, common in bf16);
//  * float32 x: the quotient in float64, whose rounding (t * 2^-53) is too small
//    to turn the nearest non-tie (t * 2^-32 away, X below 2^24) into one.
// fma(x, inv, 1.5 * 2^23) rounds to a whole number in one step, its low byte is
// the code, and fma(x, inv, -that) the distance: three operations per element
// and half a maximum; the rare cases run under a branch per 8 elements.
//
// The row stays in registers, so it is read once: bound by memory (16384 rows of
// 4096 bf16 35 us = 5.7 TB/s, 8192 of 8192 32.5 us = 6.2 TB/s; with a division, a
// rounding and a conversion per element and a workgroup per row 50 us).
#include "elems.hpp"
#include "i8_internal.hpp"

namespace tsm {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kInf = 0x7f800000u;
constexpr float kTiny = 0x1p-100f;     // below, 127 / m could overflow: every element takes the exact path
constexpr float kMagic = 12582912.f;    // 1.5 * 2^23: added, the sum's low bits are the rounded whole number
constexpr float kNearHalf = 0.5f - 0x1p-13f;

struct RowScale {
  float m, inv;
  bool ok, tiny;  // ok: neither all zeros nor a NaN or an infinity, whose rows get codes of 0
};

// From the largest magnitude's bits (a NaN's are above infinity's, so either shows).
__device__ __forceinline__ RowScale row_scale(uint32_t top, float *scale) {
  RowScale s;
  s.m = __builtin_bit_cast(float, top);
  s.ok = top != 0 && top < kInf;
  s.tiny = s.m < kTiny;
  s.inv = s.ok && !s.tiny ? 127.f / s.m : 0.f;
  *scale = top < kInf ? s.m / 127.f : __builtin_nanf("");
  return s;
}

__device__ __forceinline__ uint32_t exact_code(float x, float m) {
  return (uint32_t)(int)rint(127.0 * (double)x / (double)m);
}

// Codes of N elements (N a multiple of 4), four to a dword.
template <int FMT, int N>
__device__ __forceinline__ void codes_of(const float (&x)[N], const RowScale &s, uint32_t (&out)[N / 4]) {
  uint32_t q[N];
  float far = 0.f;
  if (s.ok && !s.tiny) {  // the same for the whole row
    float e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float r = fmaf(x[i], s.inv, kMagic);
      q[i] = __builtin_bit_cast(uint32_t, r);
      e[i] = fmaf(x[i], s.inv, kMagic - r);
      far = fmaxf(far, fabsf(e[i]));
    }
    if (far > kNearHalf) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (fabsf(e[i]) <= kNearHalf) continue;
        if constexpr (FMT == FMT_F32)
          q[i] = exact_code(x[i], s.m);
        else if ((q[i] & 1) && fabsf(e[i]) >= 0.5f - fabsf(x[i] * s.inv) * 0x1p-21f)
          q[i] += e[i] > 0.f ? 1 : -1;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = s.ok ? exact_code(x[i], s.m) : 0;
  }
#pragma unroll
  for (int h = 0; h < N / 4; ++h) {
    // the low bytes of four
    const uint32_t lo = __builtin_amdgcn_perm(q[4 * h + 1], q[4 * h], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(q[4 * h + 3], q[4 * h + 2], 0x04000c0cu);
    out[h] = lo | hi;
  }
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const uint32_t o = __shfl_xor(v, d, 64);
    v = o > v ? o : v;
  }
  return v;
}

template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *part) {
  v = wave_max(v);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = max(max(part[0], part[1]), max(part[2], part[3]));
  }
  return v;
}

// This thread's row: group z, row r; false when it lies past the group's rows.
template <int TPR>
__device__ __forceinline__ bool row_at(const QuantArgs &a, int64_t &z, int64_t &r) {
  const int64_t i = a.r0 + (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
  z = 0;
  r = i;
  if (a.groups > 1) {
    z = i / a.R;
    r = i - z * a.R;
  }
  if (z >= a.groups || r >= a.R) return false;
  return !a.rows || r < a.rows[z];
}

// A chunk is 8 elements (16 bytes, or two vectors of float32), kept as loaded; its codes are 8 bytes.
template <int FMT>
struct Chunk {
  static constexpr int V = FMT == FMT_F32 ? 2 : 1;
  Raw16 raw[V];
  __device__ __forceinline__ void load(const char *x, int64_t c) {
#pragma unroll
    for (int i = 0; i < V; ++i) raw[i] = *(const Raw16 *)(x + (c * V + i) * 16);
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

// The row stays in registers: TPR threads hold VPT chunks of 8 each.
template <int FMT, int TPR, int VPT>
__global__ __launch_bounds__(kThreads) void quantize_kernel(QuantArgs a) {
  __shared__ uint32_t part[4];
  int64_t z, r;
  // (TPR = 256: the same for the whole workgroup; else whole waves, which meet no barrier)
  if (!row_at<TPR>(a, z, r)) return;
  constexpr int ES = fmt_bytes(FMT);
  const char *x = (const char *)a.X + (z * a.strideX + r * a.ldx) * ES;
  char *q = (char *)a.Q + z * a.strideQ + r * a.ldq;
  const int lane = threadIdx.x % TPR;
  const int whole = (int)(a.C / 8), rest = (int)(a.C % 8);
  Chunk<FMT> ch[VPT];
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int c = lane + u * TPR;
    if (c < whole) ch[u].load(x, c);
    else ch[u].load_part(x, c, c == whole ? rest : 0);
  }
#pragma unroll
  for (int u = 0; u < VPT; ++u) top = max(top, ch[u].top());
  top = row_max<TPR>(top, part);
  float sc;
  const RowScale s = row_scale(top, &sc);
  if (lane == 0) a.scale[z * a.strideS + r] = sc;
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int c = lane + u * TPR;
    float v[8];
    ch[u].values(v);
    Raw8 o;
    codes_of<FMT, 8>(v, s, o.d);
    if (c < whole) {
      *(Raw8 *)(q + (int64_t)c * 8) = o;
    } else if (c == whole) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < rest) q[(int64_t)c * 8 + i] = (char)(o.d[i >> 2] >> (8 * (i & 3)));
    }
  }
}

// Rows too long for the registers: read twice (the second time from cache).
template <int FMT>
__global__ __launch_bounds__(kThreads) void quantize_long_kernel(QuantArgs a) {
  __shared__ uint32_t part[4];
  int64_t z, r;
  if (!row_at<kThreads>(a, z, r)) return;
  constexpr int ES = fmt_bytes(FMT);
  const char *x = (const char *)a.X + (z * a.strideX + r * a.ldx) * ES;
  char *q = (char *)a.Q + z * a.strideQ + r * a.ldq;
  const int64_t whole = a.C / 8;
  const int rest = (int)(a.C % 8);
  uint32_t top = 0;
  Chunk<FMT> ch;
  for (int64_t c = threadIdx.x; c < whole; c += kThreads) {
    ch.load(x, c);
    top = max(top, ch.top());
  }
  if (threadIdx.x == 0) {
    ch.load_part(x, whole, rest);
    top = max(top, ch.top());
  }
  top = row_max<kThreads>(top, part);
  float sc;
  const RowScale s = row_scale(top, &sc);
  if (threadIdx.x == 0) a.scale[z * a.strideS + r] = sc;
  float v[8];
  Raw8 o;
  for (int64_t c = threadIdx.x; c < whole; c += kThreads) {
    ch.load(x, c);
    ch.values(v);
    codes_of<FMT, 8>(v, s, o.d);
    *(Raw8 *)(q + c * 8) = o;
  }
  if (threadIdx.x == 0) {
    ch.load_part(x, whole, rest);
    ch.values(v);
    codes_of<FMT, 8>(v, s, o.d);
    for (int i = 0; i < rest; ++i) q[whole * 8 + i] = (char)(o.d[i >> 2] >> (8 * (i & 3)));
  }
}

template <int FMT>
hipError_t quantize_fmt(const QuantArgs &base, hipStream_t stream) {
  const int64_t chunks = (base.C + 7) / 8;
  const int64_t rows = base.R * base.groups;
  // a wave per row while its share of the row fits the registers and the rows fill the chip (no barrier); else a
  // workgroup per row
  const bool wave = chunks <= 64 || (chunks <= 512 && rows >= 2048);
  const int64_t per = wave ? 4 : 1;
  const int64_t most = 0xffffffffLL / kThreads * per;  // rows per launch: work-items stay below 2^32
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    QuantArgs a = base;
    a.r0 = r0;
    const int64_t n = rows - r0 < most ? rows - r0 : most;
    const dim3 grid((unsigned)((n + per - 1) / per)), block(kThreads);
    if (wave && chunks <= 64)
      hipLaunchKernelGGL((quantize_kernel<FMT, 64, 1>), grid, block, 0, stream, a);
    else if (wave && chunks <= 256)
      hipLaunchKernelGGL((quantize_kernel<FMT, 64, 4>), grid, block, 0, stream, a);
    else if (wave)
      hipLaunchKernelGGL((quantize_kernel<FMT, 64, 8>), grid, block, 0, stream, a);
    else if (chunks <= 256)
      hipLaunchKernelGGL((quantize_kernel<FMT, 256, 1>), grid, block, 0, stream, a);
    else if (chunks <= 1024)
      hipLaunchKernelGGL((quantize_kernel<FMT, 256, 4>), grid, block, 0, stream, a);
    else if (chunks <= 2048)
      hipLaunchKernelGGL((quantize_kernel<FMT, 256, 8>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((quantize_long_kernel<FMT>), grid, block, 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_quantize(const QuantArgs &a, hipStream_t stream) {
  switch (a.fmt) {
    case FMT_F32:
      return quantize_fmt<FMT_F32>(a, stream);
    case FMT_F16:
      return quantize_fmt<FMT_F16>(a, stream);
    default:
      return quantize_fmt<FMT_BF16>(a, stream);
  }
}

}  // namespace tsm
