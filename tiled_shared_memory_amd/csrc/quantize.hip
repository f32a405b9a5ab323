// Rows to int8 codes with one float32 scale each, for gemm_i8:
//   m = max_c |X[r][c]|,  scale[r] = m / 127,  Q[r][c] = nearest(127 X[r][c] / m), ties to even.
//
// The codes are those of the exact quotient 127 x / m, not of a rounded one:
// t = x * (127 / m) is off by at most 127 * 2^-23 < 2^-16, so where t is
// further than that from a half its nearest whole number is the right one;
// nearer, the sign of 254 |x| - (2n + 1) m decides, whose two products are
// exact in float64 (24 + 8 bits).  (x = m / 2 is a true tie, 63.5, and common
// in bf16.)
#include "elems.hpp"
#include "i8_internal.hpp"

namespace tsm {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kInf = 0x7f800000u;
constexpr float kTiny = 0x1p-100f;  // rows below this are scaled by 2^100 first: 127 / m stays finite

struct RowScale {
  float m, up, inv;
  bool ok;  // false: every code is 0 (the row is all zeros, or holds a NaN or an infinity)
};

// From the largest magnitude's bits (a NaN's are above infinity's, so either shows).
__device__ __forceinline__ RowScale row_scale(uint32_t top, float *scale) {
  RowScale s;
  s.m = __builtin_bit_cast(float, top);
  s.up = s.m < kTiny ? 0x1p100f : 1.f;
  s.ok = top != 0 && top < kInf;
  s.inv = s.ok ? 127.f / (s.m * s.up) : 0.f;
  *scale = top < kInf ? s.m / 127.f : __builtin_nanf("");
  return s;
}

__device__ __forceinline__ int code_of(float x, const RowScale &s) {
  const float t = x * s.up * s.inv;
  float q = rintf(t);
  const float a = fabsf(t);
  const float n = floorf(a);
  if (fabsf(a - n - 0.5f) < 0x1p-14f && s.ok) {
    const double d = 254.0 * fabs((double)x) - (2.0 * n + 1.0) * (double)s.m;
    const bool upper = d > 0 || (d == 0 && ((int)n & 1));
    q = copysignf(upper ? n + 1.f : n, x);
  }
  return s.ok ? (int)q : 0;
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

__device__ __forceinline__ uint32_t mag(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }

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

// Elements per chunk: 8 (16-bit rows: 16 bytes; float32: two vectors), codes 8 bytes.
template <int FMT>
struct Chunk {
  float v[8];
  __device__ __forceinline__ void load(const char *x, int64_t c) {
    if constexpr (FMT == FMT_F32) {
      Vec<FMT> lo, hi;
      lo.unpack(*(const Raw16 *)(x + c * 32));
      hi.unpack(*(const Raw16 *)(x + c * 32 + 16));
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = lo.v[i], v[4 + i] = hi.v[i];
    } else {
      Vec<FMT> w;
      w.unpack(*(const Raw16 *)(x + c * 16));
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = w.v[i];
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
    if (c < whole) {
      ch[u].load(x, c);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        ch[u].v[i] = c == whole && i < rest ? elem_f32<FMT>(elem_bits<FMT>(x, (int64_t)c * 8 + i)) : 0.f;
    }
  }
#pragma unroll
  for (int u = 0; u < VPT; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, mag(ch[u].v[i]));
  top = row_max<TPR>(top, part);
  float sc;
  const RowScale s = row_scale(top, &sc);
  if (lane == 0) a.scale[z * a.strideS + r] = sc;
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int c = lane + u * TPR;
    if (c > whole || (c == whole && !rest)) continue;
    Raw8 o;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t d = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) d |= ((uint32_t)code_of(ch[u].v[4 * h + i], s) & 0xffu) << (8 * i);
      o.d[h] = d;
    }
    if (c < whole) {
      *(Raw8 *)(q + (int64_t)c * 8) = o;
    } else {
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
  uint32_t top = 0;
  for (int64_t c = threadIdx.x; c < whole; c += kThreads) {
    Chunk<FMT> ch;
    ch.load(x, c);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, mag(ch.v[i]));
  }
  const int64_t tail = whole * 8 + threadIdx.x;
  const float xt = tail < a.C ? elem_f32<FMT>(elem_bits<FMT>(x, tail)) : 0.f;
  top = row_max<kThreads>(max(top, mag(xt)), part);
  float sc;
  const RowScale s = row_scale(top, &sc);
  if (threadIdx.x == 0) a.scale[z * a.strideS + r] = sc;
  for (int64_t c = threadIdx.x; c < whole; c += kThreads) {
    Chunk<FMT> ch;
    ch.load(x, c);
    Raw8 o;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t d = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) d |= ((uint32_t)code_of(ch.v[4 * h + i], s) & 0xffu) << (8 * i);
      o.d[h] = d;
    }
    *(Raw8 *)(q + c * 8) = o;
  }
  if (tail < a.C) q[tail] = (char)code_of(xt, s);
}

template <int FMT>
hipError_t quantize_fmt(const QuantArgs &base, hipStream_t stream) {
  const int64_t chunks = (base.C + 7) / 8;
  const int tpr = chunks <= 64 ? 64 : 256;
  const int64_t rows = base.R * base.groups, per = kThreads / tpr;
  const int64_t most = 0xffffffffLL / kThreads * per;  // rows per launch: work-items stay below 2^32
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    QuantArgs a = base;
    a.r0 = r0;
    const int64_t n = rows - r0 < most ? rows - r0 : most;
    const dim3 grid((unsigned)((n + per - 1) / per)), block(kThreads);
    if (tpr == 64)
      hipLaunchKernelGGL((quantize_kernel<FMT, 64, 1>), grid, block, 0, stream, a);
    else if (chunks <= 256)
      hipLaunchKernelGGL((quantize_kernel<FMT, 256, 1>), grid, block, 0, stream, a);
    else if (chunks <= 512)
      hipLaunchKernelGGL((quantize_kernel<FMT, 256, 2>), grid, block, 0, stream, a);
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
