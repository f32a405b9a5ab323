// Rows to microscaled 4-bit codes and back:
//   E = max(0, the biased exponent of max_k |X[r][k]| over a block of 32, less 2),  scale 2^(E - 127),
//   code = nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 to |X| / scale, ties to the even code, 6 above 6; sign beside it.
//
// The quotient lies below 8, and is exact, since the scale is a power of two: the
// conversion instruction divides and rounds in one step, with the scale of E = 0,
// 2^-127, given as that subnormal number.  A block with a NaN or an infinity gets
// E = 255 and codes of 0.
//
// Bound by memory: 16384 x 4096 bf16 29.4 us (5.8 TB/s), back 27-31 (5.7-6.4); columns of
// 1500 x 8195 float32 14.5 (3.8: 792 workgroups, 3 per CU), back 12.7 (4.3).
#include "mx4_codes.hpp"
#include "mx4_internal.hpp"

namespace tsm {
namespace {

constexpr int kThreads = 256;

// The group and row of pair i; false when it lies past the group's rows.
__device__ __forceinline__ bool row_at(const Mx4QuantArgs &a, int64_t i, int64_t &z, int64_t &r) {
  z = 0;
  r = i;
  if (a.groups > 1) {
    z = i / a.R;
    r = i - z * a.R;
  }
  if (z >= a.groups || r >= a.R) return false;
  return !a.rows || r < a.rows[z];
}

// Chunks of 8 per thread of the quantisation and the way back (us, 4 | 2: 16384 x 4096 bf16 29.5 | 31.9, float32 57.4 |
// 55.5; back to bf16 33.3 | 31.2, to float32 67 | 59).
constexpr int per_of(int fmt) { return fmt == FMT_F32 ? 2 : 4; }
constexpr int kBackPer = 2;

// Values of this many bytes and more are read past the caches, which could not hold them for the next reader anyway (us,
// through the caches | past them: 16384 x 4096 bf16 31.7 | 29.5; 4096 x 4096, in the cache from the kernel before, 8.7 |
// 9.7).
constexpr int64_t kOnceBytes = (int64_t)128 << 20;

// TPR threads (a power of two) per row and segment, kPer chunks each; four lanes hold a block.
template <int FMT, int TPR, int kPer, bool ONCE>
__global__ __launch_bounds__(kThreads) void quantize_mx4_kernel(Mx4QuantArgs a) {
  const int64_t g = (int64_t)(blockIdx.x / (uint32_t)a.segs);
  const int seg = (int)(blockIdx.x % (uint32_t)a.segs);
  int64_t z, r;
  if (!row_at(a, a.r0 + g * (kThreads / TPR) + threadIdx.x / TPR, z, r)) return;  // whole quads
  constexpr int ES = fmt_bytes(FMT);
  const char *x = (const char *)a.X + (z * a.strideX + r * a.ldx) * ES;
  uint8_t *const q = a.Q + z * a.strideQ + r * a.ldq, *const s = a.S + z * a.strideS + r * a.lds;
  const int64_t whole = a.C / 8, c0 = (int64_t)seg * (TPR * kPer) + threadIdx.x % TPR;
  const int rest = (int)(a.C % 8);
  Chunk<FMT> ch[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int64_t c = c0 + u * TPR;
    if (c < whole) {
      if constexpr (ONCE)
        ch[u].load_once(x, c);
      else
        ch[u].load(x, c);
    } else {
      ch[u] = Chunk<FMT>{};
      if (c == whole && rest) ch[u].load_part(x, c, rest);
    }
  }
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int64_t c = c0 + u * TPR;
    const uint32_t e = scale_byte(quad_max(ch[u].top()));
    const uint32_t codes = e == 255u ? 0u : codes_of<FMT>(ch[u], scale_of(e));
    if (c < whole) {
      reinterpret_cast<Raw4 *>(q + c * 4)->d = codes;
    } else if (c == whole) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (2 * i < rest) q[c * 4 + i] = (uint8_t)(codes >> (8 * i));
    }
    if ((c & 3) == 0 && c * 8 < a.C) s[c >> 2] = (uint8_t)e;
  }
}

// Blocks along the dimension whose elements lie ldx apart: X[c * ldx + r].  A
// workgroup takes 64 rows (of codes) by 8 blocks, so that a wave's loads are 64
// neighbours and the codes leave, through LDS, in runs of 128 bytes.
constexpr int kColRows = 64, kColBlocks = 8;

template <int FMT>
__global__ __launch_bounds__(kThreads) void quantize_mx4_columns_kernel(Mx4QuantArgs a) {
  constexpr int ES = fmt_bytes(FMT);
  __shared__ __attribute__((aligned(16))) uint8_t codes[kColRows * (kColBlocks * 16 + 16)];
  __shared__ uint8_t scales[kColRows * kColBlocks];
  constexpr int PITCH = kColBlocks * 16 + 16;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t tiles = (a.R + kColRows - 1) / kColRows;
  const int64_t g = a.r0 + (int64_t)(blockIdx.x / (uint32_t)a.segs);
  const int64_t b0 = (int64_t)(blockIdx.x % (uint32_t)a.segs) * kColBlocks;
  const int64_t z = g / tiles, r0 = (g - z * tiles) * kColRows;
  int64_t R = a.R;
  if (a.rows) R = a.rows[z] < R ? a.rows[z] : R;
  if (r0 >= R) return;  // uniform
  const int64_t r = r0 + lane < R ? r0 + lane : R - 1;
  const char *x = (const char *)a.X + (z * a.strideX + r) * ES;
#pragma unroll
  for (int u = 0; u < kColBlocks / 4; ++u) {
    const int blk = wave + 4 * u;
    const int64_t c0 = (b0 + blk) * kMxBlock;
    uint32_t w[kMxBlock];
    if (c0 + kMxBlock <= a.C) {
#pragma unroll
      for (int i = 0; i < kMxBlock; ++i) w[i] = elem_bits<FMT>(x, (c0 + i) * a.ldx);
    } else {
#pragma unroll
      for (int i = 0; i < kMxBlock; ++i) w[i] = c0 + i < a.C ? elem_bits<FMT>(x, (c0 + i) * a.ldx) : 0u;
    }
    float v[kMxBlock];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kMxBlock; ++i) {
      v[i] = elem_f32<FMT>(w[i]);
      const uint32_t m = __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu;
      top = m > top ? m : top;
    }
    const uint32_t e = scale_byte(top);
    const float scale = scale_of(e);
    uint32_t out[4] = {};
    if (e != 255u) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t q = 0;
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[8 * h + 0], v[8 * h + 1], scale, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[8 * h + 2], v[8 * h + 3], scale, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[8 * h + 4], v[8 * h + 5], scale, 2);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[8 * h + 6], v[8 * h + 7], scale, 3);
        out[h] = q;
      }
    }
    *reinterpret_cast<Raw16 *>(codes + lane * PITCH + blk * 16) = Raw16{{out[0], out[1], out[2], out[3]}};
    scales[lane * kColBlocks + blk] = (uint8_t)e;
  }
  __syncthreads();
  const int64_t kb = (a.C + 1) / 2, nb = (a.C + kMxBlock - 1) / kMxBlock;
  for (int i = threadIdx.x; i < kColRows * kColBlocks; i += kThreads) {
    const int row = i / kColBlocks, blk = i % kColBlocks;
    if (r0 + row >= R || b0 + blk >= nb) continue;
    const int64_t at = z * a.strideQ + (r0 + row) * a.ldq + (b0 + blk) * 16;
    const uint8_t *from = codes + row * PITCH + blk * 16;
    const int64_t left = kb - (b0 + blk) * 16;
    if (left >= 16) {
      *reinterpret_cast<Raw16 *>(a.Q + at) = *reinterpret_cast<const Raw16 *>(from);
    } else {
      for (int j = 0; j < (int)left; ++j) a.Q[at + j] = from[j];
    }
    a.S[z * a.strideS + (r0 + row) * a.lds + b0 + blk] = scales[i];
  }
}

// Eight values of codes and a scale byte; of block 255 NaN.
__device__ __forceinline__ void values_of(uint32_t codes, uint32_t e, float (&v)[8]) {
  const float scale = scale_of(e);
  typedef float pair __attribute__((ext_vector_type(2)));
  pair p[4];
  p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 0);
  p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 1);
  p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 2);
  p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 3);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = e == 255u ? __builtin_nanf("") : p[i / 2][i % 2];
}

template <int FMT, int TPR, int kPer>
__global__ __launch_bounds__(kThreads) void dequantize_mx4_kernel(Mx4QuantArgs a) {
  const int64_t g = (int64_t)(blockIdx.x / (uint32_t)a.segs);
  const int seg = (int)(blockIdx.x % (uint32_t)a.segs);
  int64_t z, r;
  if (!row_at(a, a.r0 + g * (kThreads / TPR) + threadIdx.x / TPR, z, r)) return;
  constexpr int ES = fmt_bytes(FMT);
  char *const y = (char *)const_cast<void *>(a.X) + (z * a.strideX + r * a.ldx) * ES;
  const uint8_t *const q = a.Q + z * a.strideQ + r * a.ldq, *const s = a.S + z * a.strideS + r * a.lds;
  const int64_t whole = a.C / 8, c0 = (int64_t)seg * (TPR * kPer) + threadIdx.x % TPR;
  const int rest = (int)(a.C % 8);
  uint32_t codes[kPer], e[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int64_t c = c0 + u * TPR;
    codes[u] = e[u] = 0;
    if (c < whole) {
      codes[u] = reinterpret_cast<const Raw4 *>(q + c * 4)->d;
    } else if (c == whole) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (2 * i < rest) codes[u] |= (uint32_t)q[c * 4 + i] << (8 * i);
    }
    if (c * 8 < a.C) e[u] = s[c >> 2];
  }
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int64_t c = c0 + u * TPR;
    float v[8];
    values_of(codes[u], e[u], v);
    if (c < whole) {
      constexpr int N = Vec<FMT>::N;
#pragma unroll
      for (int h = 0; h < 8 / N; ++h) {
        Vec<FMT> o;
#pragma unroll
        for (int i = 0; i < N; ++i) o.v[i] = v[h * N + i];
        *reinterpret_cast<Raw16 *>(y + (c * 8 + h * N) * ES) = o.pack();
      }
    } else if (c == whole) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < rest) put_bits<FMT>(y, c * 8 + i, f32_elem<FMT>(v[i]));
    }
  }
}

// f(threads per row) over launches whose work-items stay below 2^32: rows x segments of TPR * kPer chunks.
template <class F>
hipError_t over_rows(const Mx4QuantArgs &base, int kPer, F &&launch) {
  const int64_t chunks = (base.C + 7) / 8, rows = base.R * base.groups;
  const int tpr = chunks <= 16 * kPer ? 16 : 64;
  const int64_t segs = (chunks + tpr * kPer - 1) / (tpr * kPer), per = kThreads / tpr;
  const int64_t most = 0xffffffffLL / kThreads / segs * per;
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    Mx4QuantArgs a = base;
    a.r0 = r0;
    a.segs = (int32_t)segs;
    const int64_t n = rows - r0 < most ? rows - r0 : most;
    launch(a, tpr, dim3((unsigned)((n + per - 1) / per * segs)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int FMT, bool ONCE>
hipError_t quantize_rows(const Mx4QuantArgs &base, hipStream_t stream) {
  return over_rows(base, per_of(FMT), [&](const Mx4QuantArgs &a, int tpr, dim3 grid) {
    if (tpr == 16)
      hipLaunchKernelGGL((quantize_mx4_kernel<FMT, 16, per_of(FMT), ONCE>), grid, dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((quantize_mx4_kernel<FMT, 64, per_of(FMT), ONCE>), grid, dim3(kThreads), 0, stream, a);
  });
}

template <int FMT>
hipError_t quantize_rows(const Mx4QuantArgs &a, hipStream_t stream) {
  // (in double: the sizes' product may pass 64 bits where a stride of 0 lets groups share a matrix)
  const double bytes = (double)a.groups * (double)a.R * (double)a.C * fmt_bytes(FMT);
  return bytes >= (double)kOnceBytes ? quantize_rows<FMT, true>(a, stream) : quantize_rows<FMT, false>(a, stream);
}

template <int FMT>
hipError_t quantize_columns(const Mx4QuantArgs &base, hipStream_t stream) {
  const int64_t segs = (base.C + kColBlocks * kMxBlock - 1) / (kColBlocks * kMxBlock);
  const int64_t tiles = (base.R + kColRows - 1) / kColRows * base.groups;
  const int64_t most = 0xffffffffLL / kThreads / segs;
  for (int64_t t0 = 0; t0 < tiles; t0 += most) {
    Mx4QuantArgs a = base;
    a.r0 = t0;
    a.segs = (int32_t)segs;
    const int64_t n = tiles - t0 < most ? tiles - t0 : most;
    hipLaunchKernelGGL((quantize_mx4_columns_kernel<FMT>), dim3((unsigned)(n * segs)), dim3(kThreads), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int FMT>
hipError_t dequantize_rows(const Mx4QuantArgs &base, hipStream_t stream) {
  return over_rows(base, kBackPer, [&](const Mx4QuantArgs &a, int tpr, dim3 grid) {
    if (tpr == 16)
      hipLaunchKernelGGL((dequantize_mx4_kernel<FMT, 16, kBackPer>), grid, dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((dequantize_mx4_kernel<FMT, 64, kBackPer>), grid, dim3(kThreads), 0, stream, a);
  });
}

}  // namespace

hipError_t launch_quantize_mx4(const Mx4QuantArgs &a, bool columns, hipStream_t stream) {
  switch (a.fmt) {
    case FMT_F32:
      return columns ? quantize_columns<FMT_F32>(a, stream) : quantize_rows<FMT_F32>(a, stream);
    case FMT_F16:
      return columns ? quantize_columns<FMT_F16>(a, stream) : quantize_rows<FMT_F16>(a, stream);
    default:
      return columns ? quantize_columns<FMT_BF16>(a, stream) : quantize_rows<FMT_BF16>(a, stream);
  }
}

hipError_t launch_dequantize_mx4(const Mx4QuantArgs &a, hipStream_t stream) {
  switch (a.fmt) {
    case FMT_F32:
      return dequantize_rows<FMT_F32>(a, stream);
    case FMT_F16:
      return dequantize_rows<FMT_F16>(a, stream);
    default:
      return dequantize_rows<FMT_BF16>(a, stream);
  }
}

}  // namespace tsm
