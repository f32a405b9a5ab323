// Int8 products with a scale per token and per channel, the general path:
//   C[i][j] = act(sa[i] * sb[j] * sum_k A[i][k] B[j][k]),  int32 sums (exact).
//
// A 256-thread workgroup owns a T x T tile of C and walks K in slabs of 128,
// each operand's slab read into registers one slab ahead and staged through
// double-buffered LDS.  Any sizes and any alignment: a thread's 16 codes come
// with one load at any byte address; rows past M or N read the last row (their
// products are never stored); the codes past K are shifted out of the last
// vector (make_tail), so they are zeros in both operands.
#include "i8_common.hpp"

namespace tsm {
namespace {

constexpr int kThreads = 256;
constexpr int BK = 128;           // codes per slab
constexpr int PITCH = BK + 16;    // LDS row pitch: 16 rows of one fragment read fall on distinct banks

template <int T, int FMT>
__global__ __launch_bounds__(kThreads) void gemm_i8_block_kernel(I8Args p) {
  constexpr int W = T / 2, NB = W / 16;       // wave tile, 16 x 16 blocks per dimension
  constexpr int V = T * (BK / 16) / kThreads;  // vectors per thread and operand
  __shared__ __attribute__((aligned(16))) char sA[2][T * PITCH], sB[2][T * PITCH];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
  int tm, tn;
  int64_t z;
  if (!i8_tile_of<T>(p, 8, z, tm, tn)) return;  // uniform
  const int64_t m0 = (int64_t)tm * T, n0 = (int64_t)tn * T;
  const int64_t M = i8_rows(p, z);

  const int row0 = tid >> 3, kc = (tid & 7) * 16;  // 8 vectors per row, 32 rows per pass
  const int8_t *ap[V], *bp[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t m = m0 + row0 + 32 * v, n = n0 + row0 + 32 * v;
    ap[v] = p.A + z * p.strideA + (m < M ? m : M - 1) * p.lda;
    bp[v] = p.B + z * p.strideB + (n < p.N ? n : p.N - 1) * p.ldb;
  }
  u32x4 ra[V], rb[V];
  auto fetch = [&](int64_t k) {
    k += kc;
    if (k + 16 <= p.K) {
#pragma unroll
      for (int v = 0; v < V; ++v) ra[v] = load16(ap[v] + k), rb[v] = load16(bp[v] + k);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) ra[v] = load_tail(ap[v], k, p.K), rb[v] = load_tail(bp[v], k, p.K);
    }
  };
  auto commit = [&](int s) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      *reinterpret_cast<u32x4 *>(sA[s] + (row0 + 32 * v) * PITCH + kc) = ra[v];
      *reinterpret_cast<u32x4 *>(sB[s] + (row0 + 32 * v) * PITCH + kc) = rb[v];
    }
  };

  i32x4 acc[NB][NB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = i32x4{};
  const int nk = (int)((p.K + BK - 1) / BK);
  if (nk > 0) {
    fetch(0);
    commit(0);
    if (nk > 1) fetch(BK);
  }
  __syncthreads();
  for (int t = 0; t < nk; ++t) {
    const char *a = sA[t & 1], *b = sB[t & 1];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      u32x4 fa[NB], fb[NB];
      const int at = (lane & 15) * PITCH + ks * 64 + (lane >> 4) * 16;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        fa[i] = *reinterpret_cast<const u32x4 *>(a + (wm * W + i * 16) * PITCH + at);
        fb[i] = *reinterpret_cast<const u32x4 *>(b + (wn * W + i * 16) * PITCH + at);
      }
      // (B, A): a lane's accumulator holds 4 consecutive columns of one row of C
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = mfma_i8(fb[j], fa[i], acc[i][j]);
    }
    if (t + 1 < nk) {
      commit((t + 1) & 1);  // its last readers passed the previous barrier
      if (t + 2 < nk) fetch((int64_t)(t + 2) * BK);
    }
    __syncthreads();
  }

  const Epilogue ep{p.act, p.slope, false};
  constexpr int ES = fmt_bytes(FMT);
  const float *sa = p.sa ? p.sa + z * p.stride_sa : nullptr, *sb = p.sb ? p.sb + z * p.stride_sb : nullptr;
  float cb[NB][4];
#pragma unroll
  for (int j = 0; j < NB; ++j) channel_scales(p, sb, n0 + wn * W + j * 16 + 4 * (lane >> 4), cb[j]);
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int64_t m = m0 + wm * W + i * 16 + (lane & 15);
    if (m >= M) continue;
    const float ca = sa ? sa[m] : 1.f;
    char *row = (char *)p.C + (z * p.strideC + m * p.ldc) * ES;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int64_t n = n0 + wn * W + j * 16 + 4 * (lane >> 4);
      if (n < p.N) store_i8<FMT>(p, ep, row, n, ca, cb[j], acc[i][j]);
    }
  }
}

template <int T>
hipError_t block_t(const I8Args &p, hipStream_t stream) {
  return over_tiles(p, T, T, kThreads, [&](const I8Args &a, dim3 grid) {
    if (a.fmt == FMT_F32)
      hipLaunchKernelGGL((gemm_i8_block_kernel<T, FMT_F32>), grid, dim3(kThreads), 0, stream, a);
    else if (a.fmt == FMT_F16)
      hipLaunchKernelGGL((gemm_i8_block_kernel<T, FMT_F16>), grid, dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((gemm_i8_block_kernel<T, FMT_BF16>), grid, dim3(kThreads), 0, stream, a);
  });
}

}  // namespace

hipError_t launch_i8_block(const I8Args &p, int tile, hipStream_t stream) {
  return tile == 128 ? block_t<128>(p, stream) : block_t<64>(p, stream);
}

}  // namespace tsm
