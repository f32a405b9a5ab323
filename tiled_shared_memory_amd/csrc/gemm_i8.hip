// Int8 products with a scale per token and per channel, the general path:
//   C[i][j] = act(sa[i] * sb[j] * sum_k A[i][k] B[j][k]),  int32 sums (exact).
//
// A workgroup of 8 waves owns a T x T tile of C (T = 128, or 64 when those are
// too few) and walks K in slabs of 128, read into registers two slabs ahead and
// staged through double-buffered LDS.  The waves form two teams of 2 x 2
// (T/2 x T/2 each); a team multiplies one 64-deep half of every slab, and their
// sums, which are exact, meet in LDS at the end.  Two waves per SIMD overlap one
// team's LDS reads with the other's MFMAs where a grid of one workgroup per CU
// would leave each SIMD a single wave (1024 x 4096 x 4096: 29.1 us, 34.7 with one
// team; 2048^3 17.3 us, 21.9).  Bound by the slabs' chain of LDS writes, barrier,
// reads and MFMAs: counters show the MFMAs busy in 20% of the cycles and the LDS in
// 31% with one workgroup per CU (1024 x 4096 x 4096), 34% and 52% with two (8192^3);
// a third of the LDS's cycles are bank conflicts.
//
// Any sizes and any alignment: a thread's 16 codes come with one load at any
// byte address; rows past M or N read the last row (their products are never
// stored); the codes past K are shifted out of the last vectors, so they are
// zeros in both operands.  Odd row addresses cost memory throughput (1000 x 1500:
// 12.4 us at K = 777, 7.9 at K = 768, by the counters 3.3 times the L1 accesses);
// loading the dwords that cover a vector and realigning them took as long (11.7 us;
// 2047^3 28.4 us against 27.4).
// Two slabs ahead; four for up to 128 rows of K >= 4096, where the weights come
// from memory and a CU has one or two workgroups to wait for them (128 x 8192 x
// 8192 30.2 us, 34.3 with two; 64 x 16384 x 8192 38.5, 41.4; 64 x 32768 x 8192
// 60.2, 64.3; but 256 x 8192 x 8192 44.2, 43.0, and 1000 x 1500 x 777 13.6, 12.2).
#include "i8_common.hpp"

namespace tsm {
namespace {

constexpr int kThreads = 512;
constexpr int BK = 128;         // codes per slab
constexpr int PITCH = BK + 16;  // LDS row pitch, so that a fragment read's rows do not all start on one bank

// D: slabs in flight in registers (even: the LDS buffers alternate).  REST: the
// workgroups take the quarters of the 256-tiles that whole_rounds leaves.
template <int T, int FMT, int D, bool REST = false>
__global__ __launch_bounds__(kThreads) void gemm_i8_block_kernel(I8Args p) {
  constexpr int W = T / 2, NB = W / 16;            // wave tile, 16 x 16 blocks per dimension
  constexpr int PR = BK / 16, RP = kThreads / PR;  // vectors per row, rows per pass (64)
  constexpr int V = T / RP;                        // vectors per thread and operand
  __shared__ __attribute__((aligned(16))) char lds[4 * T * PITCH];
  static_assert(8 * (NB / 2) * NB * 1024 <= 4 * T * PITCH, "the teams' sums fit");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int team = wave >> 2, wm = (wave >> 1) & 1, wn = wave & 1;
  int tm, tn;
  int64_t z;
  if constexpr (REST) {
    const int V = tiles_of<2 * T>(p), pid = (int)whole_rounds(V, p.cus) + (int)(blockIdx.x >> 2);
    if (pid >= V) return;  // uniform
    tile_at<2 * T>(p, pid, tile_group(p), z, tm, tn);
    tm = 2 * tm + ((int)blockIdx.x >> 1 & 1);
    tn = 2 * tn + ((int)blockIdx.x & 1);
  } else {
    if (!tile_of<T>(p, 8, z, tm, tn)) return;  // uniform
  }
  const int64_t m0 = (int64_t)tm * T, n0 = (int64_t)tn * T;
  const int64_t M = valid_rows(p, z);
  if (REST && (m0 >= M || n0 >= p.N)) return;  // uniform

  // the scales, long before they are needed: of the rows this wave stores (see the end) and of its columns
  constexpr int H = NB / 2;
  float ca[H], cb[NB][4];
#pragma unroll
  for (int i = 0; i < H; ++i) {
    const int64_t m = m0 + wm * W + (team * H + i) * 16 + (lane & 15);
    ca[i] = p.sa ? p.sa[z * p.stride_sa + (m < M ? m : M - 1)] : 1.f;
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) channel_scales(p, z, n0 + wn * W + j * 16 + 4 * (lane >> 4), cb[j]);

  const int row0 = tid / PR, kc = (tid % PR) * 16;
  const int8_t *ap[V], *bp[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t m = m0 + row0 + RP * v, n = n0 + row0 + RP * v;
    ap[v] = p.A + z * p.strideA + (m < M ? m : M - 1) * p.lda;
    bp[v] = p.B + z * p.strideB + (n < p.N ? n : p.N - 1) * p.ldb;
  }
  // Whole slabs first, their loads without a branch (past the end the last one again), so that the count of loads in
  // flight is known and a wait never takes in younger ones.  K's rest, requested first of all, is multiplied last.
  const int nk = (int)(p.K / BK), rest = (int)(p.K % BK);
  const int64_t kt = p.K - rest + kc;  // this thread's codes of the rest:
  const int64_t kl = kt < p.K - 16 ? kt : p.K - 16;  // loaded from here, inside the row
  u32x4 ra[D][V], rb[D][V], ta[V], tb[V];
  if (p.K >= 16) {
#pragma unroll
    for (int v = 0; v < V; ++v) ta[v] = load16(ap[v] + kl), tb[v] = load16(bp[v] + kl);
  }
  auto fetch = [&](int d, int t) {
    const int64_t k = (int64_t)(t < nk ? t : nk - 1) * BK + kc;
#pragma unroll
    for (int v = 0; v < V; ++v) ra[d][v] = load16(ap[v] + k), rb[d][v] = load16(bp[v] + k);
  };
  auto at_a = [&](int s) { return lds + s * (T * PITCH); };
  auto at_b = [&](int s) { return lds + (2 + s) * (T * PITCH); };
  auto put = [&](int s, int v, u32x4 a, u32x4 b) {
    *reinterpret_cast<u32x4 *>(at_a(s) + (row0 + RP * v) * PITCH + kc) = a;
    *reinterpret_cast<u32x4 *>(at_b(s) + (row0 + RP * v) * PITCH + kc) = b;
  };
  auto commit = [&](int d, int s) {
#pragma unroll
    for (int v = 0; v < V; ++v) put(s, v, ra[d][v], rb[d][v]);
  };

  i32x4 acc[NB][NB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = i32x4{};
  auto multiply = [&](int s) {
    u32x4 fa[NB], fb[NB];
    const int at = (lane & 15) * PITCH + team * 64 + (lane >> 4) * 16;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      fa[i] = *reinterpret_cast<const u32x4 *>(at_a(s) + (wm * W + i * 16) * PITCH + at);
      fb[i] = *reinterpret_cast<const u32x4 *>(at_b(s) + (wn * W + i * 16) * PITCH + at);
    }
    // (B, A): a lane's accumulator holds 4 consecutive columns of one row of C
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = mfma_i8(fb[j], fa[i], acc[i][j]);
  };
  if (nk > 0) {
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(d, d);
    commit(0, 0);
    fetch(0, D);  // registers then hold slabs 1 .. D
    __syncthreads();
    // at slab t: LDS buffer t % 2 holds it, register set s % D slab s for s = t + 1 .. t + D
    for (int t = 0; t < nk; t += D) {
#pragma unroll
      for (int u = 0; u < D; ++u) {
        if (t + u >= nk) break;  // uniform
        multiply(u & 1);
        // (the last slab commits a copy that is not read; the buffer's last readers passed the previous barrier)
        commit((u + 1) % D, (u + 1) & 1);
        fetch((u + 1) % D, t + u + 1 + D);
        __syncthreads();
      }
    }
  }
  if (rest) {  // uniform; every wave is past its reads of both buffers
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (p.K >= 16) {
        const int drop = (int)(kt - kl);
        put(0, v, drop_front(ta[v], drop), drop_front(tb[v], drop));
      } else {
        put(0, v, load_tail(ap[v], kt, p.K), load_tail(bp[v], kt, p.K));
      }
    }
    __syncthreads();
    multiply(0);
    __syncthreads();
  }

  // The teams' sums: team g stores row blocks i with i / (NB / 2) == g; it leaves the others in LDS for the other
  // team and adds what that left.
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
      if (i / H != team)
        *reinterpret_cast<i32x4 *>(lds + (((wave * H + i % H) * NB + j) * 64 + lane) * 16) = acc[i][j];
  __syncthreads();
  const Epilogue ep{p.act, p.slope, false};
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    if (i / H != team) continue;  // uniform
    const int64_t m = m0 + wm * W + i * 16 + (lane & 15);
    if (m >= M) continue;
    char *row = (char *)p.C + (z * p.strideC + m * p.ldc) * fmt_bytes(FMT);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int64_t n = n0 + wn * W + j * 16 + 4 * (lane >> 4);
      if (n >= p.N) continue;
      const i32x4 other = *reinterpret_cast<const i32x4 *>(lds + ((((wave ^ 4) * H + i % H) * NB + j) * 64 + lane) * 16);
      store_i8<FMT>(p, ep, row, n, ca[i % H], cb[j], acc[i][j] + other);
    }
  }
}

template <int T, int D>
hipError_t block_t(const I8Args &p, hipStream_t stream) {
  return over_tiles(p, T, T, kThreads, [&](const I8Args &a, dim3 grid) {
    if (a.fmt == FMT_F32)
      hipLaunchKernelGGL((gemm_i8_block_kernel<T, FMT_F32, D>), grid, dim3(kThreads), 0, stream, a);
    else if (a.fmt == FMT_F16)
      hipLaunchKernelGGL((gemm_i8_block_kernel<T, FMT_F16, D>), grid, dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((gemm_i8_block_kernel<T, FMT_BF16, D>), grid, dim3(kThreads), 0, stream, a);
  });
}

}  // namespace

hipError_t launch_i8_rest(const I8Args &a, hipStream_t stream) {
  const dim3 grid(4 * (kFewTiles - 1)), block(kThreads);
  if (a.fmt == FMT_F32)
    hipLaunchKernelGGL((gemm_i8_block_kernel<128, FMT_F32, 2, true>), grid, block, 0, stream, a);
  else if (a.fmt == FMT_F16)
    hipLaunchKernelGGL((gemm_i8_block_kernel<128, FMT_F16, 2, true>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((gemm_i8_block_kernel<128, FMT_BF16, 2, true>), grid, block, 0, stream, a);
  return hipPeekAtLastError();
}

hipError_t launch_i8_block(const I8Args &p, int tile, hipStream_t stream) {
  if (tile == 128) return block_t<128, 2>(p, stream);
  return p.M <= 128 && p.K >= 4096 ? block_t<64, 4>(p, stream) : block_t<64, 2>(p, stream);
}

}  // namespace tsm
