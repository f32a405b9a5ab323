// Products of microscaled 4-bit codes, the general path:
//   C[i][j] = act(sum_k A[i][k] B[j][k]),  float32 sums; the matrix instruction applies the blocks' scales.
//
// The blocking is that of the general int8 kernel (gemm_i8.hip): a workgroup of 8
// waves owns a T x T tile of C (T = 128, or 64 when those are too few) and walks K
// in slabs of 256 elements (128 bytes of a row), read into registers two slabs
// ahead and staged through double-buffered LDS.  The waves form two teams of 2 x 2
// (T/2 x T/2 each); a team multiplies one half of every slab, and their sums meet
// in LDS at the end.
//
// A thread's 16 bytes of codes are one block, so its scale byte comes with them.
// In LDS the scale bytes of a wave's 16-row blocks stand beside each other, so that
// one read gives a lane all of an operand's scales of a slab and the matrix
// instruction picks the block's byte.
//
// Measured (us): 1000 x 1500 x 777 with float32 out 11.5; 2000 x 2000 x 2001 17.9; 4000 x
// 5000 x 3001 93-113, 1.1-1.3 PFLOP/s.  Rows at odd addresses cost most: a 16-byte load of
// 64 lanes there takes 72 cycles of L1, of rows at 4 bytes 20, and L1 is busy all the time
// (at 16 bytes 4000 x 5000 x 3008 takes 85).
//
// Any sizes and any alignment, as there: rows past M or N read the last row (their
// products are never stored), and the codes past K are shifted out of the last
// vectors, so they are zeros in both operands.
#include "mx4_common.hpp"

namespace tsm {
namespace {

constexpr int kThreads = 512;
constexpr int BK = 128;         // bytes of codes per slab and row
constexpr int BB = BK / 16;     // blocks of them
constexpr int PITCH = BK + 16;  // LDS row pitch, so that a fragment read's rows do not all start on one bank

// D: slabs in flight in registers (even: the LDS buffers alternate).
template <int T, int FMT, int D>
__global__ __launch_bounds__(kThreads) void gemm_mx4_block_kernel(Mx4Args p) {
  constexpr int W = T / 2, NB = W / 16;      // wave tile, 16 x 16 blocks per dimension
  constexpr int RP = kThreads / BB;          // rows per pass (64)
  constexpr int V = T / RP;                  // vectors per thread and operand
  typedef std::conditional_t<NB == 4, uint32_t, uint16_t> Scales;  // a lane's scales of a wave tile's row blocks
  static_assert(sizeof(Scales) == NB, "a byte for each row block");
  __shared__ __attribute__((aligned(16))) char lds[4 * T * PITCH];
  __shared__ __attribute__((aligned(16))) uint8_t scales[2][2][T * BB];
  static_assert(8 * (NB / 2) * NB * 1024 <= 4 * T * PITCH, "the teams' sums fit");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int team = wave >> 2, wm = (wave >> 1) & 1, wn = wave & 1;
  int tm, tn;
  int64_t z;
  if (!tile_of<T>(p, 8, z, tm, tn)) return;  // uniform
  const int64_t m0 = (int64_t)tm * T, n0 = (int64_t)tn * T;
  const int64_t M = valid_rows(p, z);

  constexpr int H = NB / 2;
  const int row0 = tid / BB, chunk = tid % BB, kc = chunk * 16;
  const int8_t *ap[V], *bp[V];
  const uint8_t *asp[V], *bsp[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t m = m0 + row0 + RP * v, n = n0 + row0 + RP * v;
    const int64_t mr = m < M ? m : M - 1, nr = n < p.N ? n : p.N - 1;
    ap[v] = p.A + z * p.strideA + mr * p.lda;
    bp[v] = p.B + z * p.strideB + nr * p.ldb;
    asp[v] = p.SA + z * p.strideSA + mr * p.ldsa;
    bsp[v] = p.SB + z * p.strideSB + nr * p.ldsb;
  }
  // Whole slabs first, their loads without a branch (past the end the last one again); K's rest, requested first of
  // all, is multiplied last.
  const int nk = (int)(p.K / (2 * BK));
  const bool rest = p.K % (2 * BK) != 0;
  const int64_t kt = (int64_t)nk * BK + kc;            // this thread's codes of the rest:
  const int64_t kl = kt < p.kb - 16 ? kt : p.kb - 16;  // loaded from here, inside the row
  u32x4 ra[D][V], rb[D][V], ta[V], tb[V];
  uint8_t sa[D][V], sb[D][V], tsa[V], tsb[V];
  if (rest) {
    const int64_t blk = (int64_t)nk * BB + chunk;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (p.kb >= 16) ta[v] = load16(ap[v] + kl), tb[v] = load16(bp[v] + kl);
      // (a block past K has codes of 0, and no NaN)
      tsa[v] = blk < p.nb ? asp[v][blk] : 0;
      tsb[v] = blk < p.nb ? bsp[v][blk] : 0;
    }
  }
  auto fetch = [&](int d, int t) {
    const int64_t s = t < nk ? t : nk - 1, k = s * BK + kc, e = s * BB + chunk;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      ra[d][v] = load16(ap[v] + k), rb[d][v] = load16(bp[v] + k);
      sa[d][v] = asp[v][e], sb[d][v] = bsp[v][e];
    }
  };
  auto at_a = [&](int s) { return lds + s * (T * PITCH); };
  auto at_b = [&](int s) { return lds + (2 + s) * (T * PITCH); };
  // scale byte of row r, block c: row blocks of a wave tile beside each other
  auto scale_at = [&](int r, int c) { return (((r / W) * 16 + r % 16) * BB + c) * NB + (r % W) / 16; };
  auto put = [&](int s, int v, u32x4 a, u32x4 b, uint8_t ea, uint8_t eb) {
    const int r = row0 + RP * v;
    *reinterpret_cast<u32x4 *>(at_a(s) + r * PITCH + kc) = a;
    *reinterpret_cast<u32x4 *>(at_b(s) + r * PITCH + kc) = b;
    scales[s][0][scale_at(r, chunk)] = ea;
    scales[s][1][scale_at(r, chunk)] = eb;
  };
  auto commit = [&](int d, int s) {
#pragma unroll
    for (int v = 0; v < V; ++v) put(s, v, ra[d][v], rb[d][v], sa[d][v], sb[d][v]);
  };

  f32x4 acc[NB][NB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{};
  auto multiply = [&](int s) {
    u32x4 fa[NB], fb[NB];
    const int blk = team * 4 + (lane >> 4), at = (lane & 15) * PITCH + blk * 16;
    const uint32_t ea = reinterpret_cast<const Scales *>(scales[s][0])[(wm * 16 + (lane & 15)) * BB + blk];
    const uint32_t eb = reinterpret_cast<const Scales *>(scales[s][1])[(wn * 16 + (lane & 15)) * BB + blk];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      fa[i] = *reinterpret_cast<const u32x4 *>(at_a(s) + (wm * W + i * 16) * PITCH + at);
      fb[i] = *reinterpret_cast<const u32x4 *>(at_b(s) + (wn * W + i * 16) * PITCH + at);
    }
    // (B, A): a lane's accumulator holds 4 consecutive columns of one row of C
    unrolled<NB>([&](auto i) {
      unrolled<NB>([&](auto j) { acc[i][j] = mfma_mx4<j.value, i.value>(fb[j], eb, fa[i], ea, acc[i][j]); });
    });
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
      u32x4 a, b;
      if (p.kb >= 16) {
        const int drop = (int)(kt - kl < 16 ? kt - kl : 16);
        a = drop_front(ta[v], drop), b = drop_front(tb[v], drop);
      } else {
        a = load_tail(ap[v], kt, p.kb), b = load_tail(bp[v], kt, p.kb);
      }
      put(0, v, without_odd(a, kt, p.K), b, tsa[v], tsb[v]);
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
        *reinterpret_cast<f32x4 *>(lds + (((wave * H + i % H) * NB + j) * 64 + lane) * 16) = acc[i][j];
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
      const f32x4 other = *reinterpret_cast<const f32x4 *>(lds + ((((wave ^ 4) * H + i % H) * NB + j) * 64 + lane) * 16);
      store_mx4<FMT>(p, ep, row, n, acc[i][j] + other);
    }
  }
}

template <int T, int D>
hipError_t block_t(const Mx4Args &p, hipStream_t stream) {
  return over_tiles(p, T, T, kThreads, [&](const Mx4Args &a, dim3 grid) {
    if (a.fmt == FMT_F32)
      hipLaunchKernelGGL((gemm_mx4_block_kernel<T, FMT_F32, D>), grid, dim3(kThreads), 0, stream, a);
    else if (a.fmt == FMT_F16)
      hipLaunchKernelGGL((gemm_mx4_block_kernel<T, FMT_F16, D>), grid, dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((gemm_mx4_block_kernel<T, FMT_BF16, D>), grid, dim3(kThreads), 0, stream, a);
  });
}

}  // namespace

hipError_t launch_mx4_block(const Mx4Args &p, int tile, hipStream_t stream) {
  return tile == 128 ? block_t<128, 2>(p, stream) : block_t<64, 2>(p, stream);
}

}  // namespace tsm
