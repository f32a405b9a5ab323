// Int8 products of few rows (decoding steps) for gfx950: bound by reading the
// weights once.
//
// A workgroup owns a block of C; its waves share out K in steps of 256 codes,
// and their int32 sums (exact, so the split does not show) meet in LDS and leave
// once, scaled.  Two kernels:
//  * stream: each wave copies its steps into an LDS ring of its own and
//    multiplies from there; for 16-byte aligned operands, K a multiple of 16.
//  * skinny: operands straight into registers, at any alignment.
// i8_skinny_plan has the rule between them and the general kernel.
// Measured on weights that no cache holds, launch included: 16 x 16384 x 8192
// 27.3 us (5.0 TB/s), 1 x 8192 x 8192 15.0 us, 256 experts of 1024 x 2048 86 us
// (6.2 TB/s).
#include "i8_common.hpp"
#include "lds_ring.hpp"

namespace tsm {
namespace {

constexpr int STEP = 256;

// ---- any alignment: operands straight into registers --------------------------
// 16 rows x 16 columns on W waves; wave w takes steps w, w + W, ...  A wave-wide
// load covers 16 rows x 64 bytes, the layout the matrix instruction wants, and a
// step's four loads cover the lines whole.  D steps are in flight per wave.
constexpr int kSkinnyWaves = 4;

template <int FMT>
__global__ __launch_bounds__(kSkinnyWaves * 64) void gemm_i8_skinny_kernel(I8Args p) {
  constexpr int W = kSkinnyWaves, D = 4;
  __shared__ i32x4 part[W][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tm, tn;
  int64_t z;
  if (!i8_tile_of<16>(p, 1, z, tm, tn)) return;  // uniform
  const int64_t M = i8_rows(p, z), m0 = (int64_t)tm * 16, n0 = (int64_t)tn * 16;

  // rows past M or N read the last one: their results are not stored
  const int64_t mr = m0 + (lane & 15), nr = n0 + (lane & 15);
  const int8_t *const ap = p.A + z * p.strideA + (mr < M ? mr : M - 1) * p.lda;
  const int8_t *const bp = p.B + z * p.strideB + (nr < p.N ? nr : p.N - 1) * p.ldb;
  const int kc = (lane >> 4) * 16;

  i32x4 acc{};
  u32x4 a[D][4], b[D][4];
  const int whole = (int)(p.K / STEP);
  auto fetch = [&](int d, int s) {
    const int64_t k = (int64_t)s * STEP + kc;
#pragma unroll
    for (int u = 0; u < 4; ++u) b[d][u] = load16(bp + k + 64 * u), a[d][u] = load16(ap + k + 64 * u);
  };
  auto mma = [&](int d) {
#pragma unroll
    for (int u = 0; u < 4; ++u) acc = mfma_i8(b[d][u], a[d][u], acc);
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (wave + d * W < whole) fetch(d, wave + d * W);
  for (int s = wave; s < whole; s += D * W) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (s + d * W >= whole) break;  // uniform
      mma(d);
      if (s + (d + D) * W < whole) fetch(d, s + (d + D) * W);
    }
  }
  // K's last, partial step
  if ((int64_t)whole * STEP < p.K && wave == whole % W) {
    const int64_t k = (int64_t)whole * STEP + kc;
#pragma unroll
    for (int u = 0; u < 4; ++u) b[0][u] = load_tail(bp, k + 64 * u, p.K), a[0][u] = load_tail(ap, k + 64 * u, p.K);
    mma(0);
  }

  part[wave][lane] = acc;
  __syncthreads();
  const int64_t m = m0 + (lane & 15), n = n0 + kc / 4;
  if (wave != 0 || m >= M || n >= p.N) return;
  i32x4 sum = part[0][lane];
#pragma unroll
  for (int w = 1; w < W; ++w) sum += part[w][lane];
  float cb[4];
  channel_scales(p, z, n, cb);
  store_i8<FMT>(p, Epilogue{p.act, p.slope, false}, (char *)p.C + (z * p.strideC + m * p.ldc) * fmt_bytes(FMT), n,
                p.sa ? p.sa[z * p.stride_sa + m] : 1.f, cb, sum);
}

hipError_t skinny_t(const I8Args &p, hipStream_t stream) {
  constexpr int T = kSkinnyWaves * 64;
  return over_tiles(p, 16, 16, T, [&](const I8Args &a, dim3 grid) {
    if (a.fmt == FMT_F32)
      hipLaunchKernelGGL((gemm_i8_skinny_kernel<FMT_F32>), grid, dim3(T), 0, stream, a);
    else if (a.fmt == FMT_F16)
      hipLaunchKernelGGL((gemm_i8_skinny_kernel<FMT_F16>), grid, dim3(T), 0, stream, a);
    else
      hipLaunchKernelGGL((gemm_i8_skinny_kernel<FMT_BF16>), grid, dim3(T), 0, stream, a);
  });
}

// ---- 16-byte aligned operands, K a multiple of 16 -----------------------------
// Loading the operand layout straight from memory (above) touches 16 rows per
// wave-load: four times the L1 accesses of the copies here (16 x 8192 x 8192: 8.4
// million against 2.1).
// Here each wave copies its own steps into LDS (rows of 256 bytes, whole lines)
// and reads the operands from there; nothing is shared until a tile's end, so
// the loop has no barrier, only the wave's own wait for its oldest copies.  The
// workgroups stay for all of the tiles and the copies run on across tile
// boundaries: a launch in several rounds of workgroups would drain the memory
// pipeline at the end of each.
struct Place {
  int64_t z, m0, n0, M;
};

constexpr int kMaxGroups = 512;  // groups of a launch, whose tiles before each are kept in LDS

// Place of tile t: row tiles fastest, then columns, then problems.  first: of a grouped call, the tiles before each
// group (in LDS, kMaxGroups of them, the ones past the launch's groups holding the total).
template <int AR, int NB>
__device__ __forceinline__ Place stream_tile(const I8Args &p, int t, const int *first, int lane) {
  Place e;
  int tm = p.tiles_m, g = 0;
  if (p.rows) {
    for (int i = 0; i < p.nz; i += 64) g += __popcll(__ballot(first[i + lane] <= t));
    g = min(g, p.nz) - 1;
    const int f = __builtin_amdgcn_readfirstlane(first[g]);
    tm = (int)((i8_rows(p, p.z0 + g) + AR - 1) / AR);
    t -= f;
  } else {
    g = t / (tm * p.tiles_n);
    t -= g * (tm * p.tiles_n);
  }
  e.z = p.z0 + g;
  e.M = i8_rows(p, e.z);
  e.m0 = (int64_t)(t % tm) * AR;
  e.n0 = (int64_t)(t / tm) * (16 * NB);
  return e;
}

template <int AR, int NB, int W, int FMT>
__device__ __forceinline__ void stream(const I8Args &p) {
  constexpr int MB = AR / 16;
  constexpr int LA = AR / 4, LB = 4 * NB, L = LA + LB;  // wave-loads (1 KiB: 4 rows) per step
  constexpr int BYTES = L * 1024;
  __shared__ __attribute__((aligned(1024))) char s0[W * BYTES], s1[W * BYTES];  // the ring's two stages
  __shared__ int first[kMaxGroups];
  static_assert(MB * NB <= L, "a wave's sums fit one stage");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tiles = p.tiles_m * p.tiles_n * p.nz;
  if (p.rows) {
    // every wave computes the sums, the first writes them
    int sum = 0;
    for (int g = 0; g < p.nz; g += 64) {
      const int v = group_tiles<AR>(p, g + lane) * p.tiles_n;
      const int s = wave_scan(v, lane);
      if (wave == 0) first[g + lane] = sum + s - v;
      sum += __builtin_amdgcn_readlane(s, 63);
    }
    tiles = sum;
    __syncthreads();
  }
  int t = blockIdx.x;
  if (t >= tiles) return;  // uniform
  // wave-load g: rows 4 g + lane / 16; LDS position lane % 16 of a row holds chunk (lane % 16) ^ (row % 16)
  auto row_of = [&](int g) { return 4 * (g < LA ? g : g - LA) + (lane >> 4); };
  auto chunk_of = [&](int g) { return ((lane & 15) ^ (row_of(g) & 15)) * 16; };  // its first code within the step
  uint32_t off[L];
#pragma unroll
  for (int g = 0; g < L; ++g) off[g] = (uint32_t)(row_of(g) * (g < LA ? p.lda : p.ldb) + chunk_of(g));
  const int steps = (int)((p.K + STEP - 1) / STEP);
  const int turns = (steps + 2 * W - 1) / (2 * W);  // of the ring, per tile
  // (kept out of the compiler's sight: every copy's LDS address held in a scalar register of its own would spill them)
  int mine = wave * BYTES;
  auto stage = [&](int d) -> char * {
    asm volatile("" : "+s"(mine));
    return (d == 0 ? s0 : s1) + mine;
  };
  // The copies run one step ahead of the products: step fq of tile ft, through resources over its valid rows
  // (others lie past them, since leading dimensions are at least K, and load as zeros).
  __amdgpu_buffer_rsrc_t ra, rb;
  int ft = blockIdx.x, fq = 0;
  auto open = [&](int t) {
    const Place e = stream_tile<AR, NB>(p, t, first, lane);
    const int64_t vm = e.M - e.m0 < AR ? e.M - e.m0 : AR, vn = p.N - e.n0 < 16 * NB ? p.N - e.n0 : 16 * NB;
    ra = make_rsrc(p.A + e.z * p.strideA + e.m0 * p.lda, (uint32_t)((vm - 1) * p.lda + p.K));
    rb = make_rsrc(p.B + e.z * p.strideB + e.n0 * p.ldb, (uint32_t)((vn - 1) * p.ldb + p.K));
  };
  // The next step's copies into stage d.  Chunks past K, and steps past the end, copy zeros without touching memory:
  // the count of copies in flight stays the same.
  auto fetch = [&](int d) {
    const int s = fq * W + wave;
    const int left = ft < tiles && s < steps ? (int)(p.K - (int64_t)s * STEP) : 0;
    char *const to = stage(d);
#pragma unroll
    for (int g = 0; g < L; ++g)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(g < LA ? ra : rb, (lds_void *)(to + g * 1024), 16,
                                               chunk_of(g) < left ? off[g] : kOutside, left ? s * STEP : 0, 0, 0);
    if (++fq == turns * 2) {
      fq = 0;
      ft += gridDim.x;
      if (ft < tiles) open(ft);
    }
  };
  open(t);
  fetch(0);
  for (; t < tiles; t += gridDim.x) {
    i32x4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = i32x4{};
    for (int q = 0; q < turns; ++q) {
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        // the stage read in the last turn is free (its reads are done): refill it
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        fetch(1 - d);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L) : "memory");
        const char *a = stage(d), *b = a + LA * 1024;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = lane & 15;
          // offset of this lane's chunk; opaque, because a read that the compiler can tell apart from a stage's first
          // copy makes it wait for every copy in flight
          int at = r * STEP + ((4 * u + (lane >> 4)) ^ r) * 16;
          asm("" : "+v"(at));
          u32x4 fa[MB], fb[NB];
#pragma unroll
          for (int i = 0; i < MB; ++i) fa[i] = *reinterpret_cast<const u32x4 *>(a + at + 16 * i * STEP);
#pragma unroll
          for (int j = 0; j < NB; ++j) fb[j] = *reinterpret_cast<const u32x4 *>(b + at + 16 * j * STEP);
#pragma unroll
          for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[i][j] = mfma_i8(fb[j], fa[i], acc[i][j]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      // (the stage just read is refilled only in the next tile)
      for (int j = 0; j < NB; ++j) *reinterpret_cast<i32x4 *>(stage(1) + ((i * NB + j) * 64 + lane) * 16) = acc[i][j];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    // the epilogue's arguments are read again for each tile: held through the loop they would spill
    const __attribute__((address_space(4))) I8Args *ka =
        (const __attribute__((address_space(4))) I8Args *)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(ka));
    const I8Args e = *(const I8Args *)ka;
    const Place o = stream_tile<AR, NB>(e, t, first, lane);
    const Epilogue ep{e.act, e.slope, false};
    const float *sa = e.sa ? e.sa + o.z * e.stride_sa : nullptr;
    for (int k = threadIdx.x; k < MB * NB * 64; k += W * 64) {
      const int blk = k >> 6, l = k & 63;
      const int64_t m = o.m0 + 16 * (blk / NB) + (l & 15), n = o.n0 + 16 * (blk % NB) + 4 * (l >> 4);
      if (m >= o.M || m >= o.m0 + AR || n >= e.N) continue;
      i32x4 sum{};
#pragma unroll
      for (int w = 0; w < W; ++w) sum += *reinterpret_cast<const i32x4 *>(s1 + w * BYTES + k * 16);
      float cb[4];
      channel_scales(e, o.z, n, cb);
      store_i8<FMT>(e, ep, (char *)e.C + (o.z * e.strideC + m * e.ldc) * fmt_bytes(FMT), n, sa ? sa[m] : 1.f, cb, sum);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();  // the sums are read: the next tile's may be written
    asm volatile("" ::: "memory");
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the copies of zeros past the end
}

template <int AR, int NB, int W, int FMT>
__global__ __launch_bounds__(W * 64) void gemm_i8_stream_kernel(I8Args p) {
  stream<AR, NB, W, FMT>(p);
}

template <int AR, int NB, int W>
hipError_t stream_t(I8Args a, hipStream_t st) {
  constexpr int LDS = 2 * W * (AR / 4 + 4 * NB) * 1024 + 4 * kMaxGroups + 64;
  a.tiles_m = (int32_t)((a.M + AR - 1) / AR);
  a.tiles_n = (int32_t)((a.N + 16 * NB - 1) / (16 * NB));
  const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
  // what 256 CUs of 160 KiB hold at once; the rest of the tiles follow in the same workgroups
  const int64_t resident = 256 * (163840 / LDS);
  int64_t most = 0x3fffffff / tiles;  // problems per launch: tile numbers stay far below 2^31
  if (a.rows && most > kMaxGroups) most = kMaxGroups;
  for (int64_t z0 = 0; z0 < a.batch; z0 += most) {
    a.z0 = z0;
    a.nz = (int32_t)(a.batch - z0 < most ? a.batch - z0 : most);
    const dim3 grid((unsigned)(tiles * a.nz < resident ? tiles * a.nz : resident));
    if (a.fmt == FMT_F32)
      hipLaunchKernelGGL((gemm_i8_stream_kernel<AR, NB, W, FMT_F32>), grid, dim3(W * 64), 0, st, a);
    else if (a.fmt == FMT_F16)
      hipLaunchKernelGGL((gemm_i8_stream_kernel<AR, NB, W, FMT_F16>), grid, dim3(W * 64), 0, st, a);
    else
      hipLaunchKernelGGL((gemm_i8_stream_kernel<AR, NB, W, FMT_BF16>), grid, dim3(W * 64), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

// Which kernel, and the streaming one's rows per workgroup (16 or 32), blocks of
// 16 columns and waves.  kernel None: the general one (64 x 64 tiles).  Timed on
// weights past the caches; "tiles" are blocks of 16 columns over all problems.
//  * Operands that the ring's copies cannot take, up to 16 rows: registers while
//    a CU has one tile (16 x 4096 x 4095 18.0 us against 23.0 in the general
//    kernel, 16 x 4096 x 8191 31.9 against 40.6); past that the L1
//    accesses of 16 rows at odd addresses, four times those of aligned ones, cost
//    more (16 x 8192 x 8191 59.5 against 43.6), and those of more rows always
//    (32 x 4096 x 4095 32.6 against 22.9).
//  * Others, up to 4 rows of K <= 4096: registers too, since a wave has few steps
//    and a ring to fill first (4 x 28672 x 4096 24.4 us against 26.7 streamed,
//    1 x 128256 x 4096 88 against 102; 1 x 65536 x 2048 28.2 against 25.0; at
//    K = 8192 1 x 16384: 33.6 against 25.2).
//  * One wave per workgroup (no barrier, no split of K) once the tiles keep
//    every CU's memory queue full, four while they do not: 16 rows, 16384 x 8192
//    (1024 tiles) 28.4 us on four waves against 30.7 on one, 28672 x 4096 30.5
//    against 27.8, 64 groups of 1024 x 2048 36.5 against 26.0, 1024 x 8192 7.0
//    against 12.6.
//  * 17-32 rows: 28672 x 4096 30.7 us on two column blocks and one wave, 32.3 on
//    one and two; 8192 x 8192 23.9 against 19.6.
//  * 33-64 rows read the weights twice in 32-row blocks (past L2 both times, by
//    the counters: neighbours run on different XCDs): 8192 x 8192 26 us against
//    34 in the general kernel, whose 64 x 64 tiles win once most CUs have one:
//    12288 x 4096 23.5 against 21.2, 16384 x 8192 42 against 39, 64 batches of
//    1024 x 2048 40 against 34, 256 of them 165 against 137.  Grouped calls, whose
//    counts mostly lie far below the capacity, keep 32 (256 groups of 1024 x
//    2048, 16 rows each of 64: 112 us against 137 in 64-row blocks).
I8Skinny i8_skinny_plan(const I8Args &p) {
  I8Skinny s;
  // (more columns than workgroups of 256 fit a launch go to the general kernel)
  if (p.M > 64 || p.K == 0 || p.N > 0xffffffffLL / 256 * 16) return s;
  const bool aligned = (((uintptr_t)p.A | (uintptr_t)p.B) & 15) == 0 && p.K % 16 == 0 && p.lda % 16 == 0 &&
                       p.ldb % 16 == 0 && p.strideA % 16 == 0 && p.strideB % 16 == 0;
  // 32-bit offsets over a block's rows
  const bool fits = 32 * p.lda + p.K < (int64_t)1 << 30 && 32 * p.ldb + p.K < (int64_t)1 << 30;
  s.can_stream = aligned && fits;
  const int64_t per = (p.N + 15) / 16;
  s.can_skinny = (p.M + 15) / 16 * per <= 0xffffffffLL / 256;
  const int64_t tiles = per > ((int64_t)1 << 40) / p.batch ? (int64_t)1 << 40 : per * p.batch;
  if (p.M <= 16) {
    s.rows = 16;
    s.nb = 1;
    s.waves = tiles >= 1024 && tiles >= p.K / 4 ? 1 : 4;
  } else {
    s.rows = 32;
    s.nb = tiles >= (p.M > 32 ? 512 : 1536) ? 2 : 1;
    s.waves = s.nb == 2 ? 1 : 2;
  }
  if (!s.can_stream)
    s.kernel = p.M <= 16 && tiles <= 256 ? I8Kernel::Skinny : I8Kernel::None;
  else if (p.M <= 4 && p.K <= 4096 && !p.rows)
    s.kernel = I8Kernel::Skinny;
  else
    s.kernel = p.M > 32 && tiles >= 768 && !p.rows ? I8Kernel::None : I8Kernel::Stream;
  return s;
}

hipError_t launch_i8_stream(const I8Args &p, hipStream_t st) {
  const I8Skinny s = i8_skinny_plan(p);
  if (s.rows == 16) return s.waves == 1 ? stream_t<16, 1, 1>(p, st) : stream_t<16, 1, 4>(p, st);
  return s.nb == 1 ? stream_t<32, 1, 2>(p, st) : stream_t<32, 2, 1>(p, st);
}

hipError_t launch_i8_skinny(const I8Args &p, hipStream_t st) { return skinny_t(p, st); }

}  // namespace tsm
