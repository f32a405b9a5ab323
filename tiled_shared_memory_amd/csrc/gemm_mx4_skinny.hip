// Products of microscaled 4-bit codes of few rows (decoding steps) for gfx950: bound
// by reading the weights once.
//
//  * stream: up to 64 rows.  Persistent workgroups of one or two waves, each tile all
//    rows by 32 or 64 columns of a problem.  The waves of a workgroup share out K in
//    steps of 512 elements (256 bytes of a row); each copies its steps' codes and
//    scales of both operands into an LDS ring of its own with direct loads, without a
//    barrier, and multiplies from there; their float32 sums meet in LDS and are added
//    in the order of the waves.  The copies run on across tile boundaries.  The
//    weights, which no other tile reads, are loaded non-temporally.
//  * rows: activations of one or two rows, quantised within the launch.  Every workgroup
//    keeps all of A in LDS, after quantising it by itself while its first copies of
//    the weights are on their way; only the weights pass through the waves' rings.
//
// A lane takes blocks 4g .. 4g + 3 of a step's sixteen (g = lane / 16) in its four
// matrix instructions, so that its scales of a step are one word per 16 rows.  What
// decides is that the copies never stop, and the compiler's waits stand in the way of
// that: an array of LDS for each stage, scales that come through LDS too, counts by
// scalar loads and writes that it does not see keep the loop free of waits for
// everything in flight.
//
// Measured, bf16 out, weights from memory (a copy reaches 5.1 TB/s on the same card):
//   16 x 16384 x 8192   16.0 us a call, 4.5 TB/s  (scales in registers, whose copies at
//                       the loop's end waited: 21.5; then weights through all caches: 18.3)
//   8 x 28672 x 8192    26.5 us, 4.7 TB/s     8 x 8192 x 28672   23.0 us, 5.4 TB/s
//   64 groups of 4 x 2048 x 4096   48.5 us, 5.9 TB/s (part of it from the cache)
//   1 x 8192 x 8192 from bf16   9.5 us, in two launches 15 (rings of 2 stages: 13.5)
#include "lds_ring.hpp"
#include "mx4_codes.hpp"
#include "mx4_common.hpp"

namespace tsm {
namespace {

constexpr int STEP = 256;  // bytes of codes per step and row
constexpr int BLOCKS = STEP / 16;

constexpr int kOnce = 2;  // (cache policy: non-temporal) of the weights, which are read once

struct Place {
  int64_t z, n0, M;
};

// Valid rows of problem z, by a scalar load: the vector load that the compiler would choose waits, in its turn, for the
// copies in flight.
__device__ __forceinline__ int64_t rows_of(const Mx4Args &p, int64_t z) {
  if (!p.rows) return p.M;
  const int64_t r = ((const __attribute__((address_space(4))) int32_t *)p.rows)[z];
  return r < 0 ? 0 : (r > p.M ? p.M : r);
}

constexpr int kMaxGroups = 512;  // groups of a launch, whose tiles before each are kept in LDS

// Place of tile t: columns, then problems.  first: of a grouped call, the tiles before each group, those of empty groups
// left out (in LDS, kMaxGroups of them, the ones past the launch's groups holding the total).
template <int NB>
__device__ __forceinline__ Place stream_tile(const Mx4Args &p, int t, const int *first, int lane) {
  Place e;
  int g = 0;
  if (p.rows) {
    for (int i = 0; i < p.nz; i += 64) g += __popcll(__ballot(first[i + lane] <= t));
    g = min(g, p.nz) - 1;
    t -= __builtin_amdgcn_readfirstlane(first[g]);
  } else {
    g = t / p.tiles_n;
    t -= g * p.tiles_n;
  }
  e.z = p.z0 + g;
  e.M = rows_of(p, e.z);
  e.n0 = (int64_t)t * (16 * NB);
  return e;
}

__device__ __forceinline__ uint32_t lds_at(const char *at) { return (uint32_t)(uintptr_t)(lds_void *)at; }

// Writes to LDS that the compiler does not see: it would wait for every copy in flight before them.
__device__ __forceinline__ void lds_write4(uint32_t at, uint32_t v) {
  asm volatile("ds_write_b32 %0, %1" ::"v"(at), "v"(v) : "memory");
}
__device__ __forceinline__ void lds_write1(uint32_t at, uint32_t v) {
  asm volatile("ds_write_b8 %0, %1" ::"v"(at), "v"(v) : "memory");
}
// (with the wait that a matrix instruction's result needs)
__device__ __forceinline__ void lds_write_sums(uint32_t at, f32x4 v) {
  asm volatile("s_nop 15\n\ts_nop 15\n\tds_write_b128 %0, %1" ::"v"(at), "v"(v) : "memory");
}

template <int AR, int NB, int W, int FMT>
__device__ __forceinline__ void stream(const Mx4Args &p) {
  constexpr int MB = AR / 16;
  constexpr int LA = AR / 4, LB = 4 * NB, L = LA + LB;  // wave-loads (1 KiB: 4 rows) per step
  constexpr int N = L + MB + NB;                  // with those of the scales, 256 bytes each
  constexpr int BYTES = L * 1024 + (MB + NB) * 256;
  // the ring's two stages (deeper ones were no faster), an array each: a read waits for the copies into its array, as
  // the compiler sees to it
  __shared__ __attribute__((aligned(1024))) char s0[W * BYTES], s1[W * BYTES];
  __shared__ int first[kMaxGroups];
  static_assert(MB * NB <= L, "a wave's sums fit one stage");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tiles = p.tiles_n * p.nz;
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
  auto chunk_of = [&](int g) { return ((lane & 15) ^ (row_of(g) & 15)) * 16; };  // its first byte within the step
  uint32_t off[L];
#pragma unroll
  for (int g = 0; g < L; ++g) off[g] = (uint32_t)(row_of(g) * (g < LA ? p.lda : p.ldb) + chunk_of(g));
  // the scales' words: row lane % 16, word lane / 16 of a step's four
  const uint32_t offa = (uint32_t)((lane & 15) * p.ldsa + (lane >> 4) * 4);
  const uint32_t offb = (uint32_t)((lane & 15) * p.ldsb + (lane >> 4) * 4);
  const int steps = (int)((p.kb + STEP - 1) / STEP);
  const int turns = (steps + 2 * W - 1) / (2 * W);  // of the ring, per tile
  // (kept out of the compiler's sight: every copy's LDS address held in a scalar register of its own would spill them)
  int mine = wave * BYTES;
  auto stage = [&](int d) -> char * {
    asm volatile("" : "+s"(mine));
    return (d == 0 ? s0 : s1) + mine;
  };
  // The copies run one step ahead of the products: step fq of tile ft, through resources over its valid rows
  // (others lie past them, since leading dimensions are at least a row's bytes, and load as zeros).
  __amdgpu_buffer_rsrc_t ra, rb, rsa, rsb;
  int ft = blockIdx.x, fq = 0;
  auto open = [&](int t) {
    const Mx4Args q = args_again();
    const Place e = stream_tile<NB>(q, t, first, lane);
    const int64_t vn = q.N - e.n0 < 16 * NB ? q.N - e.n0 : 16 * NB;
    ra = make_rsrc(q.A + e.z * q.strideA, (uint32_t)((e.M - 1) * q.lda + q.kb));
    rb = make_rsrc(q.B + e.z * q.strideB + e.n0 * q.ldb, (uint32_t)((vn - 1) * q.ldb + q.kb));
    rsa = make_rsrc(q.SA + e.z * q.strideSA, (uint32_t)((e.M - 1) * q.ldsa + q.nb));
    rsb = make_rsrc(q.SB + e.z * q.strideSB + e.n0 * q.ldsb, (uint32_t)((vn - 1) * q.ldsb + q.nb));
  };
  // The next step's copies into stage d.  Chunks past K, and steps past the end, copy zeros without touching memory
  // (their scales too: what lies behind a row may be a scale of NaN): the count of copies in flight stays the same.
  auto fetch = [&](int d) {
    const int s = fq * W + wave;
    const int left = ft < tiles && s < steps ? (int)(p.kb - (int64_t)s * STEP) : 0;
    char *const to = stage(d);
    unrolled<L>([&](auto g) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(g.value < LA ? ra : rb, (lds_void *)(to + g.value * 1024), 16,
                                               chunk_of(g.value) < left ? off[g.value] : kOutside, left ? s * STEP : 0, 0,
                                               g.value < LA ? 0 : kOnce);
    });
    const bool in = (lane >> 4) * 64 < left;
#pragma unroll
    for (int i = 0; i < MB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsa, (lds_void *)(to + L * 1024 + i * 256), 4,
                                               in ? offa + (uint32_t)(16 * i * p.ldsa) : kOutside, left ? s * BLOCKS : 0, 0, 0);
#pragma unroll
    for (int j = 0; j < NB; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsb, (lds_void *)(to + L * 1024 + (MB + j) * 256), 4,
                                               in ? offb + (uint32_t)(16 * j * p.ldsb) : kOutside, left ? s * BLOCKS : 0, 0, 0);
    if (++fq == turns * 2) {
      fq = 0;
      ft += gridDim.x;
      if (ft < tiles) open(ft);
    }
  };
  open(t);
  fetch(0);
  for (; t < tiles; t += gridDim.x) {
    f32x4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{};
    for (int q = 0; q < turns; ++q) {
      unrolled<2>([&](auto d) {
        // the stage read in the last step is free (its reads are done): refill it
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        fetch(1 - d.value);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
        const char *a = stage(d.value), *b = a + LA * 1024;
        int at_s = L * 1024 + lane * 4;
        asm("" : "+v"(at_s));
        uint32_t wa[MB], wb[NB];
#pragma unroll
        for (int i = 0; i < MB; ++i) wa[i] = *reinterpret_cast<const uint32_t *>(a + at_s + i * 256);
#pragma unroll
        for (int j = 0; j < NB; ++j) wb[j] = *reinterpret_cast<const uint32_t *>(a + at_s + (MB + j) * 256);
        unrolled<4>([&](auto u) {
          const int r = lane & 15;
          // offset of this lane's chunk; opaque, because a read that the compiler can tell apart from a stage's first
          // copy makes it wait for every copy in flight
          int at = r * STEP + ((4 * (lane >> 4) + u.value) ^ r) * 16;
          asm("" : "+v"(at));
          u32x4 fa[MB], fb[NB];
#pragma unroll
          for (int i = 0; i < MB; ++i) fa[i] = *reinterpret_cast<const u32x4 *>(a + at + 16 * i * STEP);
#pragma unroll
          for (int j = 0; j < NB; ++j) fb[j] = *reinterpret_cast<const u32x4 *>(b + at + 16 * j * STEP);
#pragma unroll
          for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
              acc[i][j] = mfma_mx4<u.value, u.value>(fb[j], wb[j], fa[i], wa[i], acc[i][j]);
        });
      });
    }
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      // (the stage just read is refilled only in the next tile)
      for (int j = 0; j < NB; ++j) lds_write_sums(lds_at(stage(1)) + ((i * NB + j) * 64 + lane) * 16, acc[i][j]);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const Mx4Args e = args_again();
    const Place o = stream_tile<NB>(e, t, first, lane);
    const Epilogue ep{e.act, e.slope, false};
    for (int k = threadIdx.x; k < MB * NB * 64; k += W * 64) {
      const int blk = k >> 6, l = k & 63;
      const int64_t m = 16 * (blk / NB) + (l & 15), n = o.n0 + 16 * (blk % NB) + 4 * (l >> 4);
      if (m >= o.M || n >= e.N) continue;
      f32x4 sum{};
#pragma unroll
      for (int w = 0; w < W; ++w) sum += *reinterpret_cast<const f32x4 *>(s1 + w * BYTES + k * 16);
      store_mx4<FMT>(e, ep, (char *)e.C + (o.z * e.strideC + m * e.ldc) * fmt_bytes(FMT), n, sum);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();  // the sums are read: the next tile's may be written
    asm volatile("" ::: "memory");
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the copies of zeros past the end
}

template <int AR, int NB, int W, int FMT>
__global__ __launch_bounds__(W * 64) void gemm_mx4_stream_kernel(Mx4Args p) {
  stream<AR, NB, W, FMT>(p);
}

template <int AR, int NB, int W>
hipError_t stream_t(Mx4Args a, hipStream_t st) {
  constexpr int LDS = 2 * W * ((AR / 4 + 4 * NB) * 1024 + (AR / 16 + NB) * 256) + 4 * kMaxGroups;
  a.tiles_m = 1;
  a.tiles_n = (int32_t)((a.N + 16 * NB - 1) / (16 * NB));
  const int64_t tiles = a.tiles_n;
  // what 256 CUs of 160 KiB hold at once; the rest of the tiles follow in the same workgroups
  const int64_t resident = 256 * (163840 / LDS);
  int64_t most = 0x3fffffff / tiles;  // problems per launch: tile numbers stay far below 2^31
  if (a.rows && most > kMaxGroups) most = kMaxGroups;
  for (int64_t z0 = 0; z0 < a.batch; z0 += most) {
    a.z0 = z0;
    a.nz = (int32_t)(a.batch - z0 < most ? a.batch - z0 : most);
    const dim3 grid((unsigned)(tiles * a.nz < resident ? tiles * a.nz : resident));
    if (a.fmt == FMT_F32)
      hipLaunchKernelGGL((gemm_mx4_stream_kernel<AR, NB, W, FMT_F32>), grid, dim3(W * 64), 0, st, a);
    else if (a.fmt == FMT_F16)
      hipLaunchKernelGGL((gemm_mx4_stream_kernel<AR, NB, W, FMT_F16>), grid, dim3(W * 64), 0, st, a);
    else
      hipLaunchKernelGGL((gemm_mx4_stream_kernel<AR, NB, W, FMT_BF16>), grid, dim3(W * 64), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// ---- activations of one or two rows, kept in LDS ---------------------------------
constexpr int kRowWaves = 4, kRowThreads = kRowWaves * 64, kRing = 4;
constexpr int kRowWave = 4096 + 256;             // a wave's ring stage: 16 columns x 256 bytes, and their scales
constexpr int kRowStage = kRowWaves * kRowWave;
constexpr int kStepRow = STEP + BLOCKS;          // a row of a step of A: codes and scale bytes
constexpr int kRowSteps = 2 * kRowWaves;         // rows times steps of A in each array
// A wave's step q takes ring stage q % 4, and its part of A lies in the same array as that stage: a read of an array
// waits for the copies into it (the compiler sees to it), and those into the other three stay in flight.
constexpr int kRowArray = kRowStage + kRowSteps * kStepRow;

// Byte offset in its array of step s of A (M rows); the arrays take wave after wave of a turn's steps.
__device__ __forceinline__ int step_at(int s, int M) {
  return kRowStage + (s / (kRing * kRowWaves) * kRowWaves + s % kRowWaves) * M * kStepRow;
}

// All of X in registers, a thread's chunks of 8 elements of each row kRowThreads apart (rows past the last one and chunks
// past K load the first in their place).
constexpr int kRowChunks = kRowSteps * kRing * (2 * STEP / 8) / kRowThreads;
template <int XF>
__device__ __forceinline__ void load_rows(const Mx4Args &p, int rows, int per, Chunk<XF> (&ch)[kRowChunks]) {
#pragma unroll
  for (int i = 0; i < kRowChunks; ++i) {
    const int r = i / 4 * 4 / per, c = (i - r * per) * kRowThreads + threadIdx.x;  // a turn's 16 steps are 4 chunks a thread
    ch[i].load((const char *)p.X + (r < rows ? r : 0) * p.ldx * fmt_bytes(XF), c * 8 < p.K ? c : 0);
  }
}

// Their codes and scales to LDS, zeros past K: four lanes hold a block of 32.  Chunk c of a row of a step lies at c ^ row.
template <int XF>
__device__ __forceinline__ void keep_rows(const Mx4Args &p, const Chunk<XF> (&ch)[kRowChunks], int rows, int per,
                                          const uint32_t (&array)[kRing]) {
#pragma unroll
  for (int i = 0; i < kRowChunks; ++i) {
    const int r = i / 4 * 4 / per, c = (i - r * per) * kRowThreads + threadIdx.x;
    if (r >= rows) break;  // uniform
    const uint32_t e = c * 8 < p.K ? scale_byte(quad_max(ch[i].top())) : 0u;
    const uint32_t codes = e == 255u || c * 8 >= p.K ? 0u : codes_of<XF>(ch[i], scale_of(e));
    const int s = c / (2 * STEP / 8), in = c % (2 * STEP / 8);
    // a thread's chunk i is of step 4 i + threadIdx.x / 64 of its row, and so of array i % 4
    static_assert(kRowThreads == kRowWaves * (2 * STEP / 8) && kRing == 4);
    const uint32_t to = array[i % 4] + step_at(s, (int)p.M) + r * kStepRow;
    lds_write4(to + (((in >> 2) ^ r) * 16) + (in & 3) * 4, codes);
    if ((in & 3) == 0) lds_write1(to + STEP + (in >> 2), e);
  }
}

template <int XF>
__device__ __forceinline__ void rows_product(const Mx4Args &p) {
  __shared__ __attribute__((aligned(1024))) char s0[kRowArray], s1[kRowArray], s2[kRowArray], s3[kRowArray];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles = p.tiles_n;
  const int steps = (int)((p.kb + STEP - 1) / STEP);
  const int turns = (steps + kRing * kRowWaves - 1) / (kRing * kRowWaves);
  const int M = (int)p.M;
  const int rows = (int)rows_of(p, 0);
  if (rows == 0) return;
  // wave-load g: rows 4 g + lane / 16 of the weights; position lane % 16 of a row holds chunk (lane % 16) ^ (row % 16)
  auto row_of = [&](int g) { return 4 * g + (lane >> 4); };
  auto chunk_of = [&](int g) { return ((lane & 15) ^ (row_of(g) & 15)) * 16; };
  uint32_t off[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) off[g] = (uint32_t)(row_of(g) * p.ldb + chunk_of(g));
  const uint32_t offb = (uint32_t)((lane & 15) * p.ldsb + (lane >> 4) * 4);
  int mine = wave * kRowWave;
  auto array = [&](int d) -> char * { return d == 0 ? s0 : d == 1 ? s1 : d == 2 ? s2 : s3; };
  auto stage = [&](int d) -> char * {
    asm volatile("" : "+s"(mine));  // (as in the streaming kernel)
    return array(d) + mine;
  };
  __amdgpu_buffer_rsrc_t rb, rsb;
  int ft = blockIdx.x, fq = 0;
  auto open = [&](int t) {
    const Mx4Args q = args_again();
    const int64_t n0 = (int64_t)t * 16, vn = q.N - n0 < 16 ? q.N - n0 : 16;
    rb = make_rsrc(q.B + n0 * q.ldb, (uint32_t)((vn - 1) * q.ldb + q.kb));
    rsb = make_rsrc(q.SB + n0 * q.ldsb, (uint32_t)((vn - 1) * q.ldsb + q.nb));
  };
  // The next step's copies into stage d; chunks past K and steps past the end copy zeros without touching memory, their
  // scales too.
  auto fetch = [&](int d) {
    const int s = fq * kRowWaves + wave;
    const int left = ft < tiles && s < steps ? (int)(p.kb - (int64_t)s * STEP) : 0;
    char *const to = stage(d);
#pragma unroll
    for (int g = 0; g < 4; ++g)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void *)(to + g * 1024), 16, chunk_of(g) < left ? off[g] : kOutside,
                                               left ? s * STEP : 0, 0, kOnce);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsb, (lds_void *)(to + 4096), 4, (lane >> 4) * 64 < left ? offb : kOutside,
                                             left ? s * BLOCKS : 0, 0, 0);
    if (++fq == turns * kRing) {
      fq = 0;
      ft += gridDim.x;
      if (ft < tiles) open(ft);
    }
  };
  {
    // the activations first: what is loaded after the copies would arrive after them
    Chunk<XF> ch[kRowChunks];
    load_rows<XF>(p, rows, 4 * turns, ch);
    open(ft);
    unrolled<kRing - 1>([&](auto d) { fetch(d.value); });
    const uint32_t at[kRing] = {lds_at(s0), lds_at(s1), lds_at(s2), lds_at(s3)};
    keep_rows<XF>(p, ch, rows, 4 * turns, at);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
  // rows past the last one multiply row 0: their results are not stored
  const int r = lane & 15, ra = r < rows ? r : 0;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    f32x4 acc{};
    for (int q = 0; q < turns; ++q) {
      unrolled<kRing>([&](auto d) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        fetch((d.value + kRing - 1) % kRing);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(5 * (kRing - 1)) : "memory");
        const char *const b = stage(d.value), *const base = array(d.value);
        int at_a = step_at((kRing * q + d.value) * kRowWaves + wave, M) + ra * kStepRow;
        asm("" : "+v"(at_a));
        const uint32_t wa = *reinterpret_cast<const uint32_t *>(base + at_a + STEP + (lane >> 4) * 4);
        int at_s = 4096 + lane * 4;
        asm("" : "+v"(at_s));
        const uint32_t wb = *reinterpret_cast<const uint32_t *>(b + at_s);
        unrolled<4>([&](auto u) {
          int at = r * STEP + ((4 * (lane >> 4) + u.value) ^ r) * 16;
          asm("" : "+v"(at));
          const u32x4 fa = *reinterpret_cast<const u32x4 *>(base + at_a + ((4 * (lane >> 4) + u.value) ^ ra) * 16);
          const u32x4 fb = *reinterpret_cast<const u32x4 *>(b + at);
          acc = mfma_mx4<u.value, u.value>(fb, wb, fa, wa, acc);
        });
      });
    }
    // the waves' sums meet in the stage just read, which the next tile's first step refills
    lds_write_sums(lds_at(stage(kRing - 1)) + lane * 16, acc);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (wave == 0) {
      const Mx4Args e = args_again();
      const int64_t n = (int64_t)t * 16 + 4 * (lane >> 4);
      if (r < rows && n < e.N) {
        f32x4 sum{};
#pragma unroll
        for (int w = 0; w < kRowWaves; ++w)
          sum += *reinterpret_cast<const f32x4 *>(array(kRing - 1) + w * kRowWave + lane * 16);
        const Epilogue ep{e.act, e.slope, false};
        char *const row = (char *)e.C + r * e.ldc * (e.fmt == FMT_F32 ? 4 : 2);
        if (e.fmt == FMT_F32) store_mx4<FMT_F32>(e, ep, row, n, sum);
        else if (e.fmt == FMT_F16) store_mx4<FMT_F16>(e, ep, row, n, sum);
        else store_mx4<FMT_BF16>(e, ep, row, n, sum);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();  // the sums are read
    asm volatile("" ::: "memory");
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the copies of zeros past the end
}

template <int XF>
__global__ __launch_bounds__(kRowThreads, 2) void gemm_mx4_rows_kernel(Mx4Args p) {
  rows_product<XF>(p);
}

}  // namespace

Mx4Few mx4_few_plan(const Mx4Args &p) {
  Mx4Few s;
  // (more columns than tile numbers hold go to the general kernel)
  if (p.M > 64 || p.K == 0 || p.N > 0xffffffffLL / 256 * 16) return s;
  const bool aligned = (((uintptr_t)p.A | (uintptr_t)p.B) & 15) == 0 && (((uintptr_t)p.SA | (uintptr_t)p.SB) & 3) == 0 &&
                       p.K % 128 == 0 && ((p.lda | p.ldb | p.strideA | p.strideB) & 15) == 0 &&
                       ((p.ldsa | p.ldsb | p.strideSA | p.strideSB) & 3) == 0;
  // 32-bit offsets over a block's rows
  const int64_t limit = (int64_t)1 << 30;
  s.can_stream = aligned && 64 * p.lda + p.kb < limit && 64 * p.ldb + p.kb < limit && 64 * p.ldsa + p.nb < limit &&
                 64 * p.ldsb + p.nb < limit;
  const int64_t per = (p.N + 63) / 64;
  const int64_t tiles = per > ((int64_t)1 << 40) / p.batch ? (int64_t)1 << 40 : per * p.batch;  // of 64 columns
  // Two waves share K, one where it has no two full turns of the ring for them (us, one | two waves):
  //   256 groups of 16 x 512 x 512   14.3 | 25.6     16 x 8192 x 8192   13.3 | 11.2     16 x 8192 x 28672   34 | 23
  // 64 columns (up to 16 rows) halve the reads of A where they still give every CU a tile (32 | 64 columns):
  //   16 x 16384 x 8192   17.4 | 17.0     8 x 28672 x 8192   27.7 | 26.5     16 x 128000 x 4096   60 | 52
  //   16 x 8192 x 8192    11.2 | 12.7
  // Rows past 32 stream while one round of workgroups holds all tiles (streaming | the general kernel's 64 x 64 tiles):
  //   64 x 8192 x 8192    16.3 | 23.1     64 x 8192 x 28672   40.7 | 68.6     64 x 10240 x 8192   25.6 | 23.7
  // and up to 32 rows always:
  //   16 x 16384 x 8192   17.0 | 22.8     32 x 16384 x 8192   20.2 | 23.3     32 x 128000 x 4096   63.8 | 74.2
  //   256 groups of 32 x 512 x 512   18.4 | 19.3     32 x 32000 x 1024   9.2 | 8.7
  s.rows = p.M <= 16 ? 16 : p.M <= 32 ? 32 : 64;
  s.waves = p.K <= 1024 && p.M <= 32 ? 1 : 2;
  s.nb = p.M <= 16 && s.waves == 2 && tiles >= 256 ? 4 : 2;
  s.use_stream = s.can_stream && (p.M <= 32 || tiles <= 128);
  return s;
}

hipError_t launch_mx4_stream(const Mx4Args &p, hipStream_t st) {
  const Mx4Few s = mx4_few_plan(p);
  if (s.rows == 16) {
    if (s.waves == 1) return stream_t<16, 2, 1>(p, st);
    return s.nb == 2 ? stream_t<16, 2, 2>(p, st) : stream_t<16, 4, 2>(p, st);
  }
  if (s.rows == 32) return s.waves == 1 ? stream_t<32, 2, 1>(p, st) : stream_t<32, 2, 2>(p, st);
  return stream_t<64, 2, 2>(p, st);
}

bool mx4_rows_supports(const Mx4Args &p) {
  const int64_t turns = (p.kb + kRing * kRowWaves * STEP - 1) / (kRing * kRowWaves * STEP);
  return p.batch == 1 && p.K > 0 && turns * kRowWaves * p.M <= kRowSteps && p.N <= 0x3fffffff && p.K % 128 == 0 &&
         ((uintptr_t)p.B & 15) == 0 && (p.ldb & 15) == 0 && (((uintptr_t)p.SB | p.ldsb) & 3) == 0 &&
         16 * p.ldb + p.kb < ((int64_t)1 << 30) && 16 * p.ldsb + p.nb < ((int64_t)1 << 30);
}

hipError_t launch_mx4_rows(const Mx4Args &p, int xfmt, hipStream_t st) {
  Mx4Args a = p;
  a.tiles_n = (int32_t)((a.N + 15) / 16);
  const dim3 grid((unsigned)(a.tiles_n < 512 ? a.tiles_n : 512)), block(kRowThreads);  // two per CU
  if (xfmt == FMT_F32)
    hipLaunchKernelGGL((gemm_mx4_rows_kernel<FMT_F32>), grid, block, 0, st, a);
  else if (xfmt == FMT_F16)
    hipLaunchKernelGGL((gemm_mx4_rows_kernel<FMT_F16>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((gemm_mx4_rows_kernel<FMT_BF16>), grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace tsm
