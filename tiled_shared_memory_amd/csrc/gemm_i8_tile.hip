// Large-tile int8 products for gfx950: 256 x 256 tiles of C, for K a multiple of
// 128, N of 8 and 16-byte aligned rows, on problems whose tiles fill most of the
// chip.  (gemm_i8.hip covers everything else.)
//
// The blocking is that of the 16-bit large-tile kernel (gemm_tile.hip): a slab of
// 128 codes has the bytes of a slab of 64 16-bit elements, and
// v_mfma_i32_16x16x64_i8 does twice the work of the 16-bit form on the same
// operand registers in the same time.  A 256-thread workgroup, one wave per
// 128 x 128 quadrant, 256 int32 accumulators per lane; slabs go global -> LDS
// with direct copies, A on a 3-stage ring and B on a 2-stage one (160 KiB), each
// half of a slab issuing half of the copies; each 64-deep sub-slice's fragments
// are read while the previous one's 64 MFMAs run.
//
// Sums are int32, so the order of K never shows.  The epilogue multiplies each
// by its token's and its channel's scale on the way out; a 16-bit C leaves
// through LDS as whole non-temporal lines.
//
// 8192^3 with bf16 output: 0.371-0.397 ms = 2.8-3.0 POP/s over boxes.  The MFMAs'
// own time is 55 us of the 93 per round of 256 tiles at 2.4 GHz; under sustained
// load the clock is lower, and by the counters the MFMAs are busy in 72% of its
// cycles, the LDS with reads in 20% (3% of that bank conflicts).  What is left is
// waits: at each slab's barrier, for the first slabs and the output's stores of
// each round.  The scales are requested together at the end of the loop; one column
// block after another they cost 3% (0.382 against 0.371 ms on one box).
#include "i8_common.hpp"
#include "lds_ring.hpp"

namespace tsm {
namespace {

constexpr int BM = 256, BN = 256, BK = 128;
constexpr int STAGE_BYTES = BM * BK;  // 32 KiB
constexpr int LOADS = 8;              // 1 KiB wave-loads per slab, operand and wave

__shared__ __attribute__((aligned(1024))) char s_a0[STAGE_BYTES], s_a1[STAGE_BYTES], s_a2[STAGE_BYTES];
__shared__ __attribute__((aligned(1024))) char s_b0[STAGE_BYTES], s_b1[STAGE_BYTES];
__device__ __forceinline__ char *stage_a(int s) { return s == 0 ? s_a0 : s == 1 ? s_a1 : s_a2; }
__device__ __forceinline__ char *stage_b(int s) { return s == 0 ? s_b0 : s_b1; }

struct Ctx {
  __amdgpu_buffer_rsrc_t ra, rb;
  uint32_t offA[LOADS], offB[LOADS];
  int nk, wave, wm, wn, lane;
};
struct Frags {
  u32x4 a[8], b[8];
};
struct Acc {
  i32x4 v[8][8];
};

// Sub-slice U (codes 64 U .. 64 U + 63) of a slab: rows (lane % 16) + 16 i, chunk 4 U + lane / 16.
template <int U>
__device__ __forceinline__ void read_frags(const char *sa, const char *sb, Frags &f, const Ctx &c) {
  const int row = c.lane & 15, chunk = swz<2>(c.lane, 4 * U + (c.lane >> 4)) * 16;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    f.a[i] = *reinterpret_cast<const u32x4 *>(sa + (c.wm * 128 + i * 16 + row) * BK + chunk);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    f.b[j] = *reinterpret_cast<const u32x4 *>(sb + (c.wn * 128 + j * 16 + row) * BK + chunk);
}

// Operands as (B, A): a lane's accumulator holds 4 consecutive columns of one row of C.  FIRST: from zeros.
template <bool FIRST>
__device__ __forceinline__ void mma(const Frags &f, Acc &acc) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc.v[i][j] = mfma_i8(f.b[j], f.a[i], FIRST ? i32x4{} : acc.v[i][j]);
}

// Sub-slice U of slab j, A in stage SA = j % 3, B in stage SB = j % 2.  U = 0
// waits for slab j (only A's copies of slab j+1 may still be in flight), passes
// the barrier and refills the B stage that slab j-1 freed; U = 1 refills the A
// stage that it freed, two slabs ahead.  MODE 1: the tile's first sub-slice
// (nothing to multiply yet); MODE 2: the second (its multiply starts the sums).
template <int SA, int SB, int U, int MODE = 0>
__device__ __forceinline__ void substep(Ctx &c, int j, Frags (&fr)[2], Acc &acc) {
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (U == 0) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LOADS) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
  read_frags<U>(stage_a(SA), stage_b(SB), fr[U], c);
  // past the end the last slab again: the count of copies in flight stays the same
  if constexpr (U == 0)
    issue<LOADS>(c.rb, c.offB, (uint32_t)min(j + 1, c.nk - 1) * BK, stage_b(SB ^ 1), c.wave);
  else
    issue<LOADS>(c.ra, c.offA, (uint32_t)min(j + 2, c.nk - 1) * BK, stage_a((SA + 2) % 3), c.wave);
  if constexpr (MODE == 0) mma<false>(fr[U ^ 1], acc);
  if constexpr (MODE == 2) mma<true>(fr[U ^ 1], acc);
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    __builtin_amdgcn_sched_group_barrier(SG_MFMA, 2, 0);
    __builtin_amdgcn_sched_group_barrier(SG_DS_READ, 1, 0);
    __builtin_amdgcn_sched_group_barrier(SG_MFMA, 2, 0);
    __builtin_amdgcn_sched_group_barrier(SG_VMEM_READ, 1, 0);
    __builtin_amdgcn_sched_group_barrier(SG_MFMA, 2, 0);
    __builtin_amdgcn_sched_group_barrier(SG_DS_READ, 1, 0);
    __builtin_amdgcn_sched_group_barrier(SG_MFMA, 2, 0);
  }
}

template <int J>
__device__ __forceinline__ void slab(Ctx &c, int j, Frags (&fr)[2], Acc &acc) {
  substep<J % 3, J % 2, 0>(c, j, fr, acc);
  substep<J % 3, J % 2, 1>(c, j, fr, acc);
}

constexpr int kNonTemporal = 2;  // buffer-store cache policy: C is written once and not read again

template <int FMT>
__global__ __launch_bounds__(256, 1) void gemm_i8_tile_kernel(I8Args p) {
  int tm, tn;
  int64_t z;
  if (!tile_of<BM, true>(p, tile_group(p), z, tm, tn)) return;  // uniform
  Ctx c;
  c.lane = threadIdx.x & 63;
  c.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  c.wm = c.wave >> 1;
  c.wn = c.wave & 1;
  const int lane = c.lane, wm = c.wm, wn = c.wn;
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int64_t M = valid_rows(p, z);
  const int vr = (int)(M - m0 < BM ? M - m0 : BM), vc = (int)(p.N - n0 < BN ? p.N - n0 : BN);
  // resources over the valid rows of the two panels (rows past them load as zeros); the host keeps each below 1 GiB
  c.ra = make_rsrc(p.A + z * p.strideA + m0 * p.lda, (uint32_t)((vr - 1) * p.lda + p.K));
  c.rb = make_rsrc(p.B + z * p.strideB + n0 * p.ldb, (uint32_t)((vc - 1) * p.ldb + p.K));
  // (in units of 2 bytes: leading dimensions are multiples of 16)
  slice_offsets<LOADS, 2>(c.offA, p.lda / 2, c.wave, lane);
  slice_offsets<LOADS, 2>(c.offB, p.ldb / 2, c.wave, lane);
  c.nk = (int)(p.K / BK);

  Acc acc;  // started by the second sub-slice
  // copies in the order the waits count on: A(0), B(0), A(1), then per slab j: B(j+1), A(j+2)
  issue<LOADS>(c.ra, c.offA, 0, s_a0, c.wave);
  issue<LOADS>(c.rb, c.offB, 0, s_b0, c.wave);
  issue<LOADS>(c.ra, c.offA, (uint32_t)min(1, c.nk - 1) * BK, s_a1, c.wave);
  Frags fr[2];
  substep<0, 0, 0, 1>(c, 0, fr, acc);
  substep<0, 0, 1, 2>(c, 0, fr, acc);
  // six slabs per trip: A's stage repeats every 3, B's every 2
  int j = 1;
  for (; j + 6 <= c.nk; j += 6) {
    slab<1>(c, j, fr, acc);
    slab<2>(c, j + 1, fr, acc);
    slab<3>(c, j + 2, fr, acc);
    slab<4>(c, j + 3, fr, acc);
    slab<5>(c, j + 4, fr, acc);
    slab<6>(c, j + 5, fr, acc);
  }
  if (j < c.nk) {
    slab<1>(c, j, fr, acc);
    if (j + 1 < c.nk) {
      slab<2>(c, j + 1, fr, acc);
      if (j + 2 < c.nk) {
        slab<3>(c, j + 2, fr, acc);
        if (j + 3 < c.nk) {
          slab<4>(c, j + 3, fr, acc);
          if (j + 4 < c.nk) slab<5>(c, j + 4, fr, acc);
        }
      }
    }
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  mma<false>(fr[1], acc);                           // the last sub-slice
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the duplicate tail copies

  // ---- epilogue: acc.v[i][j] holds C[16 i + lane % 16][16 j + 4 (lane / 16) + 0..3] of the quadrant
  const Epilogue ep{p.act, p.slope, false};
  const int t = lane & 15, g = lane >> 4;
  float ca[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = wm * 128 + 16 * i + t;
    ca[i] = p.sa ? p.sa[z * p.stride_sa + m0 + (r < vr ? r : vr - 1)] : 1.f;
  }
  float cb[8][4];
#pragma unroll
  for (int j2 = 0; j2 < 8; ++j2) channel_scales(p, z, n0 + wn * 128 + 16 * j2 + 4 * g, cb[j2]);
  constexpr int ES = fmt_bytes(FMT);
  const int64_t ldc = p.ldc;
  const __amdgpu_buffer_rsrc_t rc = make_rsrc((char *)p.C + (z * p.strideC + m0 * ldc + n0) * ES,
                                              (uint32_t)(((vr - 1) * ldc + vc) * ES));
  if constexpr (FMT != FMT_F32) {
    __syncthreads();  // every wave is past its last fragment read and copy
    // this wave's quadrant through LDS: 128 rows of 256 bytes, chunk c of row r at c ^ (r % 16)
    char *const q = c.wave == 0 ? s_a0 : c.wave == 1 ? s_a1 : c.wave == 2 ? s_b0 : s_b1;
#pragma unroll
    for (int j2 = 0; j2 < 8; ++j2) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = act_codes(ep, (float)acc.v[i][j2][e] * ca[i] * cb[j2][e]);
        *reinterpret_cast<u32x2 *>(q + (16 * i + t) * 256 + ((32 * j2 + 8 * g) ^ (16 * t))) =
            u32x2{f32_elem<FMT>(v[0]) | (f32_elem<FMT>(v[1]) << 16), f32_elem<FMT>(v[2]) | (f32_elem<FMT>(v[3]) << 16)};
      }
    }
    const int col = wn * 128 + 8 * t;
    const uint32_t coff = col < vc ? (uint32_t)(col * 2) : kOutside;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const int row = 4 * k + g;
      const u32x4 d = *reinterpret_cast<const u32x4 *>(q + row * 256 + (t ^ (row & 15)) * 16);
      __builtin_amdgcn_raw_buffer_store_b128(d, rc, coff + (uint32_t)((wm * 128 + row) * ldc * 2), 0, kNonTemporal);
    }
  } else {
#pragma unroll
    for (int j2 = 0; j2 < 8; ++j2) {
      const int col = wn * 128 + 16 * j2 + 4 * g;
      const uint32_t off = col < vc ? (uint32_t)(((wm * 128 + t) * ldc + col) * 4) : kOutside;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = act_codes(ep, (float)acc.v[i][j2][e] * ca[i] * cb[j2][e]);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rc, off + (uint32_t)(16 * i * ldc * 4), 0, 0);
      }
    }
  }
}

}  // namespace

bool i8_tile_supports(const I8Args &p) {
  if (p.N % 8 || p.K % BK || p.K == 0) return false;
  if (255 * p.lda + p.K >= (int64_t)1 << 30 || 255 * p.ldb + p.K >= (int64_t)1 << 30) return false;
  if (((uintptr_t)p.A | (uintptr_t)p.B | (uintptr_t)p.C) & 15) return false;
  if (p.lda % 16 || p.ldb % 16 || p.strideA % 16 || p.strideB % 16) return false;
  const int es = fmt_bytes(p.fmt);
  if (p.ldc * es % 16 || p.strideC * es % 16) return false;
  return 256 * p.ldc * es < (int64_t)1 << 31;  // 32-bit store offsets
}

hipError_t launch_i8_tile(const I8Args &p, bool whole_only, hipStream_t stream) {
  I8Args q = p;
  q.cus = whole_only ? device_cus() : 0;
  return over_tiles(q, BM, BN, 256, [&](const I8Args &a, dim3 grid) {
    // without counts the host knows the tiles of whole rounds
    const int64_t whole = a.rows ? (int64_t)grid.x : whole_rounds(grid.x, a.cus);
    if (whole) {
      const dim3 g((unsigned)whole);
      if (a.fmt == FMT_F32)
        hipLaunchKernelGGL((gemm_i8_tile_kernel<FMT_F32>), g, dim3(256), 0, stream, a);
      else if (a.fmt == FMT_F16)
        hipLaunchKernelGGL((gemm_i8_tile_kernel<FMT_F16>), g, dim3(256), 0, stream, a);
      else
        hipLaunchKernelGGL((gemm_i8_tile_kernel<FMT_BF16>), g, dim3(256), 0, stream, a);
      if (hipPeekAtLastError() != hipSuccess) return;
    }
    if (whole_only && (a.rows || whole < (int64_t)grid.x)) {
      const hipError_t e = launch_i8_rest(a, stream);
      (void)e;  // the launch's error is the last one
    }
  });
}

}  // namespace tsm
