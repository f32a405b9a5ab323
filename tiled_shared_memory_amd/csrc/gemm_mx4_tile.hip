// Large-tile products of microscaled 4-bit codes for gfx950: 256 x 256 tiles of C,
// for K a multiple of 128, 16-byte aligned rows of codes and 4-byte aligned rows of
// scales, on problems whose tiles fill most of the chip.  (gemm_mx4.hip covers
// everything else.)
//
// The blocking is that of the large-tile int8 kernel (gemm_i8_tile.hip), with
// v_mfma_scale_f32_32x32x64_f8f6f4: a 256-thread workgroup, one wave per 128 x 128
// quadrant (4 x 4 blocks of 32 x 32, 256 float32 accumulators per lane); slabs of 256
// elements (128 bytes of a row) go global -> LDS with direct copies, A on a 3-stage
// ring and B on a 2-stage one (160 KiB); each 64-deep sub-slice's fragments are read
// while the previous one's 16 MFMAs run.
//
// The 32 x 32 form, because a wave alone on its SIMD issues it at the full rate and
// the 16 x 16 one at little more than half of it (a loop of nothing else, codes of
// zeros: 9.8 and 5.4 PFLOP/s; random codes, which the power limit slows, 6.5 and 5.0).
//
// Scales go straight to registers, four slabs at a time: of each of its 8 fragments'
// rows a lane loads the 16 bytes of its half (h = lane / 32) of the four slabs'
// scales, and two exchanges between the halves of the wave leave it with one word a
// slab, blocks 4h .. 4h + 3 of the slab's eight.  Those are the blocks that it takes
// in the four sub-slices, in both operands, and the matrix instruction picks the
// byte.
//
// Measured: 8192 x 8192 x 8192 227-250 us, 4.4-4.8 PFLOP/s, MFMAs busy for 61% of the
// cycles.  Power bounds it: codes of zeros take 94 us for 4096 x 4096 x 16384 where
// Gaussian ones take 119, a unit of K costs the same at every size (5.1 PFLOP/s), and
// what fills the gaps between tiles gains nothing (workgroups that stay and request the
// next tile's first slabs before they store, as they are or started one after another:
// 248-251 where these take 248).  Fewer rounds: 4096 x 4096 x 4096 37 us.
//
// K's last slab, which may hold half of its elements, comes first, so that its zeros
// and its scales are the prologue's business and the loop has no branch for them.
#include "lds_ring.hpp"
#include "mx4_common.hpp"

namespace tsm {
namespace {

constexpr int BM = 256, BN = 256, BK = 128;  // BK: bytes of codes, 256 elements
constexpr int STAGE_BYTES = BM * BK;         // 32 KiB
constexpr int LOADS = 8;                     // 1 KiB wave-loads per slab, operand and wave

__shared__ __attribute__((aligned(1024))) char s_a0[STAGE_BYTES], s_a1[STAGE_BYTES], s_a2[STAGE_BYTES];
__shared__ __attribute__((aligned(1024))) char s_b0[STAGE_BYTES], s_b1[STAGE_BYTES];
__device__ __forceinline__ char *stage_a(int s) { return s == 0 ? s_a0 : s == 1 ? s_a1 : s_a2; }
__device__ __forceinline__ char *stage_b(int s) { return s == 0 ? s_b0 : s_b1; }

struct Ctx {
  __amdgpu_buffer_rsrc_t ra, rb, rsa, rsb;
  uint32_t offA[LOADS], offB[LOADS], offSA[4], offSB[4];
  int nk, wave, wm, wn, lane;  // nk: slabs
};
struct Frags {
  u32x4 a[4], b[4];
};
// Words of scales of four slabs for each of a wave's blocks of 32 rows: as loaded, and by slab.
struct Scales {
  u32x4 a[4], b[4];
};
struct Acc {
  f32x16 v[4][4];
};

// Sub-slice U of a slab: rows (lane % 32) + 32 i, chunk (block) 4 (lane / 32) + U.
template <int U>
__device__ __forceinline__ void read_frags(const char *sa, const char *sb, Frags &f, const Ctx &c) {
  const int row = c.lane & 31, chunk = swz<2>(row, 4 * (c.lane >> 5) + U) * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f.a[i] = *reinterpret_cast<const u32x4 *>(sa + (c.wm * 128 + i * 32 + row) * BK + chunk);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    f.b[j] = *reinterpret_cast<const u32x4 *>(sb + (c.wn * 128 + j * 32 + row) * BK + chunk);
}

// The scales of K's slabs 4 quad .. 4 quad + 3.  (A lane's 16 bytes may lie partly or wholly past a row's end: past the
// resource they load as zeros, before its end they are another row's; no slab uses them.)
__device__ __forceinline__ void load_scales(const Ctx &c, int quad, Scales &s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s.a[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(c.rsa, c.offSA[i], quad * 32, 0));
    s.b[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(c.rsb, c.offSB[i], quad * 32, 0));
  }
}
// Words 0, 1, 2, 3 (of lanes below 32) and 4, 5, 6, 7 (of the others) of a row, to those of slabs 0..3: 0 2 4 6 and
// 1 3 5 7.
__device__ __forceinline__ u32x4 by_slab(u32x4 v) {
  const auto p = __builtin_amdgcn_permlane32_swap(v[0], v[1], false, false);  // 0 1 and 4 5
  const auto q = __builtin_amdgcn_permlane32_swap(v[2], v[3], false, false);  // 2 3 and 6 7
  return u32x4{p[0], q[0], p[1], q[1]};
}
__device__ __forceinline__ void arrange(Scales &to, const Scales &from) {
#pragma unroll
  for (int i = 0; i < 4; ++i) to.a[i] = by_slab(from.a[i]), to.b[i] = by_slab(from.b[i]);
}

// Sub-slice U of a slab, scales of slab W of four.  Operands as (B, A): a lane's accumulator holds groups of 4
// consecutive columns of one row of C.  FIRST: from zeros.
template <int U, int W, bool FIRST = false>
__device__ __forceinline__ void mma(const Frags &f, const Scales &s, Acc &acc) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc.v[i][j] = mfma_mx4_32<U>(f.b[j], s.b[j][W], f.a[i], s.a[i][W], FIRST ? f32x16{} : acc.v[i][j]);
}

// Sub-slice U of slab j = J (mod 12), which is K's slab j - 1 (the first: K's last): A in stage J % 3, B in stage J % 2,
// scales (J + 3) % 4.  U = 0 waits for slab j (only A's copies of slab j + 1 may still be in flight), passes the barrier
// and refills the B stage that slab j - 1 freed; U = 2 refills the A stage that it freed, two slabs ahead.  At the first
// slab of four, U = 1 takes over the scales (the last slab's were used until then) and requests the next.  MODE 1: the
// tile's first sub-slice (nothing to multiply yet); MODE 2: the second (starts the sums).
template <int J, int U, int MODE = 0>
__device__ __forceinline__ void substep(Ctx &c, int j, Frags (&fr)[2], Scales &sc, Scales &next, Acc &acc) {
  constexpr int SA = J % 3, SB = J % 2, V = (U + 3) % 4;  // V: the sub-slice that is multiplied
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (U == 0) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LOADS) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
  if constexpr (U == 1 && J % 4 == 1) {
    arrange(sc, next);
    load_scales(c, (j >> 2) + 1, next);
  }
  read_frags<U>(stage_a(SA), stage_b(SB), fr[U & 1], c);
  // past the end the last one again: the count of copies in flight stays the same
  if constexpr (U == 0) issue<LOADS>(c.rb, c.offB, (uint32_t)max(min(j, c.nk - 2), 0) * BK, stage_b(SB ^ 1), c.wave);
  if constexpr (U == 2) issue<LOADS>(c.ra, c.offA, (uint32_t)max(min(j + 1, c.nk - 2), 0) * BK, stage_a((SA + 2) % 3), c.wave);
  if constexpr (MODE == 0) mma<V, (U ? J + 3 : J + 2) % 4>(fr[V & 1], sc, acc);
  if constexpr (MODE == 2) mma<V, (J + 3) % 4, true>(fr[V & 1], sc, acc);
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    __builtin_amdgcn_sched_group_barrier(SG_MFMA, 1, 0);
    __builtin_amdgcn_sched_group_barrier(SG_DS_READ, 1, 0);
    __builtin_amdgcn_sched_group_barrier(SG_MFMA, 1, 0);
    __builtin_amdgcn_sched_group_barrier(SG_VMEM_READ, 1, 0);
  }
}

template <int J>
__device__ __forceinline__ void slab(Ctx &c, int j, Frags (&fr)[2], Scales &sc, Scales &next, Acc &acc) {
  substep<J, 0>(c, j, fr, sc, next, acc);
  substep<J, 1>(c, j, fr, sc, next, acc);
  substep<J, 2>(c, j, fr, sc, next, acc);
  substep<J, 3>(c, j, fr, sc, next, acc);
}

// Sixteen bytes of results, of which the first n are stored, anywhere.
template <int FMT>
__device__ __forceinline__ void store_any(char *at, u32x4 d, int n) {
  constexpr int PER = 16 / fmt_bytes(FMT);
  struct __attribute__((packed, aligned(2))) Any {
    u32x4 v;
  };
  if (n >= PER) {
    reinterpret_cast<Any *>(at)->v = d;
    return;
  }
#pragma unroll
  for (int e = 0; e < PER - 1; ++e)
    if (e < n) put_bits<FMT>(at, e, FMT == FMT_F32 ? d[e] : d[e / 2] >> (e % 2 * 16) & 0xffff);
}

constexpr int kNonTemporal = 2;  // buffer-store cache policy: C is written once and not read again

template <int FMT>
__global__ __launch_bounds__(256, 1) void gemm_mx4_tile_kernel(Mx4Args p) {
  int tm, tn;
  int64_t z;
  if (!tile_of<BM, true, kFewMx4Tiles>(p, tile_group(p), z, tm, tn)) return;  // uniform
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
  c.ra = make_rsrc(p.A + z * p.strideA + m0 * p.lda, (uint32_t)((vr - 1) * p.lda + p.kb));
  c.rb = make_rsrc(p.B + z * p.strideB + n0 * p.ldb, (uint32_t)((vc - 1) * p.ldb + p.kb));
  c.rsa = make_rsrc(p.SA + z * p.strideSA + m0 * p.ldsa, (uint32_t)((vr - 1) * p.ldsa + p.nb));
  c.rsb = make_rsrc(p.SB + z * p.strideSB + n0 * p.ldsb, (uint32_t)((vc - 1) * p.ldsb + p.nb));
  // (in units of 2 bytes: leading dimensions are multiples of 16)
  slice_offsets<LOADS, 2>(c.offA, p.lda / 2, c.wave, lane);
  slice_offsets<LOADS, 2>(c.offB, p.ldb / 2, c.wave, lane);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c.offSA[i] = (uint32_t)((wm * 128 + i * 32 + (lane & 31)) * p.ldsa + (lane >> 5) * 16);
    c.offSB[i] = (uint32_t)((wn * 128 + i * 32 + (lane & 31)) * p.ldsb + (lane >> 5) * 16);
  }
  c.nk = (int)((p.K + 2 * BK - 1) / (2 * BK));

  Acc acc;  // started by the second sub-slice
  Scales sc, next;
  Frags fr[2];
  // copies in the order the waits count on: scales, A(0), B(0), A(1), then per slab j: B(j+1), A(j+2)
  const int last = c.nk - 1, tail = (int)(p.kb - (int64_t)last * BK);  // K's last slab, its bytes of a row: 64 or 128
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // this lane's word of it, no scales where it has no elements
    const bool in = (lane >> 5) * 64 < tail;
    const uint32_t back = (uint32_t)(lane >> 5) * 12;  // offSA, offSB: of 16 bytes for each half of the lanes
    sc.a[i][3] = __builtin_amdgcn_raw_buffer_load_b32(c.rsa, in ? c.offSA[i] - back : kOutside, last * 8, 0);
    sc.b[i][3] = __builtin_amdgcn_raw_buffer_load_b32(c.rsb, in ? c.offSB[i] - back : kOutside, last * 8, 0);
  }
  load_scales(c, 0, next);
  {
    uint32_t first[LOADS];
    auto masked = [&](const uint32_t(&off)[LOADS]) {
#pragma unroll
      for (int g = 0; g < LOADS; ++g)
        first[g] = swz<2>((c.wave * LOADS + g) * 8 + (lane >> 3), lane & 7) * 16 < tail ? off[g] : kOutside;
    };
    masked(c.offA);
    issue<LOADS>(c.ra, first, (uint32_t)last * BK, s_a0, c.wave);
    masked(c.offB);
    issue<LOADS>(c.rb, first, (uint32_t)last * BK, s_b0, c.wave);
  }
  issue<LOADS>(c.ra, c.offA, 0, s_a1, c.wave);
  substep<0, 0, 1>(c, 0, fr, sc, next, acc);
  substep<0, 1, 2>(c, 0, fr, sc, next, acc);
  substep<0, 2>(c, 0, fr, sc, next, acc);
  substep<0, 3>(c, 0, fr, sc, next, acc);
  // twelve slabs per trip: A's stage repeats every 3, B's every 2, the scales' word every 4
  int j = 1;
  for (; j + 12 <= c.nk; j += 12) {
    slab<1>(c, j, fr, sc, next, acc);
    slab<2>(c, j + 1, fr, sc, next, acc);
    slab<3>(c, j + 2, fr, sc, next, acc);
    slab<4>(c, j + 3, fr, sc, next, acc);
    slab<5>(c, j + 4, fr, sc, next, acc);
    slab<6>(c, j + 5, fr, sc, next, acc);
    slab<7>(c, j + 6, fr, sc, next, acc);
    slab<8>(c, j + 7, fr, sc, next, acc);
    slab<9>(c, j + 8, fr, sc, next, acc);
    slab<10>(c, j + 9, fr, sc, next, acc);
    slab<11>(c, j + 10, fr, sc, next, acc);
    slab<12>(c, j + 11, fr, sc, next, acc);
  }
  if (j < c.nk) {
    slab<1>(c, j, fr, sc, next, acc);
    if (j + 1 < c.nk) {
      slab<2>(c, j + 1, fr, sc, next, acc);
      if (j + 2 < c.nk) {
        slab<3>(c, j + 2, fr, sc, next, acc);
        if (j + 3 < c.nk) {
          slab<4>(c, j + 3, fr, sc, next, acc);
          if (j + 4 < c.nk) {
            slab<5>(c, j + 4, fr, sc, next, acc);
            if (j + 5 < c.nk) {
              slab<6>(c, j + 5, fr, sc, next, acc);
              if (j + 6 < c.nk) {
                slab<7>(c, j + 6, fr, sc, next, acc);
                if (j + 7 < c.nk) {
                  slab<8>(c, j + 7, fr, sc, next, acc);
                  if (j + 8 < c.nk) {
                    slab<9>(c, j + 8, fr, sc, next, acc);
                    if (j + 9 < c.nk) {
                      slab<10>(c, j + 9, fr, sc, next, acc);
                      if (j + 10 < c.nk) {
                        slab<11>(c, j + 10, fr, sc, next, acc);
                      }
                    }
                  }
                }
              }
            }
          }
        }
      }
    }
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  const int w = (c.nk + 2) & 3;  // the last slab's word of the scales
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sc.a[i][0] = w == 0 ? sc.a[i][0] : w == 1 ? sc.a[i][1] : w == 2 ? sc.a[i][2] : sc.a[i][3];
    sc.b[i][0] = w == 0 ? sc.b[i][0] : w == 1 ? sc.b[i][1] : w == 2 ? sc.b[i][2] : sc.b[i][3];
  }
  mma<3, 0>(fr[1], sc, acc);                        // the last sub-slice
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the duplicate tail copies

  // ---- epilogue: acc.v[i][j], elements 4 q .. 4 q + 3, holds C[32 i + lane % 32][32 j + 8 q + 4 (lane / 32) + 0..3] of
  // the quadrant
  const int r32 = lane & 31, h = lane >> 5;
  constexpr int ES = fmt_bytes(FMT), PER = 16 / ES, CHUNKS = 128 / PER;  // results per chunk of 16 bytes, chunks per row
  const int64_t ldc = p.ldc;
  const __amdgpu_buffer_rsrc_t rc = make_rsrc((char *)p.C + (z * p.strideC + m0 * ldc + n0) * ES,
                                              (uint32_t)(((vr - 1) * ldc + vc) * ES));
  const Epilogue ep{p.act, p.slope, false};
  __syncthreads();  // every wave is past its last fragment read and copy
  // this wave's quadrant through LDS, 32 rows at a time, chunk c of row r at c ^ (r % CHUNKS); then whole rows are stored
  char *const q = c.wave == 0 ? s_a0 : c.wave == 1 ? s_a1 : c.wave == 2 ? s_b0 : s_b1;
  const int t = lane % CHUNKS, g = lane / CHUNKS, col = wn * 128 + PER * t;
  const bool whole = p.vec_store && col + PER <= vc;
  const uint32_t coff = whole ? (uint32_t)(col * ES) : kOutside;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    char *const at = q + (i * 32 * 128 * ES) % STAGE_BYTES;
#pragma unroll
    for (int j2 = 0; j2 < 4; ++j2) {
      f32x16 v = acc.v[i][j2];
      if (p.act) {  // uniform
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = act_codes(ep, v[e]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        char *const to = at + r32 * 128 * ES;
        if constexpr (FMT == FMT_F32)
          *reinterpret_cast<f32x4 *>(to + ((8 * j2 + 2 * k + h) ^ r32) * 16) =
              f32x4{v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]};
        else
          *reinterpret_cast<u32x2 *>(to + ((64 * j2 + 16 * k + 8 * h) ^ (16 * (r32 & 15)))) =
              u32x2{pack2<FMT>(v[4 * k], v[4 * k + 1]), pack2<FMT>(v[4 * k + 2], v[4 * k + 3])};
      }
    }
#pragma unroll
    for (int k = 0; k < CHUNKS / 2; ++k) {
      const int row = 64 / CHUNKS * k + g, m = wm * 128 + i * 32 + row;
      const u32x4 d = *reinterpret_cast<const u32x4 *>(at + row * 128 * ES + (t ^ (row % CHUNKS)) * 16);
      __builtin_amdgcn_raw_buffer_store_b128(d, rc, coff + (uint32_t)(m * ldc * ES), 0, kNonTemporal);
      if (!whole && m < vr) store_any<FMT>((char *)p.C + (z * p.strideC + (m0 + m) * ldc + n0 + col) * ES, d, vc - col);
    }
  }
}

}  // namespace

bool mx4_tile_supports(const Mx4Args &p) {
  if (p.K % BK || p.K == 0) return false;
  if (255 * p.lda + p.kb >= (int64_t)1 << 30 || 255 * p.ldb + p.kb >= (int64_t)1 << 30) return false;
  if (255 * p.ldsa + p.nb >= (int64_t)1 << 30 || 255 * p.ldsb + p.nb >= (int64_t)1 << 30) return false;
  if (((uintptr_t)p.A | (uintptr_t)p.B) & 15) return false;
  if (((uintptr_t)p.SA | (uintptr_t)p.SB) & 3) return false;
  if (p.lda % 16 || p.ldb % 16 || p.strideA % 16 || p.strideB % 16) return false;
  if (p.ldsa % 4 || p.ldsb % 4 || p.strideSA % 4 || p.strideSB % 4) return false;
  const int es = fmt_bytes(p.fmt);
  return 256 * p.ldc * es < (int64_t)1 << 31;  // 32-bit store offsets
}

hipError_t launch_mx4_tile(const Mx4Args &p, bool whole_only, hipStream_t stream) {
  Mx4Args q = p;
  q.cus = whole_only ? device_cus() : 0;
  // whether rows start at 4 bytes, which vector stores through a resource want
  const int64_t es = fmt_bytes(p.fmt);
  q.vec_store = (uintptr_t)p.C % 4 == 0 && p.ldc * es % 4 == 0 && p.strideC * es % 4 == 0;
  return over_tiles(q, BM, BN, 256, [&](const Mx4Args &a, dim3 grid) {
    // without counts the host knows the tiles of whole rounds
    const int64_t whole = a.rows ? (int64_t)grid.x : whole_rounds(grid.x, a.cus, kFewMx4Tiles);
    if (whole) {
      const dim3 g((unsigned)whole);
      if (a.fmt == FMT_F32)
        hipLaunchKernelGGL((gemm_mx4_tile_kernel<FMT_F32>), g, dim3(256), 0, stream, a);
      else if (a.fmt == FMT_F16)
        hipLaunchKernelGGL((gemm_mx4_tile_kernel<FMT_F16>), g, dim3(256), 0, stream, a);
      else
        hipLaunchKernelGGL((gemm_mx4_tile_kernel<FMT_BF16>), g, dim3(256), 0, stream, a);
      if (hipPeekAtLastError() != hipSuccess) return;
    }
    if (whole_only && (a.rows || whole < (int64_t)grid.x)) {
      Mx4Args b = a;
      b.vec_store = p.vec_store;  // (of 4 elements there)
      const hipError_t e = launch_mx4_rest(b, a.rows ? kFewMx4Tiles - 1 : (int64_t)grid.x - whole, stream);
      (void)e;  // the launch's error is the last one
    }
  });
}

}  // namespace tsm
