// Mid-size products of microscaled 4-bit codes for gfx950: T x T tiles of C (T = 64 or
// 128), for K a multiple of 128, 16-byte aligned rows of codes and 4-byte aligned rows
// of scales.  (gemm_mx4.hip covers other operands.)
//
// Four waves own a quarter of the tile each.  Slabs of 256 elements (128 bytes of a row)
// and their scales go global -> LDS with direct copies on a ring of D stages, D - 1
// slabs ahead: what bounds a tile that has a CU to itself is the way of a slab from
// memory, so as many of them as LDS holds are under way.  Where there is room for it two
// slabs, 256 neighbouring bytes of each row, are requested together, which memory serves
// faster (256 x 8192 x 8192 29 us, one at a time 34.2; T = 128 has room for one ahead
// so, 42 against 35).
//
// The fragments are those of the 256-tiles (gemm_mx4_tile.hip): a lane takes blocks
// 4h .. 4h + 3 of a slab's eight (h = lane / 32), whose scales are one word.
//
// Each sub-slice's fragments are read while the one before is multiplied; that alone
// gains nothing here.  Measured (us, bf16 out): 128 x 8192 x 8192 18.9, 256 x 8192 x 8192
// 29 (T = 64); 512 x 8192 x 8192 35, 2048 x 2048 x 4096 17.8, 1.9 PFLOP/s (T = 128).  With
// operands from the Infinity Cache these are 14.0, 22.3, 28.5: the rest is memory, which
// serves 128 or 256 bytes of a row at a time.  The MFMAs are busy for 6-17% of the cycles:
// only tiles that reuse more per byte (256 x 256, or these with K split between workgroups)
// would take fewer bytes.
#include "lds_ring.hpp"
#include "mx4_common.hpp"

namespace tsm {
namespace {

constexpr int BK = 128;  // bytes of codes per slab and row

// f(j + d, d) while j + d < n, d below D - 1.
template <int D, int I = 0, class F>
__device__ __forceinline__ void last_turn(int j, int n, F &&f) {
  if constexpr (I < D - 1) {
    if (j + I < n) {  // uniform
      f(j + I, Const<I>{});
      last_turn<D, I + 1>(j, n, f);
    }
  }
}

// REST: the workgroups take the parts of the 256-tiles that whole_rounds leaves.
template <int T, int D, int FMT, bool REST>
__device__ __forceinline__ void ring(const Mx4Args &p) {
  constexpr int W = T / 2, NB = W / 32;  // wave tile, 32 x 32 blocks per dimension
  constexpr int L = T / 32;              // wave-loads (1 KiB: 8 rows) per wave, operand and slab
  constexpr int S = T / 64;              // wave-loads of scales (256 bytes: 32 rows) per wave and slab
  constexpr int N = 2 * L + S;
  // slabs are requested two at a time (not by tiles that come after whole rounds: 4112 x 4096 x 4096 48 us,
  // one at a time 46)
  constexpr bool PAIR = T == 64 && !REST;
  constexpr int CODES = T * BK, BYTES = 2 * CODES + 2 * T * 8;  // of an operand, of a stage
  // an array each: a read waits for the copies into its array, as the compiler sees to it
  __shared__ __attribute__((aligned(1024))) char s0[BYTES], s1[BYTES], s2[BYTES], s3[BYTES], s4[BYTES], s5[BYTES],
      s6[BYTES], s7[BYTES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  int tm, tn;
  int64_t z;
  if constexpr (REST) {
    constexpr int P = 256 / T;
    const int all = tiles_of<256>(p), pid = (int)whole_rounds(all, p.cus, kFewMx4Tiles) + (int)(blockIdx.x / (P * P));
    if (pid >= all) return;  // uniform
    tile_at<256>(p, pid, tile_group(p), z, tm, tn);
    tm = P * tm + (int)blockIdx.x / P % P;
    tn = P * tn + (int)blockIdx.x % P;
  } else {
    if (!tile_of<T>(p, 8, z, tm, tn)) return;  // uniform
  }
  const int64_t m0 = (int64_t)tm * T, n0 = (int64_t)tn * T;
  const int64_t M = valid_rows(p, z);
  if (REST && (m0 >= M || n0 >= p.N)) return;  // uniform
  const int vr = (int)(M - m0 < T ? M - m0 : T), vc = (int)(p.N - n0 < T ? p.N - n0 : T);
  // resources over the valid rows of the two panels (rows past them load as zeros); the host keeps each below 1 GiB
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.A + z * p.strideA + m0 * p.lda, (uint32_t)((vr - 1) * p.lda + p.kb));
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.B + z * p.strideB + n0 * p.ldb, (uint32_t)((vc - 1) * p.ldb + p.kb));
  const __amdgpu_buffer_rsrc_t rs =
      wave < 2 ? make_rsrc(p.SA + z * p.strideSA + m0 * p.ldsa, (uint32_t)((vr - 1) * p.ldsa + p.nb))
               : make_rsrc(p.SB + z * p.strideSB + n0 * p.ldsb, (uint32_t)((vc - 1) * p.ldsb + p.nb));
  // this wave's copies: rows 8 g + lane / 8 of a panel, the chunk whose swizzled position is lane % 8
  uint32_t offa[L], offb[L], offs[S];
  int chunk[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int row = (wave * L + i) * 8 + (lane >> 3);
    chunk[i] = swz<2>(row, lane & 7) * 16;
    offa[i] = (uint32_t)(row * p.lda + chunk[i]);
    offb[i] = (uint32_t)(row * p.ldb + chunk[i]);
  }
  // waves 0 and 1 copy A's scales, 2 and 3 B's: word lane / 32 of row lane % 32 of a block of 32 rows
  const int half = lane >> 5;
#pragma unroll
  for (int i = 0; i < S; ++i)
    offs[i] = (uint32_t)((((wave & 1) * S + i) * 32 + (lane & 31)) * (wave < 2 ? p.ldsa : p.ldsb) + half * 4);
  const int nk = (int)((p.kb + BK - 1) / BK);
  int codes_at = wave * (L * 1024), scales_at = 2 * CODES + wave * (S * 256);
  auto stage = [&](int d) -> char * {
    return d == 0 ? s0 : d == 1 ? s1 : d == 2 ? s2 : d == 3 ? s3 : d == 4 ? s4 : d == 5 ? s5 : d == 6 ? s6 : s7;
  };
  // Slab j into stage d: part 0 A's codes, 1 B's, 2 the scales.  Chunks past K, and slabs past the end, copy zeros without
  // touching memory (their scales too).
  auto fetch = [&](int j, int d, auto part) {
    const int left = j < nk ? (int)(p.kb - (int64_t)j * BK) : 0, at = left ? j * BK : 0;
    asm volatile("" : "+s"(codes_at), "+s"(scales_at));  // (an address in a register for every copy would spill)
    if constexpr (part.value == 0) {
#pragma unroll
      for (int i = 0; i < L; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void *)(stage(d) + codes_at + i * 1024), 16,
                                                 chunk[i] < left ? offa[i] : kOutside, at, 0, 0);
    }
    if constexpr (part.value == 1) {
#pragma unroll
      for (int i = 0; i < L; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void *)(stage(d) + CODES + codes_at + i * 1024), 16,
                                                 chunk[i] < left ? offb[i] : kOutside, at, 0, 0);
    }
    if constexpr (part.value == 2) {
#pragma unroll
      for (int i = 0; i < S; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)(stage(d) + scales_at + i * 256), 4,
                                                 half * 64 < left ? offs[i] : kOutside, at / 16, 0, 0);
    }
  };

  f32x16 acc[NB][NB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x16{};
  const int r32 = lane & 31;
  // fragments of two sub-slices, scales of two slabs (zeros before the first)
  u32x4 fa[2][NB], fb[2][NB];
  uint32_t ea[2][NB], eb[2][NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) fa[1][i] = fb[1][i] = u32x4{}, ea[1][i] = eb[1][i] = 0;
  // (B, A): a lane's accumulator holds groups of 4 consecutive columns of one row of C
  auto multiply = [&](auto u, const uint32_t(&sa)[NB], const uint32_t(&sb)[NB]) {
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int k = 0; k < NB; ++k)
        acc[i][k] = mfma_mx4_32<u.value>(fb[u.value & 1][k], sb[k], fa[u.value & 1][i], sa[i], acc[i][k]);
  };
  // Slab j in stage d: each sub-slice's fragments are read, and a part of slab j + D - 1 requested, while the one before
  // is multiplied.
  auto slab = [&](int j, auto d) {
    const char *const s = stage(d.value);
    unrolled<4>([&](auto u) {
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (u.value == 0) {
        // it is here, and every wave is past its reads of the one before, whose stage is refilled.  (A pair's copies go out
        // in any order, so its first slab waits for both.)
        constexpr int newer = PAIR && d.value % 2 == 0 ? N * (D - 4) : N * (D - 2);
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(newer) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      }
      // (opaque offsets: a read that the compiler can tell apart from a stage's first copy makes it wait for every copy)
      int at = r32 * BK + swz<2>(r32, 4 * half + u.value) * 16;
      asm("" : "+v"(at));
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        fa[u.value & 1][i] = *reinterpret_cast<const u32x4 *>(s + (wm * W + i * 32) * BK + at);
        fb[u.value & 1][i] = *reinterpret_cast<const u32x4 *>(s + CODES + (wn * W + i * 32) * BK + at);
      }
      if constexpr (u.value == 0) {
        int es = lane * 4;
        asm("" : "+v"(es));
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          ea[d.value & 1][i] = *reinterpret_cast<const uint32_t *>(s + 2 * CODES + (wm * NB + i) * 256 + es);
          eb[d.value & 1][i] = *reinterpret_cast<const uint32_t *>(s + 2 * CODES + T * 8 + (wn * NB + i) * 256 + es);
        }
      }
      if constexpr (u.value < 3 && PAIR && d.value % 2 == 0) fetch(j + D - 2, (d.value + D - 2) % D, u);
      if constexpr (u.value < 3 && !(PAIR && d.value % 2)) fetch(j + D - 1, (d.value + D - 1) % D, u);
      constexpr int e = (u.value == 0 ? d.value + 1 : d.value) & 1;
      multiply(Const<(u.value + 3) % 4>{}, ea[e], eb[e]);
      if constexpr (NB == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          __builtin_amdgcn_sched_group_barrier(SG_MFMA, 1, 0);
          __builtin_amdgcn_sched_group_barrier(SG_DS_READ, 1, 0);
          __builtin_amdgcn_sched_group_barrier(SG_VMEM_READ, 1, 0);
        }
      }
    });
  };
  if constexpr (PAIR) {
    unrolled<D / 2 - 1>([&](auto d) {
      unrolled<3>([&](auto part) {
        fetch(2 * d.value, 2 * d.value, part);
        fetch(2 * d.value + 1, 2 * d.value + 1, part);
      });
    });
  } else {
    unrolled<D - 1>([&](auto d) { unrolled<3>([&](auto part) { fetch(d.value, d.value, part); }); });
  }
  // (no branch within a turn of the ring: where ways meet the compiler waits for what either has left under way)
  int j = 0;
  for (; j + D <= nk; j += D) unrolled<D>([&](auto d) { slab(j + d.value, d); });
  last_turn<D>(j, nk, slab);
  {
    uint32_t sa[NB], sb[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) sa[i] = nk & 1 ? ea[0][i] : ea[1][i], sb[i] = nk & 1 ? eb[0][i] : eb[1][i];
    multiply(Const<3>{}, sa, sb);
    // (here, by all lanes, and not where only those with rows to store are left)
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int k = 0; k < NB; ++k) asm volatile("" : "+a"(acc[i][k]));
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the copies of zeros past the end
  const Epilogue ep{p.act, p.slope, false};
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int m = wm * W + i * 32 + r32;
    if (m >= vr) continue;
    char *const row = (char *)p.C + (z * p.strideC + (m0 + m) * p.ldc) * fmt_bytes(FMT);
#pragma unroll
    for (int k = 0; k < NB; ++k) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = wn * W + k * 32 + 8 * q + 4 * half;
        const f32x16 v = acc[i][k];
        if (n < vc)
          store_mx4<FMT>(p, ep, row, n0 + n, f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]});
      }
    }
  }
}

template <int T, int D, int FMT, bool REST = false>
__global__ __launch_bounds__(256) void gemm_mx4_ring_kernel(Mx4Args p) {
  ring<T, D, FMT, REST>(p);
}

template <int T, int D>
hipError_t ring_t(const Mx4Args &p, hipStream_t stream) {
  return over_tiles(p, T, T, 256, [&](const Mx4Args &a, dim3 grid) {
    if (a.fmt == FMT_F32)
      hipLaunchKernelGGL((gemm_mx4_ring_kernel<T, D, FMT_F32>), grid, dim3(256), 0, stream, a);
    else if (a.fmt == FMT_F16)
      hipLaunchKernelGGL((gemm_mx4_ring_kernel<T, D, FMT_F16>), grid, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((gemm_mx4_ring_kernel<T, D, FMT_BF16>), grid, dim3(256), 0, stream, a);
  });
}

}  // namespace

hipError_t launch_mx4_rest(const Mx4Args &a, int64_t tiles, hipStream_t stream) {
  const dim3 grid((unsigned)(tiles * 16)), block(256);
  if (a.fmt == FMT_F32)
    hipLaunchKernelGGL((gemm_mx4_ring_kernel<64, 4, FMT_F32, true>), grid, block, 0, stream, a);
  else if (a.fmt == FMT_F16)
    hipLaunchKernelGGL((gemm_mx4_ring_kernel<64, 4, FMT_F16, true>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((gemm_mx4_ring_kernel<64, 4, FMT_BF16, true>), grid, block, 0, stream, a);
  return hipPeekAtLastError();
}

// Rings of 8 stages where every tile has a CU to itself, of 4 where two share one (us, 8 | 4: 128 x 8192 x 8192, 256 tiles,
// 18.9 | 20.5; 256 x 8192 x 8192, 512 tiles, 33.5 | 28.5).
hipError_t launch_mx4_ring(const Mx4Args &p, int tile, hipStream_t stream) {
  if (tile == 128) return ring_t<128, 4>(p, stream);
  const int64_t tiles = ((p.M + 63) / 64) * ((p.N + 63) / 64);
  return p.batch <= 256 && tiles * p.batch <= 256 ? ring_t<64, 8>(p, stream) : ring_t<64, 4>(p, stream);
}

}  // namespace tsm
