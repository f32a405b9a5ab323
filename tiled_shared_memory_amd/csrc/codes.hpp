// Pieces shared by the products of codes (int8, microscaled 4-bit): loads of
// rows of bytes, the activation, and which tile a workgroup works on.  Args is
// I8Args or Mx4Args.
#pragma once

#include "elems.hpp"
#include "gemm_internal.hpp"
#include "mfma.hpp"

namespace tsm {

__device__ __forceinline__ u32x4 load16(const int8_t *p) {
  const Raw16 r = *(const Raw16 *)p;
  return u32x4{r.d[0], r.d[1], r.d[2], r.d[3]};
}

// 16 codes without their first `drop`, zeros behind the others (drop <= 0: as they are).
__device__ __forceinline__ u32x4 drop_front(u32x4 v, int drop) {
  if (drop <= 0) return v;
  if (drop >= 16) return u32x4{};
  const uint64_t lo = (uint64_t)v[0] | ((uint64_t)v[1] << 32), hi = (uint64_t)v[2] | ((uint64_t)v[3] << 32);
  uint64_t a, b;
  if (drop >= 8) {
    a = hi >> (8 * (drop - 8));
    b = 0;
  } else {
    a = (lo >> (8 * drop)) | (hi << (64 - 8 * drop));
    b = hi >> (8 * drop);
  }
  return u32x4{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)};
}

// Codes k .. k+15 of a row of K, zeros past K; nothing outside the row is read.
__device__ __forceinline__ u32x4 load_tail(const int8_t *row, int64_t k, int64_t K) {
  if (k + 16 <= K) return load16(row + k);
  u32x4 v = {};
  if (k >= K) return v;
  if (K >= 16) return drop_front(load16(row + K - 16), (int)(16 - (K - k)));
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (k + i < K) v[i >> 2] |= (uint32_t)(uint8_t)row[k + i] << (8 * (i & 3));
  return v;
}

// The activation of a scaled sum.  Epilogue::apply, except that a NaN stays one
// with every activation (a token of NaN scale must show in its results).
__device__ __forceinline__ float act_codes(const Epilogue &ep, float v) {
  if (ep.act == 0) return v;
  return v <= 0.f ? (ep.act == 1 ? 0.f : v * ep.slope) : v;
}

// Rows of problem z (a grouped call's count, clamped to [0, M]).
template <class Args>
__device__ __forceinline__ int64_t valid_rows(const Args &p, int64_t z) {
  if (!p.rows) return p.M;
  const int64_t r = p.rows[z];
  return r < 0 ? 0 : (r > p.M ? p.M : r);
}

// ---- grouped calls: which group a tile belongs to, by the counts in device memory ----
// Row tiles of group z0 + g (0 past the launch's groups).
template <int BM, class Args>
__device__ __forceinline__ int group_tiles(const Args &p, int g) {
  return g < p.nz ? (int)((valid_rows(p, p.z0 + g) + BM - 1) / BM) : 0;
}

// Inclusive sums over the lanes of a wave.
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d, 64);
    if (lane >= d) v += o;
  }
  return v;
}

// Row tiles of all of a launch's groups, 64 groups at a time (a loop over single
// counts takes a memory latency each: 256 groups of 16 rows x 1024 x 2048 took
// 345 us so, against 104 without counts).
template <int BM, class Args>
__device__ __forceinline__ int all_group_tiles(const Args &p, int lane) {
  int sum = 0;
  for (int g = 0; g < p.nz; g += 64) sum += group_tiles<BM>(p, g + lane);
  return __builtin_amdgcn_readlane(wave_scan(sum, lane), 63);
}

// Group (from z0), its row tiles, and the tile within it, of tile t of the launch (t below the total).
template <int BM, class Args>
__device__ __forceinline__ void find_group(const Args &p, int lane, int &t, int &g, int &tiles) {
  for (g = 0;; g += 64) {
    const int v = group_tiles<BM>(p, g + lane) * p.tiles_n;
    const int s = wave_scan(v, lane), all = __builtin_amdgcn_readlane(s, 63);
    if (t < all) {
      const int l = __builtin_ctzll(__ballot(s > t));
      t -= __builtin_amdgcn_readlane(s - v, l);
      tiles = __builtin_amdgcn_readlane(v, l) / p.tiles_n;
      g += l;
      return;
    }
    t -= all;
  }
}

// Fewer than this many 256-tiles left over from whole rounds of the CUs run as
// 128-tiles in a second launch: a round takes as long for one tile as for all
// (2304 x 2304 x 1024, 81 tiles: 19.4 us against 21.1 in 128-tiles; 2048 x 2048 x
// 2048, 64 tiles: 27.7 against 17.3).
// (cus = 0: every tile stays.)
constexpr int kFewTiles = 72;
__host__ __device__ inline int64_t whole_rounds(int64_t tiles, int64_t cus, int64_t few = kFewTiles) {
  if (!cus) return tiles;
  const int64_t left = tiles % cus;
  return left < few ? tiles - left : tiles;
}

// Tile rows per group of the 256-tiles' order: 4 from 32 tile rows up, else 8 (as the 16-bit kernel).
template <class Args>
__device__ __forceinline__ int tile_group(const Args &p) { return p.tiles_m >= 32 && !p.rows ? 4 : 8; }

// Tile pid of problem-after-problem order, BM rows of a problem's rows each.
template <int BM, class Args>
__device__ __forceinline__ void tile_at(const Args &p, int pid, int group_m, int64_t &z, int &tm, int &tn) {
  int tiles = p.tiles_m;
  if (p.rows) {
    int g;
    find_group<BM>(p, threadIdx.x & 63, pid, g, tiles);
    z = p.z0 + g;
  } else {
    const int T = p.tiles_m * p.tiles_n;
    z = p.z0 + pid / T;
    pid %= T;
  }
  tile_order(pid, tiles, p.tiles_n, group_m, tm, tn);
}
template <int BM, class Args>
__device__ __forceinline__ int tiles_of(const Args &p) {
  return (p.rows ? all_group_tiles<BM>(p, threadIdx.x & 63) : p.tiles_m * p.nz) * p.tiles_n;
}

// Where a workgroup of a flat grid works: problem z, tile (tm, tn) in the
// grouped tile order, the grid regrouped per XCD.  Grouped calls number only
// the tiles that hold rows, so the real work spreads evenly over the XCDs;
// false: nothing to do.  WHOLE: only the tiles of whole_rounds.
template <int BM, bool WHOLE = false, int FEW = kFewTiles, class Args>
__device__ __forceinline__ bool tile_of(const Args &p, int group_m, int64_t &z, int &tm, int &tn) {
  int V = tiles_of<BM>(p);
  if (WHOLE) V = (int)whole_rounds(V, p.cus, FEW);
  if ((int)blockIdx.x >= V) return false;
  tile_at<BM>(p, xcd_remap(blockIdx.x, V), group_m, z, tm, tn);
  return true;
}

// One 1-D grid of workgroups of `threads` over the tiles of as many problems as
// keep its work-items below 2^32 (the host checks that one problem does).
template <class Args, class F>
hipError_t over_tiles(Args a, int tile_m, int tile_n, int threads, F &&launch) {
  a.tiles_m = (int32_t)((a.M + tile_m - 1) / tile_m);
  a.tiles_n = (int32_t)((a.N + tile_n - 1) / tile_n);
  const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
  const int64_t most = 0xffffffffLL / threads / tiles;
  for (int64_t z0 = 0; z0 < a.batch; z0 += most) {
    const int64_t nz = a.batch - z0 < most ? a.batch - z0 : most;
    a.z0 = z0;
    a.nz = (int32_t)nz;
    launch(a, dim3((unsigned)(tiles * nz)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace tsm
