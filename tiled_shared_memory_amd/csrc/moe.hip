// Expert routing for gfx950: tokens sorted by expert, rows into the experts'
// slabs and back, with weights, and the gradients.
//
// The slabs are what gemm_grouped multiplies: expert e owns rows
// e * capacity .. of one matrix.  Entry (t, j) is choice j of token t.
//
//   sort      pos[t][j] = e * capacity + r,  e = ids[t][j],  r = the number of
//             entries before (t, j), in token order, with the same expert;
//             -1 when e names no expert or r >= capacity
//   dispatch  slab[pos[t][j]] = X[t]
//   combine   Y[t] = sum_j w[t][j] slab[pos[t][j]]
//   backward  dslab[pos[t][j]] = w[t][j] dY[t];  dw[t][j] = <dY[t], slab[pos[t][j]]>
//
// The row operators are bound by memory; a row moves as 16-byte vectors at any
// alignment, a token's choices are requested together.  8192 tokens, 2 choices,
// 4096 bf16: dispatch 33.9 us (5.9 TB/s), combine 32.6 us (6.2 TB/s), gradients
// 52.2 us (6.4 TB/s); a large device copy reaches 5.0 TB/s.  Odd rows (4095
// elements) cost a third more.  The sort is bound by latencies and launches: 64 x 8
// entries 3.1 us in one workgroup, 65536 x 8 of 256 experts 3.2 + 9.3 us
// traced one by one, 11.6 us together.
#include "elems.hpp"
#include "moe_internal.hpp"

namespace tsm {
namespace {

// ---- sort ------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;

// Expert of flat entry i, or -1 when it names none.
template <bool ID64>
__device__ __forceinline__ int expert_of(const SortArgs &a, int64_t i) {
  const int64_t at = a.ld == a.topk ? i : i / a.topk * a.ld + i % a.topk;
  if constexpr (ID64) {
    const int64_t e = ((const int64_t *)a.ids)[at];
    return e >= 0 && e < a.experts ? (int)e : -1;
  } else {
    const int32_t e = ((const int32_t *)a.ids)[at];
    return e >= 0 && e < a.experts ? e : -1;
  }
}

// Entries per expert of each tile, into hist[tile][expert] (rows of a multiple of 4 experts).  Integer sums: the
// order of the atomics does not matter.
template <bool ID64>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a) {
  extern __shared__ int32_t sh[];
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) sh[e] = 0;
  __syncthreads();
  const int64_t n = a.tokens * a.topk, i0 = (int64_t)blockIdx.x * SortInfo::kTile;
  for (int64_t i = i0 + threadIdx.x; i < i0 + SortInfo::kTile && i < n; i += kSortThreads) {
    const int e = expert_of<ID64>(a, i);
    if (e >= 0) atomicAdd(&sh[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) a.hist[(int64_t)blockIdx.x * sort_pitch(a.experts) + e] = sh[e];
}

// Many tiles: every tile's counts to the sums of the tiles before it, a workgroup per expert.
__global__ __launch_bounds__(kSortThreads) void sort_scan_kernel(int32_t *hist, int64_t pitch, int blocks) {
  __shared__ int32_t wsum[kSortWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int32_t *col = hist + blockIdx.x;
  int32_t before = 0;
  for (int b0 = 0; b0 < blocks; b0 += kSortThreads) {
    const int b = b0 + (int)threadIdx.x;
    const int32_t v = b < blocks ? col[b * pitch] : 0;
    int32_t s = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int32_t o = __shfl_up(s, d, 64);
      if (lane >= d) s += o;
    }
    if (lane == 63) wsum[wave] = s;
    __syncthreads();
    int32_t earlier = before, all = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      if (w < wave) earlier += wsum[w];
      all += wsum[w];
    }
    if (b < blocks) col[b * pitch] = earlier + s - v;
    before += all;
    __syncthreads();  // the waves' sums are read
  }
}

// Positions of one tile's entries.  Each wave owns a run of consecutive
// entries; LDS holds, per wave and expert, first the wave's count, then the
// next rank it gives out.
template <bool ID64>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs a) {
  extern __shared__ int32_t sh[];  // [waves][experts], then [experts]: entries before this tile
  volatile int32_t *next = sh;
  int32_t *before = sh + kSortWaves * a.experts;
  const int E = a.experts, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < (kSortWaves + 1) * E; i += kSortThreads) sh[i] = 0;
  __syncthreads();
  const int64_t n = a.tokens * a.topk;
  const int64_t tile = a.hist ? SortInfo::kTile : SortInfo::kOneBlock;
  const int64_t i0 = (int64_t)blockIdx.x * tile;
  const int64_t left = n - i0 < tile ? n - i0 : tile;
  const int steps = (int)((left + kSortThreads - 1) / kSortThreads);  // 64 entries per wave and step
  const int64_t w0 = i0 + (int64_t)wave * steps * 64;
  constexpr int S = (int)(SortInfo::kOneBlock / kSortThreads);
  int own[S];  // this lane's experts
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int64_t i = w0 + s * 64 + lane;
    own[s] = s < steps && i < n && i < i0 + tile ? expert_of<ID64>(a, i) : -1;
  }
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (own[s] >= 0) atomicAdd(&sh[wave * E + own[s]], 1);
  if (a.scanned) {
    for (int e = threadIdx.x; e < E; e += kSortThreads) before[e] = a.hist[(int64_t)blockIdx.x * sort_pitch(E) + e];
  } else if (a.hist) {
    // entries of the tiles before: a thread adds up 4 experts over every (1024 / (E / 4))-th tile, eight loads at a time
    // (past the tiles before this one its last again, not counted; a loop of single loads waits for each)
    const int E4 = (int)sort_pitch(E) / 4, per = kSortThreads / E4, g = threadIdx.x / E4, e4 = threadIdx.x % E4;
    if (g < per) {
      const int4 *col = (const int4 *)a.hist + e4;
      const int mine = (int)blockIdx.x;
      int4 sum{0, 0, 0, 0};
      constexpr int U = 8;
      for (int b0 = g; b0 < mine; b0 += U * per) {
        int4 h[U];
#pragma unroll
        for (int u = 0; u < U; ++u) h[u] = col[(int64_t)min(b0 + u * per, mine - 1) * E4];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (b0 + u * per < mine) sum.x += h[u].x, sum.y += h[u].y, sum.z += h[u].z, sum.w += h[u].w;
      }
      const int32_t s4[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * e4 + i < E && s4[i]) atomicAdd(&before[4 * e4 + i], s4[i]);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) {
    int32_t at = before[e], c[kSortWaves];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) c[w] = sh[w * E + e];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      sh[w * E + e] = at;
      at += c[w];
    }
    if (blockIdx.x == gridDim.x - 1) a.counts[e] = at;
  }
  __syncthreads();
  const int bits = 32 - __clz(E);  // enough for 0 .. experts
#pragma unroll
  for (int s = 0; s < S; ++s) {
    if (s >= steps) break;  // uniform
    const int64_t i = w0 + s * 64 + lane;
    const bool in = i < n && i < i0 + tile;
    const int e = own[s];
    // lanes with the same expert as this one
    const uint32_t key = e < 0 ? (uint32_t)E : (uint32_t)e;
    uint64_t same = ~0ull;
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __ballot((key >> b) & 1);
      same &= (key >> b) & 1 ? m : ~m;
    }
    const int mine = __popcll(same & ((1ull << lane) - 1)), all = __popcll(same);
    int32_t base = 0;
    if (e >= 0) base = next[wave * E + e];
    // every lane has read before the last of each expert writes (LDS
    // operations of a wave complete in order)
    if (e >= 0 && mine == all - 1) next[wave * E + e] = base + all;
    if (in) {
      const int64_t r = (int64_t)base + mine;
      a.positions[i] = e >= 0 && r < a.capacity ? (int32_t)(e * a.capacity + r) : -1;
    }
  }
}

// ---- rows --------------------------------------------------------------------
constexpr int kThreads = 256;

// Slab rows of choices j0 .. j0 + J - 1 of a token, their positions requested together (one after the other they
// would cost a memory latency each).  -1: none, past topk, or outside the slabs, so no position can reach outside them.
constexpr int kAhead = 4;
template <int J>
__device__ __forceinline__ void slots_of(const MoveArgs &a, int64_t t, int j0, int64_t (&slot)[J]) {
  int32_t p[J];
#pragma unroll
  for (int j = 0; j < J; ++j) p[j] = a.positions[t * a.topk + min(j0 + j, a.topk - 1)];
#pragma unroll
  for (int j = 0; j < J; ++j) slot[j] = j0 + j < a.topk && p[j] >= 0 && p[j] < a.slots ? p[j] : -1;
}
template <int J>
__device__ __forceinline__ void weights_of(const MoveArgs &a, int64_t t, int j0, float (&w)[J]) {
#pragma unroll
  for (int j = 0; j < J; ++j) w[j] = a.weights ? a.weights[t * a.topk + min(j0 + j, a.topk - 1)] : 1.f;
}

// Thread tid's place: token t and its first chunk, TPR threads to a row, U chunks to a thread TPR apart.
template <int TPR, int U>
__device__ __forceinline__ void place(const MoveArgs &a, int64_t &t, int64_t &c) {
  const uint32_t g = blockIdx.x / (uint32_t)a.segs, seg = blockIdx.x - g * (uint32_t)a.segs;
  t = a.t0 + (int64_t)g * (kThreads / TPR) + threadIdx.x / TPR;
  c = (int64_t)seg * (TPR * U) + threadIdx.x % TPR;
}

// Rows are read and written non-temporally at every size, unlike the combine's (past_caches).  Timed with the grouped
// product that reads the slabs behind it, non-temporal against cached: 64 x 8 rows of 4096 bf16 (4 MB) 124.1 us
// against 128.0, 512 x 2 of 4096 int8 codes (4 MB) 34.1 against 34.7, 2048 x 2 of 4096 codes (17 MB) 59.2 against
// 59.4; 34 MB lose (2048 x 2 of 4096 bf16 95.8 against 94.3, 16384 x 2 of 512 bf16 48.0 against 45.6), 134 MB are equal.
template <int FMT, int TPR, int U>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(MoveArgs a) {
  constexpr int ES = fmt_bytes(FMT), N = 16 / ES;
  int64_t t, c0;
  place<TPR, U>(a, t, c0);
  if (t >= a.tokens) return;
  const char *x = (const char *)a.X + t * a.ldx * ES;
  const int64_t chunks = (a.hidden + N - 1) / N, whole = a.hidden / N;
  Raw16 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (c0 + u * TPR < whole) v[u] = load_once(x + (c0 + u * TPR) * 16);
  for (int j0 = 0; j0 < a.topk; j0 += kAhead) {
    int64_t slot[kAhead];
    slots_of(a, t, j0, slot);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (slot[j] < 0) continue;
      char *y = (char *)a.Y + slot[j] * a.ldy * ES;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t c = c0 + u * TPR;
        if (c < whole)
          store_once(y + c * 16, v[u]);
        else if (c < chunks)
          for (int64_t i = whole * N; i < a.hidden; ++i) put_bits<FMT>(y, i, elem_bits<FMT>(x, i));
      }
      if (a.scale && c0 == 0) a.slab_scale[slot[j]] = a.scale[t];
    }
  }
}

// J choices at a time: their rows are requested together, choices without one reading row 0 (the host launches no
// choices when there are no slabs), whose values are not used.
template <int FMT, int TPR, int U, bool ONCE, int J>
__global__ __launch_bounds__(kThreads) void combine_kernel(MoveArgs a) {
  constexpr int ES = fmt_bytes(FMT), N = 16 / ES;
  int64_t t, c0;
  place<TPR, U>(a, t, c0);
  if (t >= a.tokens) return;
  const int64_t chunks = (a.hidden + N - 1) / N, whole = a.hidden / N;
  char *y = (char *)a.Y + t * a.ldy * ES;
  float acc[U][N] = {};
  for (int j0 = 0; j0 < a.topk; j0 += J) {
    int64_t slot[J];
    float w[J];
    slots_of(a, t, j0, slot);
    weights_of(a, t, j0, w);
    Raw16 r[U][J];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (c0 + u * TPR < whole)
          r[u][j] = load_vec<ONCE>((const char *)a.X + (slot[j] < 0 ? 0 : slot[j]) * a.ldx * ES + (c0 + u * TPR) * 16);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + u * TPR;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (slot[j] < 0) continue;
        if (c < whole) {
          Vec<FMT> v;
          v.unpack(r[u][j]);
#pragma unroll
          for (int i = 0; i < N; ++i) acc[u][i] = fmaf(w[j], v.v[i], acc[u][i]);
        } else if (c < chunks) {
          const char *x = (const char *)a.X + slot[j] * a.ldx * ES;
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (whole * N + i < a.hidden)
              acc[u][i] = fmaf(w[j], elem_f32<FMT>(elem_bits<FMT>(x, whole * N + i)), acc[u][i]);
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t c = c0 + u * TPR;
    Vec<FMT> v;
#pragma unroll
    for (int i = 0; i < N; ++i) v.v[i] = acc[u][i];
    if (c < whole) {
      store_vec<ONCE>(y + c * 16, v.pack());
    } else if (c < chunks) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (whole * N + i < a.hidden) put_bits<FMT>(y, whole * N + i, f32_elem<FMT>(v.v[i]));
    }
  }
}

// One workgroup (TPR = 256) or wave (TPR = 64) per token; JB choices at a time, so dY is read ceil(topk / JB)
// times (from cache after the first).
template <int FMT, int TPR, int JB, bool ONCE>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(MoveArgs a) {
  constexpr int ES = fmt_bytes(FMT), N = 16 / ES;
  __shared__ float part[kThreads / 64][JB];
  const int lane = threadIdx.x % TPR;
  const int64_t t = a.t0 + (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
  if (t >= a.tokens) return;  // whole waves; with TPR = 256 no workgroup lies past the tokens
  const int64_t chunks = (a.hidden + N - 1) / N, whole = a.hidden / N;
  const char *dy = (const char *)a.X + t * a.ldx * ES;
  for (int j0 = 0; j0 < a.topk; j0 += JB) {
    int64_t slot[JB];
    float w[JB], dot[JB];
    slots_of(a, t, j0, slot);
    weights_of(a, t, j0, w);
#pragma unroll
    for (int j = 0; j < JB; ++j) dot[j] = 0.f;
    for (int64_t c = lane; c < chunks; c += TPR) {
      if (c < whole) {
        Vec<FMT> g;
        g.unpack(*(const Raw16 *)(dy + c * 16));
        Raw16 r[JB];  // (row 0 for a choice without one, not used: hidden is 0 when there are no slabs)
#pragma unroll
        for (int j = 0; j < JB; ++j)
          r[j] = load_vec<ONCE>((const char *)a.S + (slot[j] < 0 ? 0 : slot[j]) * a.lds * ES + c * 16);
#pragma unroll
        for (int j = 0; j < JB; ++j) {
          if (slot[j] < 0) continue;
          Vec<FMT> v, d;
          v.unpack(r[j]);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            dot[j] = fmaf(g.v[i], v.v[i], dot[j]);
            d.v[i] = w[j] * g.v[i];
          }
          store_vec<ONCE>((char *)a.Y + slot[j] * a.ldy * ES + c * 16, d.pack());
        }
      } else {
        for (int64_t i = whole * N; i < a.hidden; ++i) {
          const float g = elem_f32<FMT>(elem_bits<FMT>(dy, i));
#pragma unroll
          for (int j = 0; j < JB; ++j) {
            if (slot[j] < 0) continue;
            dot[j] = fmaf(g, elem_f32<FMT>(elem_bits<FMT>((const char *)a.S + slot[j] * a.lds * ES, i)), dot[j]);
            put_bits<FMT>((char *)a.Y + slot[j] * a.ldy * ES, i, f32_elem<FMT>(w[j] * g));
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < JB; ++j) dot[j] = wave_add(dot[j]);
    if constexpr (TPR > 64) {
      __syncthreads();  // the previous choices' sums are read
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int j = 0; j < JB; ++j) part[threadIdx.x >> 6][j] = dot[j];
      __syncthreads();
#pragma unroll
      for (int j = 0; j < JB; ++j) dot[j] = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
    }
    if (lane == 0)
#pragma unroll
      for (int j = 0; j < JB; ++j)
        if (j0 + j < a.topk) a.dweights[t * a.topk + j0 + j] = dot[j];
  }
}

// Tokens in launches whose work-items stay below 2^32.
template <class F>
hipError_t over_tokens(const MoveArgs &a, int rows_per_block, F &&launch) {
  const int64_t most = (0xffffffffLL / kThreads / a.segs) * rows_per_block;
  for (int64_t t0 = 0; t0 < a.tokens; t0 += most) {
    MoveArgs b = a;
    b.t0 = t0;
    const int64_t n = a.tokens - t0 < most ? a.tokens - t0 : most;
    launch(b, (unsigned)((n + rows_per_block - 1) / rows_per_block * a.segs));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

constexpr int kU = 2;  // chunks per thread

// Slab rows of more bytes than the caches keep from their producer are read and
// written non-temporally: 8192 x 2 rows of 4096 bf16 (134 MB) combine 35.3 us
// against 40.3, gradients 59.6 against 68.1; 16384 x 2 rows of 512 (34 MB) 12.7
// against 10.4.
template <int FMT>
bool past_caches(const MoveArgs &a) {
  return (double)a.tokens * a.topk * a.hidden * fmt_bytes(FMT) > 64e6;
}

template <int FMT, int TPR>
hipError_t rows_t(MoveArgs a, bool combine, hipStream_t stream) {
  const int64_t chunks = (a.hidden * fmt_bytes(FMT) + 15) / 16;
  a.segs = (int32_t)((chunks + TPR * kU - 1) / (TPR * kU));
  if (a.segs < 1) a.segs = 1;  // (rows of no elements may still have scales)
  return over_tokens(a, kThreads / TPR, [&](const MoveArgs &b, unsigned grid) {
    if constexpr (FMT != FMT_I8) {
      if (combine) {
        const bool once = past_caches<FMT>(b);
        if (b.topk <= 2 && once)
          hipLaunchKernelGGL((combine_kernel<FMT, TPR, kU, true, 2>), dim3(grid), dim3(kThreads), 0, stream, b);
        else if (b.topk <= 2)
          hipLaunchKernelGGL((combine_kernel<FMT, TPR, kU, false, 2>), dim3(grid), dim3(kThreads), 0, stream, b);
        else if (once)
          hipLaunchKernelGGL((combine_kernel<FMT, TPR, kU, true, 4>), dim3(grid), dim3(kThreads), 0, stream, b);
        else
          hipLaunchKernelGGL((combine_kernel<FMT, TPR, kU, false, 4>), dim3(grid), dim3(kThreads), 0, stream, b);
        return;
      }
    }
    hipLaunchKernelGGL((dispatch_kernel<FMT, TPR, kU>), dim3(grid), dim3(kThreads), 0, stream, b);
  });
}

template <int FMT>
hipError_t rows_fmt(const MoveArgs &a, bool combine, hipStream_t stream) {
  const int64_t chunks = (a.hidden * fmt_bytes(FMT) + 15) / 16;
  if (chunks <= 8 * kU) return rows_t<FMT, 8>(a, combine, stream);
  if (chunks <= 64 * kU) return rows_t<FMT, 64>(a, combine, stream);
  return rows_t<FMT, 256>(a, combine, stream);
}

hipError_t rows_any(const MoveArgs &a, bool combine, hipStream_t stream) {
  switch (a.fmt) {
    case FMT_F32:
      return rows_fmt<FMT_F32>(a, combine, stream);
    case FMT_F16:
      return rows_fmt<FMT_F16>(a, combine, stream);
    case FMT_BF16:
      return rows_fmt<FMT_BF16>(a, combine, stream);
    default:
      return rows_fmt<FMT_I8>(a, false, stream);
  }
}

template <int FMT, int TPR, int JB>
hipError_t backward_j(MoveArgs a, hipStream_t stream) {
  a.segs = 1;
  return over_tokens(a, kThreads / TPR, [&](const MoveArgs &b, unsigned grid) {
    if (past_caches<FMT>(b))
      hipLaunchKernelGGL((combine_backward_kernel<FMT, TPR, JB, true>), dim3(grid), dim3(kThreads), 0, stream, b);
    else
      hipLaunchKernelGGL((combine_backward_kernel<FMT, TPR, JB, false>), dim3(grid), dim3(kThreads), 0, stream, b);
  });
}

template <int FMT, int TPR>
hipError_t backward_t(const MoveArgs &a, hipStream_t stream) {
  return a.topk <= 2 ? backward_j<FMT, TPR, 2>(a, stream) : backward_j<FMT, TPR, 4>(a, stream);
}

template <int FMT>
hipError_t backward_fmt(const MoveArgs &a, hipStream_t stream) {
  const int64_t chunks = (a.hidden * fmt_bytes(FMT) + 15) / 16;
  // a wave per token for short rows (16384 x 2 rows of 64 chunks: 18.4 us against 48.0 on a workgroup each), a
  // workgroup for long ones (8192 x 2 rows of 512 chunks: 59.5 us against 82.4 on a wave)
  return chunks <= 128 ? backward_t<FMT, 64>(a, stream) : backward_t<FMT, 256>(a, stream);
}

}  // namespace

hipError_t launch_sort(const SortArgs &args, hipStream_t stream) {
  SortArgs a = args;
  // without a workspace (no more entries than one workgroup sorts, or no experts, when there is nothing to count and
  // any number of workgroups writes its -1s) the tiles are those of one workgroup
  const int64_t n = a.tokens * a.topk;
  const int64_t blocks = a.hist ? sort_blocks(n) : n ? (n + SortInfo::kOneBlock - 1) / SortInfo::kOneBlock : 1;
  const size_t lds = (size_t)(kSortWaves + 1) * a.experts * 4;
  if (a.hist) {
    if (a.id64)
      hipLaunchKernelGGL(sort_count_kernel<true>, dim3((unsigned)blocks), dim3(kSortThreads), (size_t)a.experts * 4, stream, a);
    else
      hipLaunchKernelGGL(sort_count_kernel<false>, dim3((unsigned)blocks), dim3(kSortThreads), (size_t)a.experts * 4, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // every tile adding up all tiles before it reads their square: a launch of its own from kScanBlocks tiles
    a.scanned = blocks > SortInfo::kScanBlocks;
    if (a.scanned) {
      hipLaunchKernelGGL(sort_scan_kernel, dim3((unsigned)a.experts), dim3(kSortThreads), 0, stream, a.hist,
                         sort_pitch(a.experts), (int)blocks);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  if (a.id64)
    hipLaunchKernelGGL(sort_place_kernel<true>, dim3((unsigned)blocks), dim3(kSortThreads), lds, stream, a);
  else
    hipLaunchKernelGGL(sort_place_kernel<false>, dim3((unsigned)blocks), dim3(kSortThreads), lds, stream, a);
  return hipGetLastError();
}

hipError_t launch_dispatch(const MoveArgs &a, hipStream_t stream) { return rows_any(a, false, stream); }
hipError_t launch_combine(const MoveArgs &a, hipStream_t stream) { return rows_any(a, true, stream); }

hipError_t launch_combine_backward(const MoveArgs &a, hipStream_t stream) {
  switch (a.fmt) {
    case FMT_F32:
      return backward_fmt<FMT_F32>(a, stream);
    case FMT_F16:
      return backward_fmt<FMT_F16>(a, stream);
    default:
      return backward_fmt<FMT_BF16>(a, stream);
  }
}

}  // namespace tsm
