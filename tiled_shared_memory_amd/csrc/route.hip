// The expert router: scores, choice and weights of a token's experts, and the
// gradient of its logits.
//
//   score   s_e = exp(x_e) / sum exp(x)   or   1 / (1 + exp(-x_e))
//   key     s_e + bias_e (chooses; without a bias the logits order as the scores do, exactly)
//   groups  the top_groups with the largest sum of their `best` largest keys
//   weight  factor * s_e, renormalised over the chosen: factor * s_e / sum of their s
//
// L lanes hold a token's row (16, or 32 above 256 experts), each the experts
// l V .. l V + V - 1; a wave works on 64 / L tokens.
//
// Up to 8 choices (route8_kernel): each lane sorts its keys, the lanes' lists of 8 are
// merged pairwise (element i against the partner's 7 - i, then three exchanges), and
// the k-th of the result is the smallest key that is chosen.  The lanes list the
// experts that reach it, and up to 8 lanes order those and weigh them: about as much
// work as two rounds of searching the largest key, which it replaces.  More choices,
// and groups that lanes cannot share out evenly (route_kernel): one after another, the
// largest key of each lane, of the L lanes, the first lane that holds it.
//
// A choice is made by the exact keys.  Keys computed in float32 are off by a
// known bound (score_error); where two neighbours in the order, or two groups, lie
// nearer than that, the token's wave decides again by keys in float64.  Which
// experts are chosen is therefore the same whatever exp() rounds to.
//
// Weights of renormalised scores are formed from exp(x - max) over the chosen
// ones, so they neither underflow nor overflow.
#include "elems.hpp"
#include "route_internal.hpp"

namespace tsm {
namespace {

constexpr int kThreads = 256;
constexpr float kInf = __builtin_inff();

// How far a float32 score may be from the exact one (scores are at most 1).  exp of an argument d is off by
// |d| 2^-23 + 2^-22 relative; |d| exp(-|d|) < 0.37, so by 2^-22 of 1 at most.  A sigmoid adds a sum (2^-24) and a
// reciprocal (2^-23): below 2^-20 together.  A softmax's sum of up to 32 numbers a lane and 5 steps over the lanes adds
// 37 * 2^-24, its reciprocal and product 2^-22: below 2^-18.
__device__ __forceinline__ float score_error(bool sigmoid) { return sigmoid ? 0x1p-20f : 0x1p-18f; }

// ---- lanes of a token ----
// The value of another lane: step 0 and 1 exchange within a quad, 2 and 3 mirror 8 and 16 lanes (which, after the
// steps before, hold equal values by quads and by eights), 4 exchanges the rows of 32.
template <int STEP>
__device__ __forceinline__ int across(int v) {
  if constexpr (STEP == 0) return __builtin_amdgcn_mov_dpp(v, 0xb1, 0xf, 0xf, true);
  if constexpr (STEP == 1) return __builtin_amdgcn_mov_dpp(v, 0x4e, 0xf, 0xf, true);
  if constexpr (STEP == 2) return __builtin_amdgcn_mov_dpp(v, 0x141, 0xf, 0xf, true);
  if constexpr (STEP == 3) return __builtin_amdgcn_mov_dpp(v, 0x140, 0xf, 0xf, true);
  return __shfl_xor(v, 16, 32);
}
template <int STEP>
__device__ __forceinline__ float across(float v) {
  return __builtin_bit_cast(float, across<STEP>(__builtin_bit_cast(int, v)));
}
template <int N>
constexpr int log2_of() {
  return N == 1 ? 0 : 1 + log2_of<N / 2>();
}

template <int N>
struct Step {
  static constexpr int value = N;
};
template <int N, int I = 0, class F>
__device__ __forceinline__ void steps(F &&f) {
  if constexpr (I < N) {
    f(Step<I>{});
    steps<N, I + 1>(f);
  }
}
template <int L>
__device__ __forceinline__ float row_max(float v) {
  steps<log2_of<L>()>([&](auto s) {
    const float o = across<s.value>(v);
    v = o > v ? o : v;
  });
  return v;
}
template <int L, class T>
__device__ __forceinline__ T row_sum(T v) {
  if constexpr (sizeof(T) == 4) {
    steps<log2_of<L>()>([&](auto s) { v += across<s.value>(v); });
  } else {
#pragma unroll
    for (int d = 1; d < L; d <<= 1) v += __shfl_xor(v, d, L);
  }
  return v;
}
template <int L>
__device__ __forceinline__ double row_max(double v) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) {
    const double o = __shfl_xor(v, d, L);
    v = o > v ? o : v;
  }
  return v;
}
// Which of a token's lanes say so.
template <int L>
__device__ __forceinline__ uint32_t row_ballot(bool b) {
  return (uint32_t)(__ballot(b) >> (threadIdx.x & (64 - L))) & (uint32_t)((1ull << L) - 1);
}

__device__ __forceinline__ float expo(float x) { return __expf(x); }
__device__ __forceinline__ double expo(double x) { return exp(x); }

// LDS of one wave is written and read by that wave alone, in order.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The kernel's arguments, read again: held in scalar registers from its start they would spill.
__device__ __forceinline__ RouteArgs args_again() {
  typedef const __attribute__((address_space(4))) RouteArgs *At;
  At p = (At)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const RouteArgs *)p;
}

template <int V>
struct Row {
  float x[V];  // logits, -inf past the last expert
  int e0;      // this lane's first expert
};

template <int FMT, int L, int V>
__device__ __forceinline__ void load_row(Row<V> &w, const RouteArgs &a, int64_t t) {
  const char *p = (const char *)a.logits + t * a.ld * fmt_bytes(FMT);
  constexpr int N = Vec<FMT>::N;
  if (V % N == 0 && a.experts == L * V) {
#pragma unroll
    for (int h = 0; h < V / N; ++h) {
      Vec<FMT> v;
      v.unpack(*(const Raw16 *)(p + (w.e0 + h * N) * fmt_bytes(FMT)));
#pragma unroll
      for (int i = 0; i < N; ++i) w.x[(h * N + i) % V] = v.v[i];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    w.x[i] = w.e0 + i < a.experts ? elem_f32<FMT>(elem_bits<FMT>(p, w.e0 + i)) : -kInf;
  }
}

// The largest logit and the sum of exp(x - largest) of a token's row.
template <class T, int L, int V>
__device__ __forceinline__ void soft_stats(const Row<V> &w, T &top, T &sum) {
  T m = w.x[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = (T)w.x[i] > m ? (T)w.x[i] : m;
  top = row_max<L>(m);
  if (top == -(T)kInf) top = 0;
  sum = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) sum += expo((T)w.x[i] - top);
  sum = row_sum<L>(sum);
}

__device__ __forceinline__ float one_over(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ double one_over(double x) { return 1.0 / x; }
// by: of a softmax, one over the sum.
template <class T>
__device__ __forceinline__ T score_of(bool sigmoid, T x, T top, T by) {
  return sigmoid ? one_over(T(1) + expo(-x)) : expo(x - top) * by;
}

// Chooses a token's experts into chosen[0 .. topk) (-1: none left) and their logits; returns whether float32 keys left
// it open.  bad: by the logits alone.
template <class T, int L, int V>
__device__ __forceinline__ bool choose(const RouteArgs &a, const Row<V> &w, const float (&bias)[V], bool bad, T *keys,
                                       int *chosen, float *logit) {
  const int l = threadIdx.x % L;
  constexpr bool APPROX = sizeof(T) == 4;
  const T none = -(T)kInf, error = score_error(a.sigmoid);
  const bool grouped = a.top_groups < a.groups && !bad;
  const bool scored = a.bias && !bad, sums = grouped && (a.bias || a.best > 1);
  bool open = false;
  T key[V], top = 0, sum = 1;
  if ((scored || sums) && !a.sigmoid) {
    soft_stats<T, L>(w, top, sum);
    sum = one_over(sum);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = w.x[i] == w.x[i] ? (T)w.x[i] : none;
    T of_group = key[i];
    if (scored || sums) {
      const T s = score_of<T>(a.sigmoid, w.x[i], top, sum) + (a.bias ? (T)bias[i] : T(0));
      of_group = w.x[i] > none && s == s ? s : none;
      if (scored) key[i] = of_group;
    }
    if (grouped) keys[w.e0 + i] = of_group;
  }
  if (grouped) {
    wave_sync();
    // lane l takes groups l, l + L, ...: their largest keys, from a start of its own (no two lanes on one bank)
    const int size = a.experts / a.groups;
    constexpr int P = RouteInfo::kMaxGroups / L;
    T of[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int g = l + p * L;
      of[p] = none;
      if (g >= a.groups) continue;
      T b1 = none, b2 = none;
      int at = g % size;
      for (int i = 0; i < size; ++i) {
        const T k = keys[g * size + at];
        at = at + 1 == size ? 0 : at + 1;
        b2 = k > b1 ? b1 : (k > b2 ? k : b2);
        b1 = k > b1 ? k : b1;
      }
      of[p] = a.best > 1 && b2 > none ? b1 + b2 : b1;
    }
    wave_sync();
#pragma unroll
    for (int p = 0; p < P; ++p)
      if (l + p * L < a.groups) keys[l + p * L] = of[p];
    wave_sync();
    uint64_t kept = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (p * L >= a.groups) continue;  // uniform
      const int g = l + p * L;
      int before = 0;
      for (int o = 0; o < a.groups; ++o) {
        const T k = keys[o];
        before += k > of[p] || (k == of[p] && o < g);
        if (APPROX && sums && g < a.groups && o != g) {
          const T d = k > of[p] ? k - of[p] : of[p] - k;
          open |= d <= 8 * error + T(0x1p-21) * (k > 0 ? k : -k);
        }
      }
      kept |= (uint64_t)row_ballot<L>(g < a.groups && before < a.top_groups && of[p] > none) << (p * L);
    }
    wave_sync();
    const uint32_t magic = (65536u + size - 1) / size;  // e / size for e < 512 (past the last expert any: no key)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!((kept >> (((uint32_t)(w.e0 + i) * magic >> 16) & 63)) & 1)) key[i] = none;
    }
  }
  T last = 0;
  const int rounds = a.topk + (APPROX && scored ? 1 : 0);
  for (int j = 0; j < rounds; ++j) {
    T m = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = key[i] > m ? key[i] : m;
    const T best = row_max<L>(m);
    if (APPROX && scored) {
      if (j > 0 && best > none) open |= last - best <= 4 * error + T(0x1p-22) * (best > 0 ? best : -best);
      last = best;
      if (j == a.topk) break;
    }
    bool mine = best > none && l == __builtin_ffs((int)row_ballot<L>(m == best)) - 1;
    if (best == none && l == 0) chosen[j] = -1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (mine && key[i] == best) {
        mine = false;
        key[i] = none;
        chosen[j] = w.e0 + i;
        logit[j] = w.x[i];
      }
    }
  }
  wave_sync();
  return row_ballot<L>(open) != 0;
}

// The weights of a token's choices, which lie in chosen and logit (in LDS): lane l's are l, l + L, ...  P of them.
template <int L, int V, int P>
__device__ __forceinline__ void weigh(const RouteArgs &a, const Row<V> &w, bool bad, bool held, int64_t t,
                                      const int *chosen, const float *logit) {
  const int l = threadIdx.x % L;
  float top = 0.f, sum = 1.f, x[P], s[P], part = 0.f;
  int e[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int j = l + p * L;
    e[p] = j < a.topk ? chosen[j] : -1;
    x[p] = e[p] >= 0 ? logit[j] : -kInf;
  }
  if (a.renormalize) {
    // the largest (softmax), or the largest below 0 (sigmoid): s = exp(min(x, 0)) / (1 + exp(-|x|))
    float m = x[0];
#pragma unroll
    for (int p = 1; p < P; ++p) m = fmaxf(m, x[p]);
    top = row_max<L>(m);
    if (a.sigmoid && top > 0.f) top = 0.f;
    if (top == -kInf) top = 0.f;
  } else if (!a.sigmoid) {
    soft_stats<float, L>(w, top, sum);
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    s[p] = 0.f;
    if (e[p] >= 0) {
      if (a.sigmoid)
        s[p] = expf((a.renormalize ? fminf(x[p], 0.f) - top : fminf(x[p], 0.f))) / (1.f + expf(-fabsf(x[p])));
      else
        s[p] = expf(x[p] - top);
      part += s[p];
    }
  }
  if (a.renormalize) sum = row_sum<L>(part);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int j = l + p * L;
    if (!held || j >= a.topk) continue;
    float wt = e[p] < 0 ? 0.f : s[p] / sum * a.factor;
    if (bad && e[p] >= 0) wt = __builtin_nanf("");
    a.ids[t * a.topk + j] = e[p];
    a.weights[t * a.topk + j] = wt;
  }
}

// ---- up to 8 choices ----
// Floats in the order of their values as whole numbers (-0 as 0), and back.
__device__ __forceinline__ int ordered(float f) {
  const int b = __builtin_bit_cast(int, f + 0.f);
  return b ^ (b >> 31 & 0x7fffffff);
}
__device__ __forceinline__ float of_ordered(int i) { return __builtin_bit_cast(float, i ^ (i >> 31 & 0x7fffffff)); }
constexpr int kNone = -0x7f800001;  // -inf

__device__ __forceinline__ void exchange(int &a, int &b) {  // the larger to a
  const int m = a > b ? a : b;
  b = a > b ? b : a;
  a = m;
}
// A list that rises and then falls (or the reverse), to falling.
__device__ __forceinline__ void merge8(int (&v)[8]) {
#pragma unroll
  for (int d = 4; d >= 1; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & d)) exchange(v[i], v[i + d]);
}
// 8 numbers to falling order: Batcher's odd-even merge sort, 19 exchanges.
__device__ __forceinline__ void sort8(int (&v)[8]) {
#pragma unroll
  for (int p = 1; p < 8; p <<= 1)
#pragma unroll
    for (int k = p; k >= 1; k >>= 1)
#pragma unroll
      for (int j = k % p; j + k < 8; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (j + i + k < 8 && (j + i) / (2 * p) == (j + i + k) / (2 * p)) exchange(v[j + i], v[j + i + k]);
}
// The larger 8 of two falling lists of 8, as a list for merge8.
__device__ __forceinline__ void join8(int (&a)[8], const int (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = b[7 - i] > a[i] ? b[7 - i] : a[i];
}

template <int FMT, int L, int V>
__global__ __launch_bounds__(kThreads) void route8_kernel(RouteArgs a) {
  constexpr int kTokens = kThreads / L;
  extern __shared__ double dynamic[];  // of the groups' keys: L * V float64 per token
  struct Choice {
    float key, x, bias;
    int e;
  };
  __shared__ Choice list[kTokens][8];
  __shared__ int chosen[kTokens][8];
  __shared__ float logit[kTokens][8];
  const int slot = threadIdx.x / L, l = threadIdx.x % L;
  const int64_t t = a.t0 + (int64_t)blockIdx.x * kTokens + slot;
  const bool held = t < a.tokens;
  const int64_t row = held ? t : a.tokens - 1;
  const bool grouped = a.top_groups < a.groups, scored = a.bias != nullptr;  // uniform
  const bool sums = grouped && (scored || a.best > 1);
  Row<V> w;
  w.e0 = l * V;
  load_row<FMT, L>(w, a, row);
  float bias[V] = {};
  if (scored) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (w.e0 + i < a.experts) bias[i] = a.bias[w.e0 + i];
  }
  // a NaN is above +inf or below -inf in this order
  int key[V], hi, lo;
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = ordered(w.x[i]);
  hi = lo = key[0];
#pragma unroll
  for (int i = 1; i < V; ++i) hi = key[i] > hi ? key[i] : hi, lo = key[i] < lo ? key[i] : lo;
  const bool bad = row_ballot<L>(hi > (a.sigmoid ? 0x7f800000 : 0x7f7fffff) || lo < kNone) != 0;
  bool open = bad;
  const float error = score_error(a.sigmoid);
  float top = 0.f, by = 1.f;
  if (scored || sums) {
    if (!a.sigmoid) {
      soft_stats<float, L>(w, top, by);
      by = one_over(by);
    }
    float g[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float s = score_of<float>(a.sigmoid, w.x[i], top, by) + bias[i];
      g[i] = w.x[i] > -kInf && s == s ? s : -kInf;
      if (scored) key[i] = ordered(g[i]);
    }
    if (sums) {
      // the two largest of the lane's, then of its group's lanes
      float b1 = g[0], b2 = -kInf;
#pragma unroll
      for (int i = 1; i < V; ++i) {
        b2 = __builtin_amdgcn_fmed3f(b1, b2, g[i]);
        b1 = g[i] > b1 ? g[i] : b1;
      }
      const int lanes = a.experts / a.groups / V;  // of a group: a power of two
      steps<log2_of<L>()>([&](auto s) {
        if ((1 << s.value) < lanes) {
          const float o1 = across<s.value>(b1), o2 = across<s.value>(b2);
          const float least = o1 < b1 ? o1 : b1, rest = o2 > b2 ? o2 : b2;
          b1 = o1 > b1 ? o1 : b1;
          b2 = least > rest ? least : rest;
        }
      });
      if (a.best > 1 && b2 > -kInf) b1 += b2;
      int before = 0;
      for (int r = lanes; r < L; r += lanes) {  // the group r lanes before, around the row
        const float o = __shfl(b1, (l - r) & (L - 1), L);
        before += o > b1 || (o == b1 && l >= r);
        open |= fabsf(o - b1) <= 8 * error + 0x1p-21f * fabsf(o);
      }
      const bool in = before < a.top_groups;
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = in ? key[i] : kNone;
    }
  }
  if (grouped && !sums) {
    int b1 = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) b1 = key[i] > b1 ? key[i] : b1;
    const int lanes = a.experts / a.groups / V;
    steps<log2_of<L>()>([&](auto s) {
      if ((1 << s.value) < lanes) {
        const int o = across<s.value>(b1);
        b1 = o > b1 ? o : b1;
      }
    });
    int before = 0;
    for (int r = lanes; r < L; r += lanes) {
      const int o = __shfl(b1, (l - r) & (L - 1), L);
      before += o > b1 || (o == b1 && l >= r);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = before < a.top_groups ? key[i] : kNone;
  }

  // the 8 largest keys of the token, in every lane
  int best[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) best[i] = i < V ? key[i % V] : kNone;
  if constexpr (V > 1) sort8(best);
  if constexpr (V > 8) {
    int more[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) more[i] = key[(8 + i) % V];
    sort8(more);
    join8(best, more);
    merge8(best);
  }
  steps<log2_of<L>()>([&](auto s) {
    int other[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) other[i] = across<s.value>(best[i]);
    join8(best, other);
    merge8(best);
  });
  int least = best[0];  // the smallest chosen key
#pragma unroll
  for (int i = 1; i < 8; ++i)
    if (i < a.topk) least = best[i];
  const bool all = least <= kNone;  // fewer than topk are left
  if (all) least = kNone + 1;

  // who reaches it
  uint32_t mine = 0;
#pragma unroll
  for (int i = V - 1; i >= 0; --i) mine = mine + mine + (key[i] >= least);
  int count = __builtin_popcount(mine), upto = count, total;
  steps<log2_of<L>()>([&](auto s) {
    const int o = __shfl_up(upto, 1 << s.value, L);
    if (l >= (1 << s.value)) upto += o;
  });
  total = __shfl(upto, L - 1, L);
  const bool tied = total > a.topk;  // equal keys at the border: the lowest indices
  if (__ballot(tied)) {
    uint32_t equal = 0;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) equal = equal + equal + (key[i] == least);
    int before = __builtin_popcount(equal);
    const int own = before;
    steps<log2_of<L>()>([&](auto s) {
      const int o = __shfl_up(before, 1 << s.value, L);
      if (l >= (1 << s.value)) before += o;
    });
    const int excess = total - a.topk, sum = __shfl(before, L - 1, L);
    // of the token's `sum` equal ones the first sum - excess stay
    int drop = before - (sum - excess);
    drop = drop < 0 ? 0 : drop > own ? own : drop;
    for (; drop > 0; --drop) {
      const uint32_t last = 0x80000000u >> __builtin_clz(equal);
      equal ^= last;
      mine ^= last;
      --count;
    }
    upto = count;
    steps<log2_of<L>()>([&](auto s) {
      const int o = __shfl_up(upto, 1 << s.value, L);
      if (l >= (1 << s.value)) upto += o;
    });
  }
  const uint32_t taken = mine;
  for (int at = upto - count; mine; mine &= mine - 1) list[slot][at++].e = w.e0 + __builtin_ctz(mine);
  wave_sync();
  const int n = total < a.topk ? total : a.topk;

  // lane j orders the j-th of the list
  Choice c{-kInf, 0.f, 0.f, -1};
  if (l < n) {
    c.e = list[slot][l].e;
    c.x = elem_f32<FMT>(elem_bits<FMT>((const char *)a.logits + row * a.ld * fmt_bytes(FMT), c.e));
    c.key = c.x;
    if (scored) {
      c.bias = a.bias[c.e];
      c.key = score_of<float>(a.sigmoid, c.x, top, by) + c.bias;
    }
    list[slot][l] = c;
  }
  if (l < 8) chosen[slot][l] = -1;
  wave_sync();
  int rank = 0;
  bool close = false;
  const float tolerance = 4 * error + 0x1p-22f * fabsf(c.key);
  for (int j = 0; j < a.topk; ++j) {
    const Choice o = list[slot][j];
    const bool other = j < n && j != l;
    rank += other && (o.key > c.key || (o.key == c.key && o.e < c.e));
    // (equal logits and biases make equal keys, whatever they round to)
    close |= other && fabsf(o.key - c.key) <= tolerance && (o.x != c.x || o.bias != c.bias);
  }
  if (l < n) {
    chosen[slot][rank] = c.e;
    logit[slot][rank] = c.x;
    if (scored) open |= close;
  }
  if (scored) {
    // those that are not chosen but as near to the last chosen one as keys may be off
    const float f = of_ordered(least);
    const int near = all ? least : ordered(f - (4 * error + 0x1p-22f * fabsf(f)));
    int around = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) around += key[i] >= near;
    if (__ballot(row_sum<L>(around) > n)) {
      // (the last chosen one's logit and bias)
      float lx = 0.f, lb = 0.f;
      for (int j = 0; j < n; ++j)
        if (ordered(list[slot][j].key) == least) lx = list[slot][j].x, lb = list[slot][j].bias;
#pragma unroll
      for (int i = 0; i < V; ++i)
        open |= key[i] >= near && !(taken >> i & 1) && (w.x[i] != lx || bias[i] != lb);
    }
  }
  wave_sync();
  if (__ballot(open)) {  // the whole wave, so that its lanes stay together; what was decided is decided again, equally
    double *const keys = dynamic + slot * (grouped ? L * V : 0);
    choose<double, L>(a, w, bias, bad, keys, chosen[slot], logit[slot]);
  }
  weigh<L, V, 1>(a, w, bad, held, t, chosen[slot], logit[slot]);
}

// Whether lanes of V experts share out the groups evenly, a power of two lanes each.
inline bool even_groups(const RouteArgs &a, int V) {
  if (a.top_groups == a.groups) return true;
  const int size = a.experts / a.groups, lanes = size / V;
  return size % V == 0 && (lanes & (lanes - 1)) == 0;
}

template <int FMT, int L, int V>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs first) {
  RouteArgs a = first;
  constexpr int kTokens = kThreads / L;
  extern __shared__ double dynamic[];  // of the groups' keys: L * V float64 per token
  __shared__ int chosen[kTokens][RouteInfo::kMaxTopk];
  __shared__ float logit[kTokens][RouteInfo::kMaxTopk];
  const int slot = threadIdx.x / L, l = threadIdx.x % L;
  const int64_t t = a.t0 + (int64_t)blockIdx.x * kTokens + slot;
  const bool held = t < a.tokens;
  Row<V> w;
  w.e0 = l * V;
  load_row<FMT, L>(w, a, held ? t : a.tokens - 1);
  float bias[V] = {};
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (w.e0 + i < a.experts) bias[i] = a.bias[w.e0 + i];
  }
  bool nan = false, inf = false;
#pragma unroll
  for (int i = 0; i < V; ++i) nan |= w.x[i] != w.x[i], inf |= w.x[i] == kInf;
  const bool bad = row_ballot<L>(nan || (inf && !a.sigmoid)) != 0;
  double *const keys = dynamic + slot * (a.top_groups < a.groups ? L * V : 0);
  const bool open = choose<float, L>(a, w, bias, bad, (float *)keys, chosen[slot], logit[slot]);
  // (the whole wave, so that its lanes stay together; what was decided is decided again, equally)
  a = args_again();
  if (__ballot(open)) choose<double, L>(a, w, bias, bad, keys, chosen[slot], logit[slot]);

  a = args_again();
  weigh<L, V, RouteInfo::kMaxTopk / L>(a, w, bad, held, t, chosen[slot], logit[slot]);
}

// With g the gradients of the weights times the factor, q the chosen scores over their sum:
//   renormalised  dx_e = q (g - sum g q)       (sigmoid: times 1 - s_e), 0 where not chosen
//   softmax       dx_e = s_e (g_e - sum g s)
//   sigmoid       dx_e = s_e (1 - s_e) g_e
template <int FMT, int L, int V>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(RouteArgs a) {
  constexpr int kLanes = L, kTokens = kThreads / L;
  __shared__ int chosen[kTokens][RouteInfo::kMaxTopk];
  __shared__ float grad[kTokens][RouteInfo::kMaxTopk];
  constexpr int ES = fmt_bytes(FMT), P = RouteInfo::kMaxTopk / kLanes;
  const int slot = threadIdx.x / kLanes, l = threadIdx.x % kLanes;
  const int64_t t = a.t0 + (int64_t)blockIdx.x * kTokens + slot;
  const bool held = t < a.tokens;
  const int64_t row = held ? t : a.tokens - 1;
  const char *p = (const char *)a.logits + row * a.ld * ES;
  Row<V> w;
  w.e0 = l * V;
  float x[P], g[P], top = 0.f, sum = 1.f;
  int e[P];
#pragma unroll
  for (int q = 0; q < P; ++q) {
    const int j = l + q * kLanes;
    e[q] = j < a.topk ? a.ids[row * a.topk + j] : -1;
    if (e[q] >= a.experts) e[q] = -1;
    g[q] = 0.f;
    x[q] = -kInf;
    if (e[q] >= 0) {
      g[q] = a.weights[row * a.topk + j] * a.factor;
      x[q] = elem_f32<FMT>(elem_bits<FMT>(p, e[q]));
    }
  }
  const bool whole = !a.sigmoid && !a.renormalize;  // the probabilities of every expert
  if (whole) {
    load_row<FMT, L>(w, a, row);
    soft_stats<float, L>(w, top, sum);
  } else if (a.renormalize) {
    float m = -kInf;
#pragma unroll
    for (int q = 0; q < P; ++q) m = fmaxf(m, x[q]);
    top = row_max<L>(m);
    if (a.sigmoid && top > 0.f) top = 0.f;
    if (top == -kInf) top = 0.f;
  }
  // s: scores, of renormalised weights q; left: 1 - s of a sigmoid
  float s[P], left[P], part = 0.f;
#pragma unroll
  for (int q = 0; q < P; ++q) {
    s[q] = 0.f;
    left[q] = 1.f;
    if (e[q] < 0) continue;
    if (a.sigmoid) {
      const float d = 1.f + expf(-fabsf(x[q]));
      s[q] = expf(a.renormalize ? fminf(x[q], 0.f) - top : fminf(x[q], 0.f)) / d;
      left[q] = expf(fminf(-x[q], 0.f)) / d;
    } else {
      s[q] = expf(x[q] - top);
    }
    part += s[q];
  }
  if (a.renormalize) sum = row_sum<L>(part);
  if (sum == 0.f) sum = 1.f;  // no expert, or only ones of logit -inf
  float dot = 0.f;
#pragma unroll
  for (int q = 0; q < P; ++q) {
    if (e[q] < 0) continue;
    s[q] /= sum;
    dot += g[q] * s[q];
  }
  dot = a.renormalize || whole ? row_sum<L>(dot) : 0.f;
#pragma unroll
  for (int q = 0; q < P; ++q) {
    const int j = l + q * kLanes;
    if (j >= a.topk) continue;
    chosen[slot][j] = e[q];
    grad[slot][j] = whole ? g[q] : s[q] * left[q] * (g[q] - dot);
  }
  wave_sync();
  float d[V] = {};
  for (int j = 0; j < a.topk; ++j) {
    const int at = chosen[slot][j] - w.e0;
    const float v = grad[slot][j];
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] += at == i ? v : 0.f;
  }
  if (whole) {
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = expf(w.x[i] - top) / sum * (d[i] - dot);
  }
  if (!held) return;
  char *out = (char *)a.dlogits + t * a.ldd * ES;
  constexpr int N = Vec<FMT>::N;
  if (V % N == 0 && a.experts == kLanes * V) {
#pragma unroll
    for (int h = 0; h < V / N; ++h) {
      Vec<FMT> v;
#pragma unroll
      for (int i = 0; i < N; ++i) v.v[i] = d[(h * N + i) % V];
      *(Raw16 *)(out + (w.e0 + h * N) * ES) = v.pack();
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (w.e0 + i < a.experts) put_bits<FMT>(out, w.e0 + i, f32_elem<FMT>(d[i]));
}

// Launches of 2^24 workgroups at most (work-items below 2^32).
template <int FMT, int L, int V>
hipError_t route_v(const RouteArgs &base, bool backward, hipStream_t stream) {
  constexpr int kTokens = kThreads / L;
  const int64_t most = ((int64_t)1 << 23) * kTokens;
  for (int64_t t0 = 0; t0 < base.tokens; t0 += most) {
    RouteArgs a = base;
    a.t0 = t0;
    const int64_t n = base.tokens - t0 < most ? base.tokens - t0 : most;
    const dim3 grid((unsigned)((n + kTokens - 1) / kTokens));
    const size_t lds = a.top_groups < a.groups ? (size_t)kTokens * L * V * 8 : 0;
    if (backward)
      hipLaunchKernelGGL((route_backward_kernel<FMT, L, V>), grid, dim3(kThreads), 0, stream, a);
    else if (a.topk <= 8 && even_groups(a, V))
      hipLaunchKernelGGL((route8_kernel<FMT, L, V>), grid, dim3(kThreads), lds, stream, a);
    else
      hipLaunchKernelGGL((route_kernel<FMT, L, V>), grid, dim3(kThreads), lds, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int FMT>
hipError_t route_fmt(const RouteArgs &a, bool backward, hipStream_t stream) {
  if (a.experts <= 16) return route_v<FMT, 16, 1>(a, backward, stream);
  if (a.experts <= 64) return route_v<FMT, 16, 4>(a, backward, stream);
  if (a.experts <= 128) return route_v<FMT, 16, 8>(a, backward, stream);
  if (a.experts <= 256) return route_v<FMT, 16, 16>(a, backward, stream);
  return route_v<FMT, 32, 16>(a, backward, stream);
}

hipError_t route_any(const RouteArgs &a, bool backward, hipStream_t stream) {
  switch (a.fmt) {
    case FMT_F32:
      return route_fmt<FMT_F32>(a, backward, stream);
    case FMT_F16:
      return route_fmt<FMT_F16>(a, backward, stream);
    default:
      return route_fmt<FMT_BF16>(a, backward, stream);
  }
}

}  // namespace

hipError_t launch_route(const RouteArgs &a, hipStream_t stream) { return route_any(a, false, stream); }
hipError_t launch_route_backward(const RouteArgs &a, hipStream_t stream) { return route_any(a, true, stream); }

}  // namespace tsm
