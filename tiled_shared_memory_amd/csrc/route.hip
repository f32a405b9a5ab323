// The expert router: scores, choice and weights of a token's experts, and the
// gradient of its logits.
//
//   score   s_e = exp(x_e) / sum exp(x)   or   1 / (1 + exp(-x_e))
//   key     s_e + bias_e (chooses; without a bias the logits order as the scores do, exactly)
//   groups  the top_groups with the largest sum of their `best` largest keys
//   weight  factor * s_e, renormalised over the chosen: factor * s_e / sum of their s
//
// L lanes hold a token's row, each up to V experts that follow each other; a wave works
// on 64 / L tokens.
//
// Up to 8 choices (route8_kernel): each lane sorts its keys, the lanes' lists of 8 are
// merged pairwise (element i against the partner's 7 - i, then three exchanges), and
// the k-th of the result is the smallest key that is chosen.  The lanes list the
// experts that reach it, and up to 8 lanes order those and weigh them: about as much
// work as two rounds of searching the largest key, which it replaces.
// More choices, and groups for which the lanes are too few (route_kernel): one after
// another, the largest key of each lane, of the L lanes, the first lane that
// holds it.
//
// A choice is made by the exact keys.  Keys computed in float32 are off by a
// known bound (score_error; route_keys.hpp has what follows from it); where two
// neighbours in the order, or a group that is kept and one that is not, lie nearer
// than that, the token is decided again by a whole wave in float64.  Which experts
// are chosen is therefore the same whatever exp() rounds to.  (That takes five times
// as long, so what decides nothing, such as a group without an expert to choose, must
// not read as near: 65536 x 60 in 12 groups 41 us, 116 with the four groups that fill
// up its lanes taken for near ones.)
//
// Weights of renormalised scores are formed from exp(x - max) over the chosen
// ones, so they neither underflow nor overflow.
//
// What bounds it is the arithmetic: 65536 x 256 float32 with sigmoid scores, a bias and
// 4 of 8 groups takes 35-41 us, 1140 vector instructions per wave (four tokens), which
// keep the SIMDs busy for 70% of its cycles; 20 us of it are the bias and the groups
// (scores of every expert, near ties).  The logits alone would take 14 us from memory.
// More than 8 choices cost a search of the whole row each: 16 of 65536 x 256 in 4 of 8
// groups 124 us, 33 without groups 145, 16 of 65536 x 512 132 and in 16 groups 207.
// The gradient of the same, 18.5 us, moves its 113 MB at 6.1 TB/s.
#include "elems.hpp"
#include "route_internal.hpp"
#include "route_keys.hpp"

namespace tsm {
namespace {

constexpr int kThreads = 256;
constexpr float kInf = __builtin_inff();

// How far a float32 score may be from the exact one.  exp of d is off by |d| 1.5 * 2^-24 (the product with log2 e) and
// 2^-23, relative; of a difference d by another |d| 2^-24.
//  * A sigmoid s = 1 / (1 + exp(-x)) takes s (1 - s) of that, at most 0.224 / |x| and 1/4 of it, and adds a sum (2^-24)
//    and a reciprocal (2^-23): below 2^-21.
//  * A softmax's score takes it whole, relative to itself, and |d| exp(-|d|) < 0.37; the sum's error is that of its
//    terms in the mean (|d| is at most ln 512 in that mean, plus the logarithm of the largest score's share) and of 21
//    additions, 16 in a lane and 5 over the lanes; with reciprocal and product below 2^-18 of the largest score.
__device__ __forceinline__ float score_error(bool sigmoid, float largest) {
  return sigmoid ? 0x1p-21f : 0x1p-18f * largest;
}

// ---- lanes of a token ----
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
constexpr int log2_of(int n) { return n == 1 ? 0 : 1 + log2_of(n / 2); }

// The value of another lane: step 0 and 1 exchange within a quad, 2 and 3 mirror 8 and 16 lanes (which, after the
// steps before, hold equal values by quads and by eights), 4 and 5 exchange rows of 16 and halves.
template <int STEP>
__device__ __forceinline__ int across(int v) {
  if constexpr (STEP == 0) return __builtin_amdgcn_mov_dpp(v, 0xb1, 0xf, 0xf, true);
  if constexpr (STEP == 1) return __builtin_amdgcn_mov_dpp(v, 0x4e, 0xf, 0xf, true);
  if constexpr (STEP == 2) return __builtin_amdgcn_mov_dpp(v, 0x141, 0xf, 0xf, true);
  if constexpr (STEP == 3) return __builtin_amdgcn_mov_dpp(v, 0x140, 0xf, 0xf, true);
  return __shfl_xor(v, 1 << STEP, 64);
}
template <int STEP>
__device__ __forceinline__ float across(float v) {
  return __builtin_bit_cast(float, across<STEP>(__builtin_bit_cast(int, v)));
}
template <int STEP>
__device__ __forceinline__ double across(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)across<STEP>((int)(uint32_t)b), hi = (uint32_t)across<STEP>((int)(uint32_t)(b >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// f(the value r lanes before, around the token's lanes, and r) for the multiples of `apart` (a power of two) below L.
template <int L, class T, class F>
__device__ __forceinline__ void around_row(T v, int apart, F &&f) {
  if constexpr (L == 16) {
    steps<15>([&](auto s) {
      constexpr int R = s.value + 1;
      if ((R & (apart - 1)) == 0)  // uniform
        f(__builtin_bit_cast(T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x120 + R, 0xf, 0xf, true)), R);
    });
  } else {
    for (int r = apart; r < L; r += apart) f(__shfl(v, ((threadIdx.x & (L - 1)) - r) & (L - 1), L), r);
  }
}
template <int L, class T>
__device__ __forceinline__ T row_max(T v) {
  steps<log2_of(L)>([&](auto s) {
    const T o = across<s.value>(v);
    v = o > v ? o : v;
  });
  return v;
}
template <int L, class T>
__device__ __forceinline__ T row_sum(T v) {
  steps<log2_of(L)>([&](auto s) { v += across<s.value>(v); });
  return v;
}
// Inclusive sums over a token's lanes.
template <int L>
__device__ __forceinline__ int row_scan(int v) {
  const int l = threadIdx.x % L;
  steps<log2_of(L)>([&](auto s) {
    const int o = __shfl_up(v, 1 << s.value, L);
    if (l >= (1 << s.value)) v += o;
  });
  return v;
}
// Which of a token's lanes say so.
template <int L>
__device__ __forceinline__ uint64_t row_ballot(bool b) {
  const uint64_t all = __ballot(b);
  if constexpr (L == 64) return all;
  return (all >> (threadIdx.x & (64 - L))) & ((1ull << (L & 63)) - 1);
}

__device__ __forceinline__ float one_over(float x) { return __builtin_amdgcn_rcpf(x); }

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

// A lane's logits of a token's row, from expert e0: n of its V, -inf behind them.
template <int FMT, int L, int V>
__device__ __forceinline__ void load_row(float (&x)[V], const RouteArgs &a, int64_t t, int e0, int n) {
  const char *p = (const char *)a.logits + t * a.ld * fmt_bytes(FMT);
  constexpr int N = Vec<FMT>::N;
  if (V % N == 0 && a.experts == L * V) {  // uniform: n = V (gfx950 takes vectors at any alignment of the element)
#pragma unroll
    for (int h = 0; h < V / N; ++h) {
      Vec<FMT> v;
      v.unpack(*(const Raw16 *)(p + (e0 + h * N) * fmt_bytes(FMT)));
#pragma unroll
      for (int i = 0; i < N; ++i) x[(h * N + i) % V] = v.v[i];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = i < n ? elem_f32<FMT>(elem_bits<FMT>(p, e0 + i)) : -kInf;
}

// The largest logit and the sum of exp(x - largest) of a token's row.
template <int L, int V>
__device__ __forceinline__ void soft_stats(const float (&x)[V], float &top, float &sum) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = x[i] > m ? x[i] : m;
  top = row_max<L>(m);
  if (top == -kInf) top = 0.f;
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) sum += __expf(x[i] - top);
  sum = row_sum<L>(sum);
}

// by: of a softmax, one over the sum.
__device__ __forceinline__ float score_of(bool sigmoid, float x, float top, float by) {
  return sigmoid ? one_over(1.f + __expf(-x)) : __expf(x - top) * by;
}

// Which groups of experts a token may choose from (a bit each), from the keys of its experts in LDS, whose place is
// used for the groups' sums then; open: whether that hangs on less than float32 holds (error: of a key).
template <int L, class T>
__device__ __forceinline__ uint64_t best_groups(const RouteArgs &a, T *keys, T error, bool *open) {
  const int l = threadIdx.x % L, size = a.experts / a.groups;
  const T none = -(T)kInf;
  constexpr int P = (RouteInfo::kMaxGroups + L - 1) / L;
  T of[P];
  float tolerance[P];
  wave_sync();
  // lane l takes groups l, l + L, ...: their largest keys, from a start of its own (no two lanes on one bank)
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int g = l + p * L;
    of[p] = none;
    tolerance[p] = 0.f;
    if (g >= a.groups) continue;
    T b1 = none, b2 = none;
    int at = g % size;
#pragma unroll 4
    for (int i = 0; i < size; ++i) {
      const T k = keys[g * size + at];
      at = at + 1 == size ? 0 : at + 1;
      b2 = k > b1 ? b1 : (k > b2 ? k : b2);
      b1 = k > b1 ? k : b1;
    }
    if (a.best == 1 || !(b2 > none)) b2 = 0;
    of[p] = group_sum(b1, b2);
    tolerance[p] = group_tolerance((float)error, (float)b1, (float)b2);
  }
  wave_sync();
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (l + p * L < a.groups) keys[l + p * L] = of[p];
  wave_sync();
  uint64_t kept = 0;
  bool close = false;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (p * L >= a.groups) continue;  // uniform
    const int g = l + p * L;
    int before = 0;
    for (int o = 0; o < a.groups; ++o) {
      const T k = keys[o];
      before += k > of[p] || (k == of[p] && o < g);
      if (error > 0) close |= g < a.groups && o != g && near_sums((float)k, (float)of[p], tolerance[p]);
    }
    kept |= row_ballot<L>(g < a.groups && before < a.top_groups && of[p] > none) << (p * L % 64);
  }
  if (error > 0 && __ballot(close)) {  // it matters between one that is kept and one that is not
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int g = l + p * L;
      if (g >= a.groups) continue;
      for (int o = 0; o < a.groups; ++o)
        *open |= ((kept >> o ^ kept >> g) & 1) && near_sums((float)keys[o], (float)of[p], tolerance[p]);
    }
  }
  wave_sync();
  return kept;
}

// Chooses a token's experts into chosen[0 .. topk) (-1: none left) and their logits, by float32 keys; returns whether
// those left it open.
template <int L, int V>
__device__ __forceinline__ bool choose(const RouteArgs &a, const float (&x)[V], int e0, const float (&bias)[V],
                                       float *keys, int *chosen, float *logit) {
  const int l = threadIdx.x % L;
  const bool grouped = a.top_groups < a.groups, scored = a.bias != nullptr;
  const bool sums = grouped && (scored || a.best > 1);
  bool open = false;
  float key[V], top = 0.f, by = 1.f;
  if ((scored || sums) && !a.sigmoid) {
    soft_stats<L>(x, top, by);
    by = one_over(by);
  }
  const float error = score_error(a.sigmoid, by);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = x[i];
    float of_group = key[i];
    if (scored || sums) {
      const float s = score_of(a.sigmoid, x[i], top, by) + bias[i];
      of_group = x[i] > -kInf ? s : -kInf;
      if (scored) key[i] = of_group;
    }
    if (grouped) keys[e0 + i] = of_group;
  }
  if (grouped) {
    const uint64_t kept = best_groups<L>(a, keys, sums ? error : 0.f, &open);
    const uint32_t magic = group_magic(a.experts / a.groups);
#pragma unroll
    for (int i = 0; i < V; ++i)  // (past the last expert any: no key)
      if (!((kept >> (group_of(e0 + i, magic) & 63)) & 1)) key[i] = -kInf;
  }
  float last = 0.f;
  const int rounds = a.topk + (scored ? 1 : 0);
  for (int j = 0; j < rounds; ++j) {
    float m = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = key[i] > m ? key[i] : m;
    const float best = row_max<L>(m);
    if (scored) {
      if (j > 0 && best > -kInf) open |= last - best <= key_error(error, best);
      last = best;
      if (j == a.topk) break;
    }
    bool mine = best > -kInf && l == __builtin_ffsll((long long)row_ballot<L>(m == best)) - 1;
    if (best == -kInf && l == 0) chosen[j] = -1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (mine && key[i] == best) {
        mine = false;
        key[i] = -kInf;
        chosen[j] = e0 + i;
        logit[j] = x[i];
      }
    }
  }
  wave_sync();
  return row_ballot<L>(open) != 0;
}

// The same by keys in float64, by a whole wave, a lane every 64th expert; bad: by the logits alone.  (In loops of one
// score each, and keys in LDS: this is rare, and must not cost the usual way its registers.)
template <int FMT>
__device__ __forceinline__ void choose_exactly(const RouteArgs &a, const char *row, bool bad, double *keys, int *chosen,
                                               float *logit) {
  const int lane = threadIdx.x & 63;
  const double none = -(double)kInf;
  const bool grouped = a.top_groups < a.groups && !bad;
  const bool scored = a.bias && !bad, sums = grouped && (a.bias || a.best > 1);
  double top = none, sum = 0;
  if ((scored || sums) && !a.sigmoid) {
    for (int e = lane; e < a.experts; e += 64) {
      const double x = elem_f32<FMT>(elem_bits<FMT>(row, e));
      top = x > top ? x : top;
    }
    top = row_max<64>(top);
    if (top == none) top = 0;
    for (int e = lane; e < a.experts; e += 64) sum += exp((double)elem_f32<FMT>(elem_bits<FMT>(row, e)) - top);
    sum = row_sum<64>(sum);
  }
  uint64_t kept = ~0ull;
  // first the groups' keys, then the experts'
#pragma unroll 1
  for (int pass = grouped ? 0 : 1; pass < 2; ++pass) {
    const bool score = pass == 0 ? sums : scored;
    for (int e = lane; e < a.experts; e += 64) {
      const double x = elem_f32<FMT>(elem_bits<FMT>(row, e));
      double k = x;
      if (score) {
        const double d = exp(a.sigmoid ? -x : x - top);
        k = (a.sigmoid ? 1.0 / (1.0 + d) : d / sum) + (a.bias ? (double)a.bias[e] : 0.0);
      }
      const bool held = pass == 0 || !grouped || (kept >> (e / (a.experts / a.groups)) & 1);
      keys[e] = x > none && k == k && held ? k : none;
    }
    bool open = false;
    if (pass == 0) kept = best_groups<64>(a, keys, 0.0, &open);
  }
  wave_sync();
  for (int j = 0; j < a.topk; ++j) {
    double m = none;
    int at = a.experts;
    for (int e = lane; e < a.experts; e += 64) {
      const double k = keys[e];
      if (k > m) m = k, at = e;
    }
    const double best = row_max<64>(m);
    // of the lanes that hold it, the lowest expert
    int e = m == best ? at : a.experts;
    steps<6>([&](auto s) {
      const int o = across<s.value>(e);
      e = o < e ? o : e;
    });
    if (lane == 0) {
      chosen[j] = best > none ? e : -1;
      if (best > none) keys[e] = none;
    }
    wave_sync();
  }
  if (lane < a.topk && chosen[lane] >= 0) logit[lane] = elem_f32<FMT>(elem_bits<FMT>(row, chosen[lane]));
  wave_sync();
}

// An expert of a lane's i-th place, and the place in LDS of its bias: a token's lanes read their i-th ones beside each
// other.
struct Pick {
  int both;  // bias place << 16 | expert
  __device__ __forceinline__ int expert() const { return both & 0xffff; }
  __device__ __forceinline__ int place() const { return both >> 16; }
};
template <int L>
__device__ __forceinline__ Pick pick(int e0, int i) {
  return Pick{(i * L + (int)(threadIdx.x % L)) << 16 | (e0 + i)};
}

// The order by keys in float64 of a token's experts that may be among the chosen: bits `within` of each lane's, up to L
// in the token, `before` of them in the lanes before.  All of a wave's lanes come here, also those of tokens that do not
// ask for it.
template <int FMT, int L>
__device__ __forceinline__ void order_exactly(const RouteArgs &a, const char *row, const float *bias, bool asked,
                                              uint32_t within, int before, int around, int e0, double *keys, Pick *ids,
                                              int *chosen, float *logit) {
  const int l = threadIdx.x % L;
  double top = -(double)kInf, sum = 0;
  if (!a.sigmoid) {
    for (int e = l; e < a.experts; e += L) {
      const double x = elem_f32<FMT>(elem_bits<FMT>(row, e));
      top = x > top ? x : top;
    }
    top = row_max<L>(top);
    if (top == -(double)kInf) top = 0;
    for (int e = l; e < a.experts; e += L) sum += exp((double)elem_f32<FMT>(elem_bits<FMT>(row, e)) - top);
    sum = row_sum<L>(sum);
  }
  if (asked)
    for (; within; within &= within - 1) ids[before++] = pick<L>(e0, __builtin_ctz(within));
  wave_sync();
  const bool held = asked && l < around;
  const Pick own = held ? ids[l] : Pick{0};
  const int e = own.expert();
  const float x = elem_f32<FMT>(elem_bits<FMT>(row, e));
  const double d = exp(a.sigmoid ? -(double)x : x - top);
  const double key = (a.sigmoid ? 1.0 / (1.0 + d) : d / sum) + (double)bias[own.place()];
  if (held) keys[l] = key;
  wave_sync();
  if (held) {
    int rank = 0;
    for (int j = 0; j < around; ++j) rank += keys[j] > key || (keys[j] == key && ids[j].expert() < e);
    if (rank < a.topk) {
      chosen[rank] = e;
      logit[rank] = x;
    }
  }
  wave_sync();
}

// choose_exactly for each of a wave's tokens whose lanes say `again`; t0, slot: the first of them, and its place in
// chosen and logit.
template <int FMT, int L, int K>
__device__ __forceinline__ void choose_again(bool again, bool bad, int64_t t0, int slot, double *keys,
                                             int (*chosen)[K], float (*logit)[K]) {
  if (!__ballot(again)) return;
  const int flags = (again ? 1 : 0) | (bad ? 2 : 0);
#pragma unroll 1
  for (int n = 0; n < 64 / L; ++n) {
    const int of = __builtin_amdgcn_readlane(flags, n * L);
    if (!(of & 1)) continue;  // uniform
    const RouteArgs a = args_again();
    const int64_t t = t0 + n < a.tokens ? t0 + n : a.tokens - 1;
    choose_exactly<FMT>(a, (const char *)a.logits + t * a.ld * fmt_bytes(FMT), (of & 2) != 0, keys, chosen[slot + n],
                        logit[slot + n]);
  }
}

// The weights of a token's choices, which lie in chosen and logit (in LDS): lane l's are l, l + L, ...  P of them.
// top, sum: of the row, for a softmax that is not renormalised.
template <int L, int P>
__device__ __forceinline__ void weigh(const RouteArgs &a, float top, float sum, bool bad, bool held, int64_t t,
                                      const int *chosen, const float *logit) {
  const int l = threadIdx.x % L;
  float x[P], s[P], part = 0.f;
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
    for (int p = 1; p < P; ++p) m = x[p] > m ? x[p] : m;
    top = row_max<L>(m);
    if (a.sigmoid && top > 0.f) top = 0.f;
    if (top == -kInf) top = 0.f;
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
  if (a.sigmoid && !a.renormalize) sum = 1.f;
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
// The 8 largest of V, falling.
template <int V>
__device__ __forceinline__ void largest8(int (&best)[8], const int (&key)[V]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) best[i] = i < V ? key[i % V] : kNone;
  if constexpr (V > 1) sort8(best);
#pragma unroll
  for (int n = 8; n < V; n += 8) {
    int more[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) more[i] = key[(n + i) % V];
    sort8(more);
    join8(best, more);
    merge8(best);
  }
}

struct Choice {
  float key, x, bias;
  Pick e;
};

template <int FMT, int L, int V>
__global__ __launch_bounds__(kThreads) void route8_kernel(RouteArgs first) {
  constexpr int kTokens = kThreads / L;
  __shared__ double keys[4][L * V < 64 ? 64 : L * V];  // of the choice in float64: a wave's
  __shared__ float bias_of[L * V];         // -inf for NaN; by places
  __shared__ Choice list[kTokens][9];      // (8; the rows of a wave's tokens on different banks)
  __shared__ double near_keys[kTokens][L];
  __shared__ Pick near_ids[kTokens][L];
  __shared__ int chosen[kTokens][8];
  __shared__ float logit[kTokens][8];
  RouteArgs a = first;
  const int slot = threadIdx.x / L, l = threadIdx.x % L;
  // Each group's experts on lanes of its own (a power of two): lane l has n from e0.
  auto first_of = [&](int lane) { return (lane >> a.shift) * a.size + (lane & ((1 << a.shift) - 1)) * a.per; };
  auto count_of = [&](int lane) {
    const int in = (lane & ((1 << a.shift) - 1)) * a.per, left = a.experts - first_of(lane);
    const int n = a.size - in < a.per ? a.size - in : a.per;
    return n < left ? n : left;  // (0 and less: none)
  };
  const int e0 = first_of(l);
  if (a.bias) {
    for (int i = threadIdx.x; i < L * V; i += kThreads) {
      if (i / L >= count_of(i % L)) continue;
      const float b = a.bias[first_of(i % L) + i / L];
      bias_of[i] = b == b ? b : -kInf;
    }
    __syncthreads();
  }
  const int64_t t = a.t0 + (int64_t)blockIdx.x * kTokens + slot;
  {
    const bool held = t < a.tokens;
    const bool grouped = a.top_groups < a.groups, scored = a.bias != nullptr;  // uniform
    const bool sums = grouped && (scored || a.best > 1);
    int key[V];
    bool open, bad;
    float top = 0.f, sum = 1.f, by = 1.f, error;
    {
      float x[V];
      load_row<FMT, L>(x, a, held ? t : a.tokens - 1, e0, count_of(l));
      // a NaN is above +inf or below -inf in this order
      int hi, lo;
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = ordered(x[i]);
      hi = lo = key[0];
#pragma unroll
      for (int i = 1; i < V; ++i) hi = key[i] > hi ? key[i] : hi, lo = key[i] < lo ? key[i] : lo;
      bad = row_ballot<L>(hi > (a.sigmoid ? 0x7f800000 : 0x7f7fffff) || lo < kNone) != 0;
      open = bad;
      if (!a.sigmoid && (scored || sums || !a.renormalize)) {
        soft_stats<L>(x, top, sum);
        by = one_over(sum);
      }
      error = score_error(a.sigmoid, by);
      if (scored || sums) {
        float g[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float s = score_of(a.sigmoid, x[i], top, by) + (scored ? bias_of[i * L + l] : 0.f);
          g[i] = x[i] > -kInf ? s : -kInf;
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
          const int lanes = 1 << a.shift;  // of a group
          steps<log2_of(L)>([&](auto s) {
            if ((1 << s.value) < lanes) {
              const float o1 = across<s.value>(b1), o2 = across<s.value>(b2);
              const float least = o1 < b1 ? o1 : b1, rest = o2 > b2 ? o2 : b2;
              b1 = o1 > b1 ? o1 : b1;
              b2 = least > rest ? least : rest;
            }
          });
          if (a.best == 1 || !(b2 > -kInf)) b2 = 0.f;
          const float tolerance = group_tolerance(error, b1, b2);
          b1 = group_sum(b1, b2);
          int before = 0;
          bool close = false;
          around_row<L>(b1, lanes, [&](float o, int r) {  // the other groups'
            before += o > b1 || (o == b1 && l >= r);
            close |= near_sums(o, b1, tolerance);
          });
          if (__ballot(close)) {  // it matters between one that is kept and one that is not
            for (int r = lanes; r < L; r += lanes) {
              const float o = __shfl(b1, (l - r) & (L - 1), L);
              const int ob = __shfl(before, (l - r) & (L - 1), L);
              open |= near_sums(o, b1, tolerance) && (ob < a.top_groups) != (before < a.top_groups);
            }
          }
#pragma unroll
          for (int i = 0; i < V; ++i) key[i] = before < a.top_groups ? key[i] : kNone;
        }
      }
      if (grouped && !sums) {
        int b1 = key[0];
#pragma unroll
        for (int i = 1; i < V; ++i) b1 = key[i] > b1 ? key[i] : b1;
        const int lanes = 1 << a.shift;
        steps<log2_of(L)>([&](auto s) {
          if ((1 << s.value) < lanes) {
            const int o = across<s.value>(b1);
            b1 = o > b1 ? o : b1;
          }
        });
        int before = 0;
        around_row<L>(b1, lanes, [&](int o, int r) { before += o > b1 || (o == b1 && l >= r); });
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = before < a.top_groups ? key[i] : kNone;
      }
    }

    // the smallest chosen key: the topk-th of the token's 8 largest, which every lane then has
    int least;
    {
      int best[8];
      largest8(best, key);
      steps<log2_of(L)>([&](auto s) {
        int other[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) other[i] = across<s.value>(best[i]);
        join8(best, other);
        merge8(best);
      });
      least = best[0];
#pragma unroll
      for (int i = 1; i < 8; ++i)
        if (i < a.topk) least = best[i];
    }
    const bool all = least <= kNone;  // fewer than topk are left
    if (all) least = kNone + 1;

    // who reaches it
    uint32_t mine = 0;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) mine = mine + mine + (key[i] >= least);
    int count = __builtin_popcount(mine), upto = row_scan<L>(count);
    const int total = __shfl(upto, L - 1, L);
    if (__ballot(total > a.topk)) {  // equal keys at the border: the lowest indices
      uint32_t equal = 0;
#pragma unroll
      for (int i = V - 1; i >= 0; --i) equal = equal + equal + (key[i] == least);
      const int own = __builtin_popcount(equal), before = row_scan<L>(own);
      const int excess = total > a.topk ? total - a.topk : 0, sum_equal = __shfl(before, L - 1, L);
      // of the token's equal ones the first sum_equal - excess stay
      int drop = before - (sum_equal - excess);
      drop = drop < 0 ? 0 : drop > own ? own : drop;
      for (; drop > 0; --drop) {
        const uint32_t last = 0x80000000u >> __builtin_clz(equal);
        equal ^= last;
        mine ^= last;
        --count;
      }
      upto = row_scan<L>(count);
    }
    const uint32_t taken = mine;
    for (int at = upto - count; mine; mine &= mine - 1) list[slot][at++].e = pick<L>(e0, __builtin_ctz(mine));
    wave_sync();
    const int n = total < a.topk ? total : a.topk;

    // lane j orders the j-th of the list
    Choice c{-kInf, 0.f, 0.f, {0}};
    const char *const row = (const char *)a.logits + (held ? t : a.tokens - 1) * a.ld * fmt_bytes(FMT);
    if (l < n) {
      c.e = list[slot][l].e;
      c.x = elem_f32<FMT>(elem_bits<FMT>(row, c.e.expert()));
      c.key = c.x;
      if (scored) {
        c.bias = bias_of[c.e.place()];
        c.key = score_of(a.sigmoid, c.x, top, by) + c.bias;
      }
      list[slot][l] = c;
    }
    if (l < 8) chosen[slot][l] = -1;
    wave_sync();
    int rank = 0;
    bool close = false;
    const float tolerance = key_error(error, c.key);
    for (int j = 0; j < a.topk; ++j) {
      const Choice o = list[slot][j];
      const bool other = j < n && j != l;
      rank += other && (o.key > c.key || (o.key == c.key && o.e.expert() < c.e.expert()));
      // (equal logits and biases make equal keys, whatever they round to)
      close |= other && fabsf(o.key - c.key) <= tolerance && (o.x != c.x || o.bias != c.bias);
    }
    if (l < n) {
      chosen[slot][rank] = c.e.expert();
      logit[slot][rank] = c.x;
    }
    if (scored) {
      // those that are not chosen but as near to the last chosen one as keys may be off
      const int near = all ? least : near_limit(least, error);
      uint32_t within = 0;
#pragma unroll
      for (int i = V - 1; i >= 0; --i) within = within + within + (key[i] >= near);
      const int own = __builtin_popcount(within), around = row_sum<L>(own);
      bool unclear = l < n && close;
      if (__ballot(around > n)) {
        // (the last chosen one's logit and bias)
        float lx = 0.f, lb = 0.f;
        for (int j = 0; j < n; ++j)
          if (ordered(list[slot][j].key) == least) lx = list[slot][j].x, lb = list[slot][j].bias;
        for (uint32_t rest = within & ~taken; rest; rest &= rest - 1) {
          const int i = __builtin_ctz(rest);
          unclear |= elem_f32<FMT>(elem_bits<FMT>(row, e0 + i)) != lx || bias_of[i * L + l] != lb;
        }
      }
      unclear = row_ballot<L>(unclear) != 0;
      open |= unclear && around > L;
      if (__ballot(unclear && !open))
        order_exactly<FMT, L>(a, row, bias_of, unclear && around <= L, within, row_scan<L>(own) - own, around, e0,
                              near_keys[slot], near_ids[slot], chosen[slot], logit[slot]);
    }
    wave_sync();
    choose_again<FMT, L>(row_ballot<L>(open) != 0, bad, t - slot % (64 / L), slot - slot % (64 / L),
                                 keys[threadIdx.x >> 6], chosen, logit);
    a = args_again();
    weigh<L, 8 / L ? 8 / L : 1>(a, top, sum, bad, held, t, chosen[slot], logit[slot]);
  }
}

// ---- any number of choices, any groups ----
template <int FMT, int L, int V>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs first) {
  constexpr int kTokens = kThreads / L, K = RouteInfo::kMaxTopk, E = L * V < 64 ? 64 : L * V;
  __shared__ double keys[kTokens / 2][E];  // of a token in float32, of a wave's in float64
  __shared__ int chosen[kTokens][K];
  __shared__ float logit[kTokens][K];
  static_assert(kTokens / 2 >= 4, "the waves' keys fit");
  RouteArgs a = first;
  const int slot = threadIdx.x / L, l = threadIdx.x % L, e0 = l * V;
  const int64_t t = a.t0 + (int64_t)blockIdx.x * kTokens + slot;
  const bool held = t < a.tokens;
  float x[V], bias[V] = {}, top = 0.f, sum = 1.f;
  load_row<FMT, L>(x, a, held ? t : a.tokens - 1, e0, a.experts - e0);
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < a.experts) {
        const float b = a.bias[e0 + i];
        bias[i] = b == b ? b : -kInf;
      }
  }
  bool nan = false, inf = false;
#pragma unroll
  for (int i = 0; i < V; ++i) nan |= x[i] != x[i], inf |= x[i] == kInf;
  const bool bad = row_ballot<L>(nan || (inf && !a.sigmoid)) != 0;
  if (!a.sigmoid && !a.renormalize) soft_stats<L>(x, top, sum);
  const bool open = choose<L>(a, x, e0, bias, (float *)keys + slot * E, chosen[slot], logit[slot]);
  const int of_wave = slot - slot % (64 / L);
  choose_again<FMT, L>(open || bad, bad, t - slot % (64 / L), of_wave, (double *)((float *)keys + of_wave * E), chosen,
                       logit);
  a = args_again();
  weigh<L, K / L>(a, top, sum, bad, held, t, chosen[slot], logit[slot]);
}

// ---- the gradient ----
// With g the gradients of the weights times the factor, q the chosen scores over their sum:
//   renormalised  dx_e = q (g - sum g q)       (sigmoid: times 1 - s_e), 0 where not chosen
//   softmax       dx_e = s_e (g_e - sum g s)
//   sigmoid       dx_e = s_e (1 - s_e) g_e
// A token's row is put together in LDS: zeros, then the chosen experts' entries (those of an expert that is chosen
// twice added in their order), and leaves in vectors.  P: choices per lane.
template <int FMT, int L, int V, int P>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(RouteArgs a) {
  constexpr int kTokens = kThreads / L, ES = fmt_bytes(FMT), K = L * P;
  struct Entry {
    int e;
    float d;
  };
  __shared__ __attribute__((aligned(16))) float rows[kTokens][L * V];
  __shared__ __attribute__((aligned(16))) Entry entries[kTokens][K];
  const int slot = threadIdx.x / L, l = threadIdx.x % L;
  const int64_t t = a.t0 + (int64_t)blockIdx.x * kTokens + slot;
  const bool held = t < a.tokens;
  const int64_t at = held ? t : a.tokens - 1;
  const char *const in = (const char *)a.logits + at * a.ld * ES;
  const bool whole = !a.sigmoid && !a.renormalize;  // the probabilities of every expert
  float x[P], g[P], top = 0.f, sum = 1.f;
  int e[P];
#pragma unroll
  for (int q = 0; q < P; ++q) {
    const int j = l + q * L;
    e[q] = j < a.topk ? a.ids[at * a.topk + j] : -1;
    g[q] = j < a.topk ? a.weights[at * a.topk + j] * a.factor : 0.f;
    if (e[q] >= a.experts) e[q] = -1;
    x[q] = -kInf;
    if (e[q] < 0) g[q] = 0.f;
    else x[q] = elem_f32<FMT>(elem_bits<FMT>(in, e[q]));
  }
  // this lane's elements of the row: vectors of N, L of them apart
  constexpr int N = V % (16 / ES) == 0 ? 16 / ES : 1;
  const bool vec = N > 1 && a.experts == L * V;
  float row[V];
  auto index = [&](int i) { return vec ? (i / N * L + l) * N + i % N : i * L + l; };
#pragma unroll
  for (int i = 0; i < V; ++i) rows[slot][i * L + l] = 0.f;
  if (whole) {
    if (vec) {
#pragma unroll
      for (int h = 0; h < V / N; ++h) {
        Vec<FMT> v;
        v.unpack(*(const Raw16 *)(in + (h * L + l) * N * ES));
#pragma unroll
        for (int i = 0; i < N; ++i) row[(h * N + i) % V] = v.v[i % Vec<FMT>::N];
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) row[i] = index(i) < a.experts ? elem_f32<FMT>(elem_bits<FMT>(in, index(i))) : -kInf;
    }
    soft_stats<L>(row, top, sum);
  } else if (a.renormalize) {
    float m = x[0];
#pragma unroll
    for (int q = 1; q < P; ++q) m = x[q] > m ? x[q] : m;
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
    s[q] /= sum;
    dot += g[q] * s[q];
  }
  dot = a.renormalize || whole ? row_sum<L>(dot) : 0.f;
#pragma unroll
  for (int q = 0; q < P; ++q) {
    g[q] = whole ? g[q] : s[q] * left[q] * (g[q] - dot);
    entries[slot][l + q * L] = Entry{e[q], g[q]};
  }
  wave_sync();
#pragma unroll
  for (int q = 0; q < P; ++q) {
    const int j = l + q * L;
    float d = 0.f;
    bool one = e[q] >= 0;
    for (int o = 0; o < a.topk; ++o) {
      const Entry other = entries[slot][o];
      if (other.e == e[q]) {
        d += other.d;
        one &= o >= j;
      }
    }
    if (one) rows[slot][e[q]] = d;
  }
  wave_sync();
  if (!held) return;
  char *const out = (char *)a.dlogits + t * a.ldd * ES;
  auto entry = [&](float d, float v) { return whole ? expf(v - top) / sum * (d - dot) : d; };
  if (vec) {
#pragma unroll
    for (int h = 0; h < V / N; ++h) {
      Vec<FMT> v;
#pragma unroll
      for (int i = 0; i < N; ++i)
        v.v[i % Vec<FMT>::N] = entry(rows[slot][(h * L + l) * N + i], whole ? row[(h * N + i) % V] : 0.f);
      *(Raw16 *)(out + (h * L + l) * N * ES) = v.pack();
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (index(i) < a.experts)
        put_bits<FMT>(out, index(i), f32_elem<FMT>(entry(rows[slot][index(i)], whole ? row[i] : 0.f)));
  }
}

// Places a row on L lanes of up to V experts, where groups are chosen each on lanes of its own, a power of two of them;
// false: they do not hold it.
bool place(RouteArgs &a, int L, int V) {
  if (a.experts > L * V) return false;
  int lanes = L;
  a.size = a.experts;
  a.per = V;
  if (a.top_groups < a.groups) {
    while (lanes > 0 && L / lanes < a.groups) lanes /= 2;
    if (lanes == 0) return false;
    a.size = a.experts / a.groups;
    a.per = (a.size + lanes - 1) / lanes;
  }
  a.shift = 0;
  while (1 << a.shift < lanes) ++a.shift;
  return a.per <= V;
}

// f(arguments, workgroups) over launches of 2^23 workgroups at most (work-items below 2^32).
template <class F>
hipError_t over_tokens(const RouteArgs &base, int tokens, F &&launch) {
  const int64_t most = ((int64_t)1 << 23) * tokens;
  for (int64_t t0 = 0; t0 < base.tokens; t0 += most) {
    RouteArgs a = base;
    a.t0 = t0;
    const int64_t n = base.tokens - t0 < most ? base.tokens - t0 : most;
    launch(a, (unsigned)((n + tokens - 1) / tokens));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int FMT, int L, int V>
hipError_t route8(const RouteArgs &base, hipStream_t stream) {
  return over_tokens(base, kThreads / L, [&](const RouteArgs &a, unsigned blocks) {
    hipLaunchKernelGGL((route8_kernel<FMT, L, V>), dim3(blocks), dim3(kThreads), 0, stream, a);
  });
}
template <int FMT, int L, int V>
hipError_t route_any(const RouteArgs &base, hipStream_t stream) {
  return over_tokens(base, kThreads / L, [&](const RouteArgs &a, unsigned blocks) {
    hipLaunchKernelGGL((route_kernel<FMT, L, V>), dim3(blocks), dim3(kThreads), 0, stream, a);
  });
}
template <int FMT, int L, int V>
hipError_t backward(const RouteArgs &base, hipStream_t stream) {
  return over_tokens(base, kThreads / L, [&](const RouteArgs &a, unsigned blocks) {
    if (a.topk <= L)
      hipLaunchKernelGGL((route_backward_kernel<FMT, L, V, 1>), dim3(blocks), dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((route_backward_kernel<FMT, L, V, RouteInfo::kMaxTopk / L>), dim3(blocks), dim3(kThreads), 0,
                         stream, a);
  });
}

template <int FMT>
hipError_t route_fmt(const RouteArgs &a, hipStream_t stream) {
  const int E = a.experts;
  // The fewest lanes that hold a row in 16 experts each: what is done for each lane's list is done for fewer (65536 tokens,
  // us, 16 | 8 lanes: 8 experts 11.2 | 6.5, 64 14.8 | 9.7, 128 16.9 | 13.0).  Of 32 experts a lane's own work takes over
  // (16 | 8 lanes of 256 experts: 65536 tokens 24.3 | 20.9, with a bias 34.8 | 37; 64 tokens in groups 7.1 | 9.6).
  if (a.topk <= 8) {
    RouteArgs b = a;
    if (place(b, 8, 1)) return route8<FMT, 8, 1>(b, stream);
    if (place(b, 8, 2)) return route8<FMT, 8, 2>(b, stream);
    if (place(b, 8, 8)) return route8<FMT, 8, 8>(b, stream);
    if (place(b, 8, 16)) return route8<FMT, 8, 16>(b, stream);
    if (place(b, 16, 16)) return route8<FMT, 16, 16>(b, stream);
    if (place(b, 32, 16)) return route8<FMT, 32, 16>(b, stream);
  }
  if (E <= 16) return route_any<FMT, 16, 1>(a, stream);
  if (E <= 64) return route_any<FMT, 16, 4>(a, stream);
  if (E <= 128) return route_any<FMT, 16, 8>(a, stream);
  if (E <= 256) return route_any<FMT, 16, 16>(a, stream);
  return route_any<FMT, 32, 16>(a, stream);
}

template <int FMT>
hipError_t backward_fmt(const RouteArgs &a, hipStream_t stream) {
  if (a.experts <= 16) return backward<FMT, 16, 1>(a, stream);
  if (a.experts <= 64) return backward<FMT, 16, 4>(a, stream);
  if (a.experts <= 128) return backward<FMT, 16, 8>(a, stream);
  if (a.experts <= 256) return backward<FMT, 16, 16>(a, stream);
  return backward<FMT, 32, 16>(a, stream);
}

}  // namespace

hipError_t launch_route(const RouteArgs &a, hipStream_t stream) {
  return a.fmt == FMT_F32 ? route_fmt<FMT_F32>(a, stream)
                          : a.fmt == FMT_F16 ? route_fmt<FMT_F16>(a, stream) : route_fmt<FMT_BF16>(a, stream);
}
hipError_t launch_route_backward(const RouteArgs &a, hipStream_t stream) {
  return a.fmt == FMT_F32 ? backward_fmt<FMT_F32>(a, stream)
                          : a.fmt == FMT_F16 ? backward_fmt<FMT_F16>(a, stream) : backward_fmt<FMT_BF16>(a, stream);
}

}  // namespace tsm
