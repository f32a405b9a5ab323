// What the expert router decides from float32 keys, and what it leaves to float64: plain arithmetic, for the kernels and
// for programs on the host.
#pragma once

#include <stdint.h>

namespace tsm {

// Floats in the order of their values as whole numbers (-0 as 0), and back.
constexpr int ordered(float f) {
  const int b = __builtin_bit_cast(int, f + 0.f);
  return b ^ (b >> 31 & 0x7fffffff);
}
constexpr float of_ordered(int i) { return __builtin_bit_cast(float, i ^ (i >> 31 & 0x7fffffff)); }
constexpr int kNone = -0x7f800001;  // -inf: the key of what may not be chosen, and of places without an expert

// How far two float32 keys may lie apart and be in the other order, where a score is off by `error` (score_error).
constexpr float key_error(float error, float key) { return 2 * error + 0x1p-22f * __builtin_fabsf(key); }

// The sum of a group's largest keys (b2 0: of one key; b1 -inf: it has none).  Of finite keys it is kept within float32's
// range, where it is near (group_tolerance) all that it now equals: of two keys of the lowest value, a mask, it must not
// become -inf.
constexpr float group_sum(float b1, float b2) {
  constexpr float top = __FLT_MAX__;
  const float sum = b1 + b2;
  return !(__builtin_fabsf(b1) <= top) ? b1 : sum < -top ? -top : sum > top ? top : sum;
}
constexpr double group_sum(double b1, double b2) { return b1 + b2; }

// How far a group's sum of keys b1 and b2 (0: of one key) may lie from another's and be in the other order.  Each key is
// off by `error` and its own rounding, whatever their sum leaves of them, and the sum by one more: 2 error + 2^-23 (|b1| +
// |b2|) for a group.  Twice that holds for two groups, whichever is the larger one's: of two groups one at least finds the
// other near.  (And twice the roundings' part, for those of the comparison.)  Finite for infinite keys too, so that a
// group of none, or of an infinite key, is near nothing.
constexpr float group_tolerance(float error, float b1, float b2) {
  constexpr float top = __FLT_MAX__;
  const float m1 = __builtin_fabsf(b1), m2 = __builtin_fabsf(b2);
  return 4 * error + 0x1p-21f * (m1 < top ? m1 : top) + 0x1p-21f * (m2 < top ? m2 : top);
}
constexpr bool near_sums(float other, float own, float tolerance) { return __builtin_fabsf(other - own) <= tolerance; }

// The least key that may be as large as the smallest chosen one: that one at most, and above kNone, since places without
// an expert hold it (from a key of float32's lowest value the difference is -inf, from an infinite one NaN).
constexpr int near_limit(int least, float error) {
  const float f = of_ordered(least);
  const int near = ordered(f - key_error(error, f));
  return near > least ? least : near > kNone ? near : kNone + 1;
}

// e / size of an expert e < 512, by a product with group_magic(size).  Exact: size * magic passes 2^20 by less than size,
// and e times that stays below 2^20.
constexpr uint32_t group_magic(uint32_t size) { return ((1u << 20) + size - 1) / size; }
constexpr uint32_t group_of(uint32_t e, uint32_t magic) { return e * magic >> 20; }

}  // namespace tsm
