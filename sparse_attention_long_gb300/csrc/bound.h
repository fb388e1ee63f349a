// The search for a bound among logits (sample.cu), over any way of counting, so that it
// also compiles for the host.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define DSA_BOUND_FN __device__ __forceinline__
#else
#define DSA_BOUND_FN inline
#endif

namespace dsa {
namespace sample {

// A key (ordered_key) that `need` threads or more reach, reach(key) being how many do; the
// search ends at `need`, a quarter and one, or at the largest such key.  0: fewer have a finite logit.
// top: the largest key of all (with lo, any number above); lo: 0, or a key that is known to be
// reached by so many.
//
// Keys are near where logits are near in their exponents, so first come steps down from top
// that double, four powers of two in all.  What lies further is mostly on the other side of
// zero, most of the keys away (the keys from 1 to -1 are half of all): the
// next guess is top with its sign changed, and then halves of the larger end.  After that
// every step halves the keys left, so that any logits take some 50 counts at most.
template <typename F>
DSA_BOUND_FN uint32_t reached_by(int need, uint32_t top, uint32_t lo, F reach) {
  constexpr uint32_t kZero = 0x80000000u, kLowest = 0x00800000u, kOctave = 1u << 23;  // of 0, of -FLT_MAX; a power of two
  if (need == 1) return top;
  const int few = need + need / 4 + 1;
  uint32_t hi = top + 1, step = 1u << 18;          // fewer than `need` threads reach hi
  const auto narrowed = [&](uint32_t mid) {        // true: near enough
    const int n = reach(mid);
    if (n >= need) lo = mid;
    else hi = mid;
    return n >= need && n <= few;
  };
  if (lo) {
    if (narrowed(lo)) return lo;
    // up from below (halves are compared: step stays below 2^31, where twice the step would pass 2^32 and the
    // search not end)
    for (; hi == top + 1 && (hi - lo) / 2 > step; step *= 2)
      if (narrowed(lo + step)) return lo;
  } else {
    for (;;) {
      const uint32_t mid = hi - kLowest > step ? hi - step : kLowest;
      if (narrowed(mid)) return lo;
      if (lo) break;
      if (mid == kLowest) return 0;
      if (top < kZero || step < 2 * kOctave) step *= 2;  // (below zero to the end: step is 2^31 then)
      else step = hi > ~top ? hi - ~top : hi;      // ~top: the key of the negated logit
    }
  }
  for (int i = 0; i < 8 && lo < kZero && hi > kZero && hi - lo > 2 * kOctave; ++i)
    if (narrowed(~lo > hi ? lo + kOctave : hi - kOctave)) return lo;
  while (hi - lo > 1)
    if (narrowed(lo + (hi - lo) / 2)) return lo;
  return lo;
}

}  // namespace sample
}  // namespace dsa
