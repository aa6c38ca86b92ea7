// runs.cuh -- equal runs of a call's work for one persistent CTA per SM.
//
// The units of all items are laid end to end (total of them); CTA c of n takes
// units [lo(c), lo(c + 1)), lengths that differ by one at most.  n is at most
// total, so no run is empty and an item's pieces lie in consecutive CTAs.
#pragma once

#include <stdint.h>

namespace attn {

// 64-bit division is a routine of a hundred instructions, and counts are small
// almost always: a prologue full of them cost 7 us
__device__ __forceinline__ int div_pos(int a, int b) { return a / b; }
__device__ __forceinline__ int64_t div_pos(int64_t a, int64_t b) {
  if (((a | b) >> 31) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

template <typename I>
struct RunsOf {
  I q;  // units of a run; the first r runs have one more
  int n, r;
  __device__ static RunsOf make(I total, int grid) {
    RunsOf x;
    x.n = static_cast<int>(total < grid ? total : grid);
    x.q = x.n > 0 ? div_pos(total, static_cast<I>(x.n)) : 0;
    x.r = static_cast<int>(total - x.q * x.n);
    return x;
  }
  __device__ I lo(int c) const { return c * q + (c < r ? c : r); }
  __device__ int of(I unit) const {  // the run that holds the unit
    const I big = r * (q + 1);
    return static_cast<int>(unit < big ? div_pos(unit, q + 1) : r + div_pos(unit - big, q));
  }
};

using Runs = RunsOf<int>;
using Runs64 = RunsOf<int64_t>;

}  // namespace attn
