// Rows shared out to experts: device int32 offsets [E + 1], rows [offsets[e], offsets[e + 1]) of
// expert e (null: one expert of all the rows).  Kernels find their unit's expert from the table
// itself, so that a captured call follows what the table holds when it runs.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace sbp {

constexpr int64_t MAX_GROUPS = 1024;

struct Group {
  int e = 0;            // expert
  int i = 0;            // unit of the expert
  int row0 = 0, rows = 0;   // the expert's first row, how many it has
  int total = 0;        // units of all experts
  bool found = false, bad = false;
};

// Unit b of the units of `unit` rows that the experts' rows make up, each expert's from its first
// row on.  Called by all lanes of a warp, the same answer in each; a table that does not begin at
// 0, decreases or passes T is bad.
__device__ __forceinline__ Group find_unit(const int32_t* off, int E, int64_t T, int unit, int b) {
  Group g;
  if (!off) {
    g.total = (int)((T + unit - 1) / unit);
    g.found = b < g.total;
    g.i = b;
    g.rows = (int)T;
    return g;
  }
  const int lane = threadIdx.x % 32;
  int base = 0;
  bool bad = false;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < E) {
      lo = off[e];
      hi = off[e + 1];
      bad |= lo < 0 || hi < lo || hi > T || (e == 0 && lo != 0);
    }
    const int n = bad ? 0 : (int)(((int64_t)hi - lo + unit - 1) / unit);
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, b >= base + x - n && b < base + x);
    if (hit) {
      const int src = __ffs(hit) - 1;
      g.found = true;
      g.e = e0 + src;
      g.i = b - base - __shfl_sync(0xffffffffu, x - n, src);
      g.row0 = __shfl_sync(0xffffffffu, lo, src);
      g.rows = __shfl_sync(0xffffffffu, hi - lo, src);
    }
    base += __shfl_sync(0xffffffffu, x, 31);
  }
  g.total = base;
  g.bad = __any_sync(0xffffffffu, bad);
  return g;
}

// The most units of `unit` rows that T rows of E experts can make up.
inline int64_t max_units(int64_t T, int64_t E, int64_t unit) {
  const int64_t used = E < T ? E : T;
  return (T + (unit - 1) * used) / unit;
}

}  // namespace sbp
