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
// 0, decreases or passes T is bad.  (With e1 > 0: unit b of those of the experts from e1 on.)
__device__ __forceinline__ Group find_unit(const int32_t* off, int E, int64_t T, int unit, int b, int e1 = 0) {
  Group g;
  if (!off) {
    g.total = (int)((T + unit - 1) / unit);
    g.found = b < g.total;
    g.i = b;
    g.rows = (int)T;
    return g;
  }
  // 32 experts at a time: their units' sum, by which the 32 that unit b lies in are known; the
  // prefix over those is formed once, at the end.
  const int lane = threadIdx.x % 32;
  int base = 0, at = 0, e0 = -1;
  int lo = 0, n = 0, rows = 0;   // of this lane's expert among the 32
  bool bad = false;
#pragma unroll 4
  for (int i = e1; i < E; i += 32) {
    const int e = i + lane;
    int l = 0, h = 0;
    if (e < E) {
      l = off[e];
      h = off[e + 1];
    }
    const bool wrong = l < 0 || h < l || h > T || (e == 0 && l != 0);
    const int m = wrong ? 0 : (int)(((int64_t)h - l + unit - 1) / unit);
    const int sum = (int)__reduce_add_sync(0xffffffffu, (unsigned)m);
    bad |= wrong;
    if (b >= base && b < base + sum) {
      at = base;
      e0 = i;
      lo = l;
      n = m;
      rows = h - l;
    }
    base += sum;
  }
  if (e0 >= 0) {
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, b < at + x)) - 1;
    g.found = true;
    g.e = e0 + src;
    g.i = b - at - __shfl_sync(0xffffffffu, x - n, src);
    g.row0 = __shfl_sync(0xffffffffu, lo, src);
    g.rows = __shfl_sync(0xffffffffu, rows, src);
  }
  g.total = base;
  g.bad = __any_sync(0xffffffffu, bad);
  return g;
}

// The same, called by all 256 threads of a block, whose warps share out long tables (16384 tokens x
// 2048 columns of 256 and 1024 equal experts into tiles: 38 and 134 us, 40 and 245 by each warp alone).
__device__ __forceinline__ Group find_unit_of_block(const int32_t* off, int E, int64_t T, int unit, int b) {
  if (!off || E <= 32) return find_unit(off, E, T, unit, b);
  __shared__ int units[8], at[4];
  const int warp = threadIdx.x / 32, per = ((E + 255) / 256) * 32;
  const int e1 = min(warp * per, E), e2 = min(e1 + per, E);
  Group g = find_unit(off, e2, T, unit, -1, e1);
  if (threadIdx.x % 32 == 0) units[warp] = g.total;
  g.bad = __syncthreads_or(g.bad);
  if (g.bad) return g;
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    before += w < warp ? units[w] : 0;
    total += units[w];
  }
  if (b >= before && b < before + units[warp]) {   // in one warp at most
    const Group f = find_unit(off, e2, T, unit, b - before, e1);
    if (threadIdx.x % 32 == 0) {
      at[0] = f.e;
      at[1] = f.i;
      at[2] = f.row0;
      at[3] = f.rows;
    }
  }
  __syncthreads();
  g.total = total;
  g.found = b < total;
  if (g.found) {
    g.e = at[0];
    g.i = at[1];
    g.row0 = at[2];
    g.rows = at[3];
  }
  return g;
}

// A call without rows (T = 0): the status of its table, which may hold nothing but zeros, and, where it
// is good, n floats of zeros (a multiple of 4; null: none).
int no_rows(const int32_t* offsets, int64_t E, float* zeros, int64_t n, int32_t* status, cudaStream_t s);

// The most units of `unit` rows that T rows of E experts can make up.
inline int64_t max_units(int64_t T, int64_t E, int64_t unit) {
  const int64_t used = E < T ? E : T;
  return (T + (unit - 1) * used) / unit;
}

}  // namespace sbp
