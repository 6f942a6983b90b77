// Shared by the kernels of the block-scaled 8-bit product.
#pragma once

#include "sbp_groups.cuh"

namespace sbp {
namespace mm8 {

constexpr int64_t MAX_SIDE = 1 << 20;
static_assert(MAX_GROUPS * MAX_SIDE < INT32_MAX - 256, "rows of all matrices are counted in 32 bits");

struct P {
  const uint8_t* A;   // rows: [T, K]; columns: [na, 128 * kblocks]
  const float* sa;    // a scale for each row and block
  int64_t lda, sa_pitch;
  const uint8_t* B;   // rows: [E, nb, K]; columns: [nb, 128 * kblocks]
  const float* sb;    // a scale for each 128 rows and block
  int64_t ldb, sb_pitch, b_stride, sb_stride;   // strides: of an expert
  const int32_t* offsets;
  int64_t T, K;       // rows (tokens) of all experts; bytes of a row of A and B
  int E, na, nb, kblocks;
  int columns;        // the sum goes over an expert's tokens
  int out, accumulate;
  int64_t c_stride;
  void* C;
  int32_t* status;
  uint64_t limit_ns;
  int stall;          // failure-detection hook: the products wait for what never comes
};

// A unit's rows of A (row0 .., at most `unit`), its expert, its blocks of 128 of the sum.
struct Unit {
  int e, row0, rows, kb0, kb1;
};

// Unit u of `unit` rows of A; every lane of a warp calls it, with a table that has been checked.
__device__ __forceinline__ Unit unit_of(const P& p, int unit, int u) {
  Unit w;
  if (p.columns) {
    const int per = (p.na + unit - 1) / unit;
    w.e = u / per;
    w.row0 = (u - w.e * per) * unit;
    w.rows = min(unit, p.na - w.row0);
    // the expert's blocks of 128 tokens lie behind those of the experts before it
    if (!p.offsets) {
      w.kb0 = 0;
      w.kb1 = p.kblocks;
      return w;
    }
    const int lane = threadIdx.x % 32;
    int before = 0;
    for (int e = lane; e < w.e; e += 32) before += (p.offsets[e + 1] - p.offsets[e] + 127) / 128;
#pragma unroll
    for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    w.kb0 = before;
    w.kb1 = before + (p.offsets[w.e + 1] - p.offsets[w.e] + 127) / 128;
    return w;
  }
  const Group g = find_unit(p.offsets, p.E, p.T, unit, u);
  w.e = g.e;
  w.row0 = g.row0 + g.i * unit;
  w.rows = min(unit, g.rows - g.i * unit);
  w.kb0 = 0;
  w.kb1 = p.kblocks;
  return w;
}

// How many units of `unit` rows of A the call has, as far as the host knows: experts that few rows
// go to have at least one each, long ones a last unit that is half full on average, and there are no
// more than T rows can make (one row to one of 64 experts is one unit and not 32).
inline int64_t about_units(const P& p, int64_t unit) {
  if (p.columns) return (int64_t)p.E * ((p.na + unit - 1) / unit);
  if (p.E == 1) return (p.T + unit - 1) / unit;
  const int64_t used = p.E < p.T ? p.E : p.T, more = p.T / unit + p.E / 2;
  const int64_t units = used > more ? used : more, most = max_units(p.T, p.E, unit);
  return units < most ? units : most;
}
// Blocks of 128 that a unit sums over, on average.
inline int64_t about_blocks(const P& p) {
  return p.columns ? (p.kblocks + p.E - 1) / p.E : p.kblocks;
}

void ran(int kernel);   // for sbp_last_product_kernel

// The kernel for many rows (sbp_mm8_tc.cu): enqueues the status word's reset and the product.
cudaError_t many(const P& p, cudaStream_t s);
int64_t many_ns(const P& p);   // about how long it takes
// Few rows of many experts (sbp_mm8_swap.cu; rows only): the same.
cudaError_t swap(const P& p, cudaStream_t s);
int64_t swap_ns(const P& p);

}  // namespace mm8
}  // namespace sbp
