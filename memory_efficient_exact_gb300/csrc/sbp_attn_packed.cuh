// Attention over packed documents (bf16, sm_103a): what its translation units share.
//
// The T tokens of a call are documents packed one behind the other, document s holding the
// rows [cu[s], cu[s+1]); rows at and after cu[n_seq] are padding.  With p_s the prefix
// length of document s, query i sees key j of its own document when j <= i or j lies in the
// prefix, so what a query sees is one interval of keys, and what a key is seen by is one
// interval of queries:
//   [lo_i, hi_i)   = [cu[s], max(i + 1, cu[s] + p_s))
//   [qlo_j, qhi_j) = [j < cu[s] + p_s ? cu[s] : j, cu[s+1])
// All four ends are non-decreasing, so a tile's blocks are found from its first and last
// row, and a tile is free of masking when its last row's lower end and its first row's
// upper end lie outside it.
// The score of a visible pair is  x = cap(scale q.k) - slope_h |i - j|  with
// cap(t) = c tanh(t / c) (c > 0) or t (c = 0).
#pragma once

#include "sbp_tc_common.cuh"

namespace sbp {

// Work of one unit of 256 queries: key blocks (of 128) [ja0, jb0) for its first 128
// queries and [ja1, jb1) for the others; ja0 <= ja1 <= jb0 <= jb1 (no gap between them).
// sums: the blocks that the dQ kernel walks first (see kSumBlocks), 8 * the first + how many.
struct __align__(16) PackedQUnit { int qp, ja0, jb0, ja1, jb1, sums, pad[2]; };
// A unit of up to this many key blocks walks them all first.
constexpr int kSumBlocks = 3;
// Work of one unit of 256 keys: query blocks (of 128) [b0, b0 + nb).
struct __align__(16) PackedKvUnit { int kp, b0, nb, pad; };

// What the kernels read besides the tensors; pointers into the workspace.
struct PackedWork {
  const int32_t *lo, *hi, *qlo, *qhi;   // [T]; rows behind the documents hold T in all four
  const PackedQUnit* qunits;            // [ceil(T / 256)], the longest first
  const PackedKvUnit* kvunits;          // [ceil(T / 256)], the longest first (backward)
  // Where the documents end inside a block of 128 rows and padding follows: that block's
  // number (else -1), and copies of its rows with the padding zeroed, [heads, 128, hd].  The
  // products that sum over rows read these: a probability of 0 times whatever the padding
  // holds would be NaN for an infinity or a NaN.
  const int32_t* tail;
  const void *tail_q, *tail_do;         // backward, H heads
  const void* tail_kv;                  // V in the forward, K in the backward, Hkv heads
  float* D;                             // [H, T] dO . O (backward)
  // [H, ceil(T / 256), 4] bytes: whether some of 64 queries need D from all of their keys (see
  // PackedScores::q_sums)
  const uint8_t* large;
};

struct PackedArgs {
  const void *Q, *K, *V, *O, *dO;
  const float* lse;
  const int32_t *cu, *prefix;
  const float* slopes;
  int64_t H, Hkv, T, hd;
  int32_t n_seq;
  float scale, softcap;
  int32_t* status;
};

namespace tc {
namespace pk {

// The unit of round t of SM pair pid: the units come longest first, so the rounds alternate
// in direction, which evens out what the pairs get.
__device__ __forceinline__ int next_unit(int t, int pid, int npairs) {
  return (t & 1) ? (t + 1) * npairs - 1 - pid : t * npairs + pid;
}

// Constants of the score in log2 units: with a cap, c tanh(y) = c - 2 c / (1 + e^(2 y)),
// y = s scale / c: one exponential and one reciprocal, the absolute error about c 2^-22
// (tanh.approx would leave c 2^-11; caps above 256, where it would pass 2^-14, are refused).  An
// odd polynomial of degree 11, where all of a warp's scores are within it, was slower: nine
// operations at the rate of the FMA pipe against two special-function ones (forward of 8192
// tokens, cap 50: 408 us against 309).
struct Scale { float sl2, c2, k; };
struct ScaleZ : Scale { float slope2; };

__device__ __forceinline__ ScaleZ scale_z(const Scale& s, float slope) {
  ScaleZ z;
  static_cast<Scale&>(z) = s;
  z.slope2 = slope * L2E;
  return z;
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float rcp(float a) {
  float d;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(a));
  return d;
}

// r = 1 / (1 + 2^(k s)) of two raw scores, tanh being 1 - 2 r.  The special-function unit is the
// busiest one of capped scores (55% of the forward's cycles), so the two share a reciprocal: 1 / a = b / (a b), with a and b below 2^60 (r is
// under half a step of fp32 from 0 there).  A NaN then reaches both: the two belong to one row of
// every sum they enter, but where one of them may be masked (MASK) each has its own.
template <bool MASK>
__device__ __forceinline__ float2 cap_parts(const Scale& sc, float2 s) {
  const float2 t = mul2(s, make_float2(sc.k, sc.k));
  if (MASK) {
    const float2 e = add2(make_float2(ex2(t.x), ex2(t.y)), make_float2(1.f, 1.f));
    return make_float2(rcp(e.x), rcp(e.y));
  }
  const float2 e = add2(make_float2(ex2(min_nan(t.x, 60.f)), ex2(min_nan(t.y, 60.f))), make_float2(1.f, 1.f));
  const float q = rcp(e.x * e.y);
  return make_float2(e.y * q, e.x * q);
}

inline Scale make_scale(float scale, float softcap) {
  Scale s{};
  s.sl2 = scale * L2E;
  s.c2 = softcap * L2E;
  if (softcap > 0.f) s.k = 2.f * L2E * scale / softcap;
  return s;
}

}  // namespace pk
}  // namespace tc

// O, lse of every row (sbp_attn_fwd.cu)
cudaError_t packed_forward(const PackedArgs& a, const PackedWork& w, void* O, float* lse, cudaStream_t s);

}  // namespace sbp
