// Rotary positions with several axes on a token-major projection, given out head-major, and
// the gradient on the way back (bf16, sm_103a).
//
// Pair p of a head's first rot_dim elements turns by the angle pos[axis(p)][t] f_p.  The
// angle is kept as a fraction of a full turn in 64-bit fixed point, F_p = 2^64 f_p / (2 pi):
// pos F_p wraps modulo 2^64 exactly as the angle wraps modulo 2 pi, so far positions cost no
// precision (an fp32 angle at position 10^6 is off by 0.03), and the cosine and sine come from
// the top 32 bits of the product, in half turns, rounded to fp32: 2^-25 of a turn.  F_p is within
// 2^-63 of a turn of the fp64 frequency's (turns_of), 2^-32 at the ends of int32.
//
// Bound by device memory: every element is read and written once, 16 bytes at a time.  A
// thread keeps the cosines and sines of its eight pairs of one token in registers and walks
// the heads, UNROLL of them at a time with their loads issued together; the lanes run over a
// head's vectors, then tokens, so that both the token-major and the head-major side move
// whole 128-byte lines.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "sbp_internal.h"

namespace sbp {
namespace {

constexpr int MAX_PAIRS = 128, MAX_AXES = 4;
constexpr int TB = 8;   // tokens of a block
// Heads in flight a thread.  T = 16384, 32 / 8 heads of 128: 72 us with one, 66 with two, 70 with
// four (registers); neighbouring pairs, T = 8191: 37.5, 39.6, 41.6.
constexpr int UNROLL = 2;

struct RopeP {
  uint64_t F[MAX_PAIRS];
  uint8_t axis[MAX_PAIRS];
  const int32_t* pos;        // [axes, T]
  int64_t T, ld;             // ld: row stride of the token-major side (elements)
  int H, Hkv, hd, pairs;
  int upr;                   // units (two 16-byte vectors) of a head's row
  __nv_bfloat16* x;          // token-major side
  void *q, *k, *v;           // head-major side
};

// Eight elements: bf16 as they lie in memory, or fp32.
struct V16 {
  uint4 u;
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at);
  }
  __device__ __forceinline__ void f(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
struct V32 {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    a = q[0];
    b = q[1];
  }
  __device__ __forceinline__ void f(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Heads h0, h0 + step, ... below h1 of one token: elements e0 .. e0+7 and e1 .. e1+7 of each.
// The token-major row is tok + h hd, the head-major one side + (h - hbase) T hd.
template <bool BWD, bool IL, typename V>
__device__ __forceinline__ void walk(const RopeP& p, int h0, int h1, int step, __nv_bfloat16* tok, void* side, int hbase,
                                     int64_t t, int e0, int e1, bool turns, const float (&cs)[8], const float (&sn)[8]) {
  for (int h = h0; h < h1; h += UNROLL * step) {
    V va[UNROLL], vb[UNROLL];
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      const int hk = h + k * step;
      if (hk < h1) {
        const int64_t at = BWD ? ((int64_t)(hk - hbase) * p.T + t) * p.hd : (int64_t)hk * p.hd;
        va[k].load(BWD ? side : tok, at + e0);
        vb[k].load(BWD ? side : tok, at + e1);
      }
    }
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      const int hk = h + k * step;
      if (hk < h1) {
        float a[8], b[8];
        va[k].f(a);
        vb[k].f(b);
        if (turns) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float &x = IL ? (i < 4 ? a[2 * (i & 3)] : b[2 * (i & 3)]) : a[i];   // pairs 8u + i: neighbours (four in
            float &y = IL ? (i < 4 ? a[2 * (i & 3) + 1] : b[2 * (i & 3) + 1]) : b[i];   // each vector), or halves
            const float n = x * cs[i] - y * sn[i];
            y = y * cs[i] + x * sn[i];
            x = n;
          }
        }
        __nv_bfloat16* d = BWD ? tok + (int64_t)hk * p.hd
                               : static_cast<__nv_bfloat16*>(side) + ((int64_t)(hk - hbase) * p.T + t) * p.hd;
        store(d + e0, a);
        store(d + e1, b);
      }
    }
  }
}

// BWD: head-major gradients in, token-major gradient out, turned back.  KV32: dK and dV are
// fp32.  IL: the pairs are neighbouring elements (2p, 2p + 1), else (p, p + rot_dim / 2).
template <bool BWD, bool KV32, bool IL>
__global__ void __launch_bounds__(256) k_rope(const __grid_constant__ RopeP p) {
  const int u = threadIdx.x % p.upr, r = threadIdx.x / p.upr;
  const int tl = r % TB, hg = r / TB, groups = blockDim.x / (p.upr * TB);
  const int64_t t = (int64_t)blockIdx.x * TB + tl;
  if (t >= p.T || hg >= groups) return;
  // the unit's two vectors: elements e0 and e1
  const bool turns = 8 * u < p.pairs;
  const int e0 = turns && !IL ? 8 * u : 16 * u, e1 = turns && !IL ? 8 * u + p.pairs : 16 * u + 8;
  float cs[8], sn[8];
  if (turns) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t pos = p.pos[p.axis[8 * u + i] * p.T + t];
      const uint64_t turn = (uint64_t)pos * p.F[8 * u + i];
      sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &sn[i], &cs[i]);   // 2^-31: in half turns
      if (BWD) sn[i] = -sn[i];
    }
  }
  using KV = typename std::conditional<KV32, V32, V16>::type;
  __nv_bfloat16* tok = p.x + t * p.ld;
  const int k0 = p.H, v0 = p.H + p.Hkv, v1 = p.H + 2 * p.Hkv;
  walk<BWD, IL, V16>(p, hg, k0, groups, tok, p.q, 0, t, e0, e1, turns, cs, sn);
  walk<BWD, IL, KV>(p, k0 + hg, v0, groups, tok, p.k, k0, t, e0, e1, turns, cs, sn);
  walk<BWD, IL, KV>(p, v0 + hg, v1, groups, tok, p.v, v0, t, e0, e1, false, cs, sn);
}

// f / (2 pi) less its whole part, in 2^-64 of a turn.  Whole turns of a step do not matter, and
// they take bits: 1 / (2 pi) is two fp64 values, the product's rounding is kept (fma), and the whole
// part leaves exactly, which makes the rest good to 2^-63 for |f| up to 2^40.  (With one product in
// fp64 a frequency of 10^6 was off by 0.05 turns at position 2^31.)
constexpr double MAX_FREQ = 1099511627776.0;   // 2^40
uint64_t turns_of(double f) {
  constexpr double C1 = 0x1.45f306dc9c883p-3, C2 = -0x1.6b01ec5417056p-57;   // 1 / (2 pi) = C1 + C2
  const double a = std::fabs(f), hi = a * C1, lo = std::fma(a, C1, -hi) + a * C2;
  const uint64_t t = (uint64_t)((hi - std::floor(hi)) * 18446744073709551616.0) +
                     (uint64_t)(int64_t)std::floor(lo * 18446744073709551616.0);
  return f < 0 ? 0u - t : t;
}

struct RopeArgs {
  const int32_t* pos; int32_t n_axes; const int32_t* sections; const double* inv_freq; double theta;
  int64_t rot_dim; int interleaved;
  int64_t T, H, Hkv, hd, ld;
  void *x, *q, *k, *v;
  int kv_dtype;
};

int run_rope(const RopeArgs& a, bool bwd, cudaStream_t s) {
  if (a.T < 0 || a.H < 1 || a.Hkv < 0 || a.hd < 1 || a.rot_dim < 0 || a.rot_dim > a.hd || a.n_axes < 1 ||
      !a.sections || (a.interleaved != 0 && a.interleaved != 1) || (a.kv_dtype != SBP_BF16 && a.kv_dtype != SBP_FP32))
    return SBP_ERR_INVALID_ARG;
  const int64_t heads = a.H + 2 * a.Hkv;
  if (a.ld < heads * a.hd) return SBP_ERR_INVALID_ARG;
  if (a.hd % 16 != 0 || a.hd > 256 || a.rot_dim % 16 != 0 || a.n_axes > MAX_AXES || a.ld % 8 != 0 ||
      heads > 1 << 20 || a.T > (int64_t)1 << 31)
    return SBP_ERR_UNSUPPORTED;
  RopeP p;
  p.pairs = (int)(a.rot_dim / 2);
  int64_t n = 0;
  for (int i = 0; i < a.n_axes; ++i) {
    if (a.sections[i] < 0 || (n += a.sections[i]) > p.pairs) return SBP_ERR_INVALID_ARG;
    for (int64_t k = n - a.sections[i]; k < n; ++k) p.axis[k] = (uint8_t)i;
  }
  if (n != p.pairs) return SBP_ERR_INVALID_ARG;
  if (!a.inv_freq && p.pairs > 0 && (!(a.theta > 0.0) || std::isinf(a.theta))) return SBP_ERR_INVALID_ARG;
  for (int i = 0; i < p.pairs; ++i) {
    const double f = a.inv_freq ? a.inv_freq[i] : std::pow(a.theta, -2.0 * i / (double)a.rot_dim);
    if (std::isnan(f) || std::isinf(f)) return SBP_ERR_INVALID_ARG;
    if (std::fabs(f) > MAX_FREQ) return SBP_ERR_UNSUPPORTED;
    p.F[i] = turns_of(f);
  }
  if (a.T > 0 && (!a.pos || !a.x || !a.q || (a.Hkv > 0 && (!a.k || !a.v)))) return SBP_ERR_INVALID_ARG;
  for (const void* q : {(const void*)a.x, (const void*)a.q, (const void*)a.k, (const void*)a.v})
    if (!aligned16(q)) return SBP_ERR_ALIGNMENT;
  if (reinterpret_cast<uintptr_t>(a.pos) & 3u) return SBP_ERR_ALIGNMENT;
  set_launch_count(0);
  if (a.T == 0) return SBP_OK;
  p.pos = a.pos; p.T = a.T; p.ld = a.ld; p.H = (int)a.H; p.Hkv = (int)a.Hkv; p.hd = (int)a.hd;
  p.upr = (int)(a.hd / 16);
  p.x = static_cast<__nv_bfloat16*>(a.x);
  p.q = a.q; p.k = a.k; p.v = a.v;
  const unsigned grid = (unsigned)((a.T + TB - 1) / TB);
  // whole heads' rows of TB tokens, as many head groups as fit in 256 threads
  const int threads = p.upr * TB * std::max(1, 256 / (p.upr * TB));
  const bool kv32 = bwd && a.kv_dtype == SBP_FP32;
  if (!bwd) {
    if (a.interleaved) k_rope<false, false, true><<<grid, threads, 0, s>>>(p);
    else k_rope<false, false, false><<<grid, threads, 0, s>>>(p);
  } else if (kv32) {
    if (a.interleaved) k_rope<true, true, true><<<grid, threads, 0, s>>>(p);
    else k_rope<true, true, false><<<grid, threads, 0, s>>>(p);
  } else {
    if (a.interleaved) k_rope<true, false, true><<<grid, threads, 0, s>>>(p);
    else k_rope<true, false, false><<<grid, threads, 0, s>>>(p);
  }
  if (cudaGetLastError() != cudaSuccess) return SBP_ERR_CUDA;
  set_launch_count(1);
  return SBP_OK;
}

}  // namespace
}  // namespace sbp

using namespace sbp;

extern "C" {

int sbp_rope_qkv_forward(const void* qkv, int64_t row_stride, const int32_t* positions, int32_t n_axes,
                         const int32_t* sections, const double* inv_freq, double theta, int64_t rot_dim,
                         int interleaved, int64_t T, int64_t H, int64_t Hkv, int64_t hd, void* Q, void* K, void* V,
                         void* stream) {
  NvtxRange nv("sbp_rope_qkv_forward");
  return run_rope({positions, n_axes, sections, inv_freq, theta, rot_dim, interleaved, T, H, Hkv, hd, row_stride,
                   const_cast<void*>(qkv), Q, K, V, SBP_BF16}, false, static_cast<cudaStream_t>(stream));
}

int sbp_rope_qkv_backward(const void* dQ, const void* dK, const void* dV, int kv_dtype, const int32_t* positions,
                          int32_t n_axes, const int32_t* sections, const double* inv_freq, double theta,
                          int64_t rot_dim, int interleaved, int64_t T, int64_t H, int64_t Hkv, int64_t hd,
                          void* dqkv, int64_t row_stride, void* stream) {
  NvtxRange nv("sbp_rope_qkv_backward");
  return run_rope({positions, n_axes, sections, inv_freq, theta, rot_dim, interleaved, T, H, Hkv, hd, row_stride, dqkv,
                   const_cast<void*>(dQ), const_cast<void*>(dK), const_cast<void*>(dV), kv_dtype}, true,
                  static_cast<cudaStream_t>(stream));
}

}  // extern "C"
