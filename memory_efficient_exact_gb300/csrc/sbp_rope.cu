// Rotary positions with several axes on a token-major projection, given out head-major, and
// the gradient on the way back (bf16, sm_103a).
//
// Pair p of a head's first rot_dim elements turns by the angle pos[axis(p)][t] f_p.  The
// angle is kept as a fraction of a full turn in 64-bit fixed point, F_p = 2^64 f_p / (2 pi):
// pos F_p wraps modulo 2^64 exactly as the angle wraps modulo 2 pi, so far positions lose
// nothing (an fp32 angle at position 10^6 is off by 0.03), and the cosine and sine come from
// the top 32 bits of the product, in half turns.
//
// Bound by device memory: every element is read and written once, 16 bytes at a time.  A
// block takes TB tokens: their cosines and sines once into shared memory (all heads use the
// same), then all heads; the lanes run over a head's vectors, then tokens, so that both the
// token-major and the head-major side move whole 128-byte lines.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "sbp_internal.h"

namespace sbp {
namespace {

constexpr int MAX_PAIRS = 128, MAX_AXES = 4;
constexpr int TB = 8;   // tokens of a block

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

struct Pack { uint32_t w[4]; };
__device__ __forceinline__ Pack ldp(const __nv_bfloat16* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  return Pack{{u.x, u.y, u.z, u.w}};
}
__device__ __forceinline__ Pack ldp(const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  Pack r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return r;
}
__device__ __forceinline__ void stp(__nv_bfloat16* p, const Pack& r) {
  *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
}
__device__ __forceinline__ float2 up(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
__device__ __forceinline__ uint32_t down(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// BWD: head-major gradients in, token-major gradient out, turned back.  KV32: dK and dV are
// fp32 (rounded to bf16 when they do not turn; turned in fp32).  IL: the pairs are
// neighbouring elements (2p, 2p + 1), else (p, p + rot_dim / 2).
template <bool BWD, bool KV32, bool IL>
__global__ void __launch_bounds__(256) k_rope(const __grid_constant__ RopeP p) {
  __shared__ float2 cs[TB * MAX_PAIRS];
  const int64_t t0 = (int64_t)blockIdx.x * TB;
  const int nt = (int)min((int64_t)TB, p.T - t0);
  for (int i = threadIdx.x; i < nt * p.pairs; i += blockDim.x) {
    const int tl = i / p.pairs, pr = i - tl * p.pairs;
    const int64_t pos = p.pos[p.axis[pr] * p.T + t0 + tl];
    const uint64_t turn = (uint64_t)pos * p.F[pr];
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31: in half turns
    cs[tl * p.pairs + pr] = make_float2(c, BWD ? -s : s);
  }
  __syncthreads();
  const int u = threadIdx.x % p.upr;
  const int rows = blockDim.x / p.upr;
  const int heads = p.H + 2 * p.Hkv;
  const int rot_units = p.pairs / 8;
  // the unit's two vectors: elements e0 and e1
  const bool turns = u < rot_units;
  const int e0 = turns && !IL ? 8 * u : 16 * u, e1 = turns && !IL ? 8 * u + p.pairs : 16 * u + 8;
  for (int r = threadIdx.x / p.upr; r < heads * TB; r += rows) {
    const int tl = r % TB, h = r / TB;
    if (tl >= nt) continue;
    const int64_t t = t0 + tl;
    __nv_bfloat16* tok = p.x + t * p.ld + (int64_t)h * p.hd;
    const bool isq = h < p.H, isv = h >= p.H + p.Hkv;
    const int hh = isq ? h : h - p.H - (isv ? p.Hkv : 0);
    void* side = isq ? p.q : isv ? p.v : p.k;
    const int64_t ho = ((int64_t)hh * p.T + t) * p.hd;
    float a[8], b[8];
    Pack pa, pb;
    if (BWD && KV32 && !isq) {
      const float* s = static_cast<const float*>(side) + ho;
      if (turns && !isv) {
#pragma unroll
        for (int i = 0; i < 8; ++i) { a[i] = s[e0 + i]; b[i] = s[e1 + i]; }
      } else {
        pa = ldp(s + e0);
        pb = ldp(s + e1);
      }
    } else {
      const __nv_bfloat16* s = BWD ? static_cast<const __nv_bfloat16*>(side) + ho : tok;
      pa = ldp(s + e0);
      pb = ldp(s + e1);
      if (turns && !isv) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = up(pa.w[i]), y = up(pb.w[i]);
          a[2 * i] = x.x; a[2 * i + 1] = x.y;
          b[2 * i] = y.x; b[2 * i + 1] = y.y;
        }
      }
    }
    if (turns && !isv) {
      const float2* w = cs + tl * p.pairs + 8 * u;
      float oa[8], ob[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 c = w[i];
        if (IL) {   // vector a holds pairs 8u .. 8u + 3, vector b the next four
          float* x = i < 4 ? a : b;
          float* o = i < 4 ? oa : ob;
          const int j = 2 * (i & 3);
          o[j] = x[j] * c.x - x[j + 1] * c.y;
          o[j + 1] = x[j + 1] * c.x + x[j] * c.y;
        } else {
          oa[i] = a[i] * c.x - b[i] * c.y;
          ob[i] = b[i] * c.x + a[i] * c.y;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pa.w[i] = down(oa[2 * i], oa[2 * i + 1]);
        pb.w[i] = down(ob[2 * i], ob[2 * i + 1]);
      }
    }
    __nv_bfloat16* d = BWD ? tok : static_cast<__nv_bfloat16*>(side) + ho;
    stp(d + e0, pa);
    stp(d + e1, pb);
  }
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
    double turn = std::fmod(f / 6.283185307179586476925, 1.0);   // whole turns of a step do not matter
    if (turn < 0.0) turn += 1.0;
    const double fx = std::ldexp(turn, 64);
    p.F[i] = fx >= 18446744073709551616.0 ? 0u : (uint64_t)fx;
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
  const int threads = p.upr * (256 / p.upr);
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
