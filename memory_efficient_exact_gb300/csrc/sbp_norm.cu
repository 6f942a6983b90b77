// Root-mean-square norm with the residual's addition, forward and backward, and its output
// in 8 bits (sm_103a).
//
//   R = X + residual,  rstd = 1 / sqrt(mean(R^2) + eps),  Y = R rstd gamma
//   g = dY gamma,  dX = rstd (g - R (rstd^2 / d) sum(g R)) + dR,  dgamma = sum_t dY R rstd
//
// All three kernels are bound by device memory: each row is read once into registers (16
// bytes a load, every load of the row issued before the first sum), reduced by its WPR
// warps, and written once.  A block holds several rows of few warps, or one row of many.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "sbp_internal.h"

namespace sbp {
namespace {

constexpr int MAXW = 32;            // warps of a block
constexpr int64_t MAX_D = 16384;    // 32 warps x 32 lanes x 2 vectors x 8 elements

// Eight elements of a row.
struct F8 { float v[8]; };
__device__ __forceinline__ F8 load8(const __nv_bfloat16* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    f.v[2 * i] = x.x;
    f.v[2 * i + 1] = x.y;
  }
  return f;
}
__device__ __forceinline__ F8 load8(const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const F8& f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.v[2 * i], f.v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const F8& f) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f.v[0], f.v[1], f.v[2], f.v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f.v[4], f.v[5], f.v[6], f.v[7]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the wpr warps of this warp's row.  Every warp of the block calls it; the slots of
// two calls in a row are different (flip), so one barrier a call is enough.
__device__ __forceinline__ float row_sum(float v, float (*red)[MAXW], int flip, int wpr) {
  v = warp_sum(v);
  if (wpr == 1) return v;
  const int warp = threadIdx.x / 32;
  if (threadIdx.x % 32 == 0) red[flip][warp] = v;
  __syncthreads();
  const int w0 = warp / wpr * wpr;
  float s = 0.f;
  for (int i = 0; i < wpr; ++i) s += red[flip][w0 + i];
  return s;
}

struct FwdP {
  const void *X, *res, *gamma;
  int64_t T;
  int d, nvec, wpr, rpb;   // 8-element vectors and warps of a row, rows of a block
  float eps;
  void *R, *Y;
  float* scales;   // 8-bit output: [T, nblk]
  int nblk;
};

// E: bf16 or fp32.  NV vectors a thread.  Q8: Y in e4m3 with a scale for each 128 columns,
// the 128 columns of a block being 16 neighbouring lanes of one warp and vector.
template <typename E, int NV, bool Q8>
__global__ void __launch_bounds__(1024) k_rmsnorm_fwd(const FwdP p) {
  __shared__ float red[2][MAXW];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int sub = warp / p.wpr;                                  // row of the block
  const int t0 = (warp - sub * p.wpr) * 32 + lane;               // thread of the row
  const int64_t row = (int64_t)blockIdx.x * p.rpb + sub;
  const bool live = row < p.T;
  const int step = 32 * p.wpr;
  const int64_t at = row * p.d;
  F8 r[NV];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t0 + i * step;
    if (live && v < p.nvec) {
      r[i] = load8(static_cast<const E*>(p.X) + at + 8 * v);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) r[i].v[k] = 0.f;
    }
  }
  if (p.res) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t0 + i * step;
      if (live && v < p.nvec) {
        const F8 q = load8(static_cast<const E*>(p.res) + at + 8 * v);
#pragma unroll
        for (int k = 0; k < 8; ++k) r[i].v[k] += q.v[k];
        if (p.R) store8(static_cast<E*>(p.R) + at + 8 * v, r[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(r[i].v[k], r[i].v[k], ss);
  ss = row_sum(ss, red, 0, p.wpr);
  const float rstd = 1.f / sqrtf(ss / (float)p.d + p.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t0 + i * step;
    const bool in = live && v < p.nvec;
    if (in) {
      const F8 g = load8(static_cast<const E*>(p.gamma) + 8 * v);
#pragma unroll
      for (int k = 0; k < 8; ++k) r[i].v[k] = r[i].v[k] * rstd * g.v[k];
    }
    if constexpr (!Q8) {
      if (in) store8(static_cast<E*>(p.Y) + at + 8 * v, r[i]);
    } else {
      float a = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) a = fmaxf(a, fabsf(r[i].v[k]));
#pragma unroll
      for (int o = 8; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      // 448: e4m3's largest value.  A block of zeros keeps the scale 1.
      const float s = a > 0.f ? a / 448.f : 1.f;
      if (in) {
        uint32_t w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(r[i].v[4 * k] / s, r[i].v[4 * k + 1] / s),
                                                       __NV_SATFINITE, __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(r[i].v[4 * k + 2] / s, r[i].v[4 * k + 3] / s),
                                                       __NV_SATFINITE, __NV_E4M3);
          w[k] = lo | (hi << 16);
        }
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.Y) + at + 8 * v) = make_uint2(w[0], w[1]);
        if (lane % 16 == 0) p.scales[row * p.nblk + v / 16] = s;
      }
    }
  }
}

struct BwdP {
  const void *dY, *R, *gamma, *dR;
  int64_t T;
  int d, nvec, wpr, rpb;
  float eps;
  void* dX;
  float* part;   // [gridDim.x * rpb, d]: each row group's share of dgamma
};

// A block walks rows blockIdx.x * rpb + k gridDim.x * rpb; each row group keeps its share of
// dgamma in registers and leaves it in `part` (summed in a fixed order by k_dgamma).
// MAXT: the most threads of a block, which sets the registers a thread may have.
template <typename E, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) k_rmsnorm_bwd(const BwdP p) {
  __shared__ float red[4][MAXW];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int sub = warp / p.wpr;
  const int t0 = (warp - sub * p.wpr) * 32 + lane;
  const int step = 32 * p.wpr;
  F8 dg[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) dg[i].v[k] = 0.f;
  int flip = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * p.rpb; r0 < p.T; r0 += (int64_t)gridDim.x * p.rpb) {
    const int64_t row = r0 + sub;
    const bool live = row < p.T;
    const int64_t at = row * p.d;
    F8 r[NV], y[NV];
    float ss = 0.f, gr = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t0 + i * step;
      if (live && v < p.nvec) {
        r[i] = load8(static_cast<const E*>(p.R) + at + 8 * v);
        y[i] = load8(static_cast<const E*>(p.dY) + at + 8 * v);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) r[i].v[k] = y[i].v[k] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t0 + i * step;
      F8 g;
      if (v < p.nvec) g = load8(static_cast<const E*>(p.gamma) + 8 * v);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        ss = fmaf(r[i].v[k], r[i].v[k], ss);
        if (v < p.nvec) gr = fmaf(y[i].v[k] * g.v[k], r[i].v[k], gr);
      }
    }
    ss = row_sum(ss, red, flip, p.wpr);
    gr = row_sum(gr, red, flip + 1, p.wpr);
    flip ^= 2;
    const float rstd = 1.f / sqrtf(ss / (float)p.d + p.eps);
    const float c = rstd * rstd * (gr / (float)p.d);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t0 + i * step;
      if (live && v < p.nvec) {
        const F8 g = load8(static_cast<const E*>(p.gamma) + 8 * v);
        F8 o;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          dg[i].v[k] = fmaf(y[i].v[k], r[i].v[k] * rstd, dg[i].v[k]);
          o.v[k] = rstd * (y[i].v[k] * g.v[k] - r[i].v[k] * c);
        }
        if (p.dR) {
          const F8 q = load8(static_cast<const E*>(p.dR) + at + 8 * v);
#pragma unroll
          for (int k = 0; k < 8; ++k) o.v[k] += q.v[k];
        }
        store8(static_cast<E*>(p.dX) + at + 8 * v, o);
      }
    }
  }
  float* part = p.part + ((int64_t)blockIdx.x * p.rpb + sub) * p.d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t0 + i * step;
    if (v < p.nvec) store8(part + 8 * v, dg[i]);
  }
}

// dgamma[c] (+)= sum over the n parts, 32 columns a block, 32 threads a column.
__global__ void __launch_bounds__(1024) k_dgamma(const float* __restrict__ part, int n, int d, int accumulate,
                                                 float* __restrict__ out) {
  __shared__ float s[32][33];
  const int cx = threadIdx.x % 32, py = threadIdx.x / 32, c = blockIdx.x * 32 + cx;
  float a = 0.f;
  if (c < d)
    for (int i = py; i < n; i += 32) a += part[(int64_t)i * d + c];
  s[py][cx] = a;
  __syncthreads();
  const float v = warp_sum(s[cx][py]);   // warp py sums column py
  const int oc = blockIdx.x * 32 + py;
  if (cx == 0 && oc < d) out[oc] = accumulate ? out[oc] + v : v;
}

// Y = q * scale, eight elements a thread.
template <typename O>
__global__ void __launch_bounds__(256) k_e4m3_expand(const uint8_t* __restrict__ q, const float* __restrict__ scales,
                                                     int64_t n, int d, int nblk, O* __restrict__ out) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  const int64_t row = i / d;
  const float s = scales[row * nblk + (int)(i - row * d) / 128];
  const uint2 u = *reinterpret_cast<const uint2*>(q + i);
  const uint32_t w[2] = {u.x, u.y};
  F8 f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[k / 2] >> (16 * (k % 2))), __NV_E4M3);
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f.v[2 * k] = x.x * s;
    f.v[2 * k + 1] = x.y * s;
  }
  store8(out + i, f);
}

// Rows in a block: NV vectors a thread, whole warps a row, up to 8 warps' worth of rows
// together.
struct Shape { int nv, wpr, rpb, threads; };
Shape shape_of(int64_t d) {
  const int nvec = (int)(d / 8);
  Shape s;
  s.nv = nvec <= 32 ? 1 : 2;
  s.wpr = (nvec + 32 * s.nv - 1) / (32 * s.nv);
  s.rpb = std::max(1, 8 / s.wpr);
  s.threads = 32 * s.wpr * s.rpb;
  return s;
}

int norm_check(int64_t T, int64_t d, int dtype) {
  if (T < 0 || d < 1 || (dtype != SBP_BF16 && dtype != SBP_FP32)) return SBP_ERR_INVALID_ARG;
  if (d % 8 != 0 || d > MAX_D || T > (int64_t)1 << 31) return SBP_ERR_UNSUPPORTED;
  return SBP_OK;
}

template <typename E, bool Q8>
cudaError_t launch_fwd(const FwdP& p, const Shape& s, cudaStream_t st) {
  const unsigned grid = (unsigned)((p.T + s.rpb - 1) / s.rpb);
  if (s.nv == 1) k_rmsnorm_fwd<E, 1, Q8><<<grid, s.threads, 0, st>>>(p);
  else k_rmsnorm_fwd<E, 2, Q8><<<grid, s.threads, 0, st>>>(p);
  return cudaGetLastError();
}

int run_fwd(const void* X, const void* res, const void* gamma, int64_t T, int64_t d, float eps, int dtype, void* R,
            void* Y, float* scales, bool q8, cudaStream_t s) {
  const int rc = norm_check(T, d, dtype);
  if (rc != SBP_OK) return rc;
  if (!(eps >= 0.f) || std::isinf(eps)) return SBP_ERR_INVALID_ARG;
  if (T > 0 && (!X || !gamma || !Y || (q8 && !scales) || (!res && R))) return SBP_ERR_INVALID_ARG;
  for (const void* q : {X, res, gamma, (const void*)R, (const void*)Y})
    if (!aligned16(q)) return SBP_ERR_ALIGNMENT;
  if (reinterpret_cast<uintptr_t>(scales) & 3u) return SBP_ERR_ALIGNMENT;
  set_launch_count(0);
  if (T == 0) return SBP_OK;
  const Shape sh = shape_of(d);
  FwdP p{X, res, gamma, T, (int)d, (int)(d / 8), sh.wpr, sh.rpb, eps, R, Y, scales, (int)((d + 127) / 128)};
  cudaError_t e;
  if (dtype == SBP_BF16)
    e = q8 ? launch_fwd<__nv_bfloat16, true>(p, sh, s) : launch_fwd<__nv_bfloat16, false>(p, sh, s);
  else
    e = q8 ? launch_fwd<float, true>(p, sh, s) : launch_fwd<float, false>(p, sh, s);
  if (e != cudaSuccess) return SBP_ERR_CUDA;
  set_launch_count(1);
  return SBP_OK;
}

// Blocks of the backward: all that fit at once, so that each walks the same number of rows.
int64_t bwd_blocks(int64_t T, const Shape& s) {
  const int per_sm = std::max(1, std::min(4, 1024 / s.threads));
  return std::max<int64_t>(1, std::min<int64_t>((T + s.rpb - 1) / s.rpb, (int64_t)num_sms() * per_sm));
}

struct BwdLayout {
  size_t off_part = 0, total = 0;
  int64_t blocks = 0;
  Guards guards;   // checked build only
};
bool bwd_layout(int64_t T, int64_t d, int dtype, BwdLayout* L) {
  if (norm_check(T, d, dtype) != SBP_OK) return false;
  BwdLayout l;
  const Shape s = shape_of(d);
  l.blocks = bwd_blocks(T, s);
  size_t o = 0;
  l.off_part = take_region(o, (size_t)l.blocks * s.rpb * d * sizeof(float), l.guards);
  l.total = o;
  *L = l;
  return true;
}

template <typename E>
cudaError_t launch_bwd(const BwdP& p, const Shape& s, unsigned grid, cudaStream_t st) {
  if (s.nv == 1) k_rmsnorm_bwd<E, 1, 512><<<grid, s.threads, 0, st>>>(p);
  else if (s.threads <= 512) k_rmsnorm_bwd<E, 2, 512><<<grid, s.threads, 0, st>>>(p);
  else k_rmsnorm_bwd<E, 2, 1024><<<grid, s.threads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace sbp

using namespace sbp;

extern "C" {

int sbp_rmsnorm_forward(const void* X, const void* residual, const void* gamma, int64_t T, int64_t d, float eps,
                        int dtype, void* R, void* Y, void* stream) {
  NvtxRange nv("sbp_rmsnorm_forward");
  return run_fwd(X, residual, gamma, T, d, eps, dtype, R, Y, nullptr, false, static_cast<cudaStream_t>(stream));
}

int sbp_rmsnorm_forward_e4m3(const void* X, const void* residual, const void* gamma, int64_t T, int64_t d, float eps,
                             int dtype, void* R, void* Y8, float* scales, void* stream) {
  NvtxRange nv("sbp_rmsnorm_forward_e4m3");
  return run_fwd(X, residual, gamma, T, d, eps, dtype, R, Y8, scales, true, static_cast<cudaStream_t>(stream));
}

int sbp_e4m3_expand(const void* Y8, const float* scales, int64_t T, int64_t d, int dtype, void* Y, void* stream) {
  const int rc = norm_check(T, d, dtype);
  if (rc != SBP_OK) return rc;
  if (T > 0 && (!Y8 || !scales || !Y)) return SBP_ERR_INVALID_ARG;
  if (!aligned16(Y8) || !aligned16(Y) || (reinterpret_cast<uintptr_t>(scales) & 3u)) return SBP_ERR_ALIGNMENT;
  NvtxRange nv("sbp_e4m3_expand");
  set_launch_count(0);
  if (T == 0) return SBP_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t n = T * d, blocks = (n / 8 + 255) / 256;
  if (blocks > INT32_MAX) return SBP_ERR_UNSUPPORTED;
  const int nblk = (int)((d + 127) / 128);
  if (dtype == SBP_BF16)
    k_e4m3_expand<<<(unsigned)blocks, 256, 0, s>>>(static_cast<const uint8_t*>(Y8), scales, n, (int)d, nblk,
                                                   static_cast<__nv_bfloat16*>(Y));
  else
    k_e4m3_expand<<<(unsigned)blocks, 256, 0, s>>>(static_cast<const uint8_t*>(Y8), scales, n, (int)d, nblk,
                                                   static_cast<float*>(Y));
  if (cudaGetLastError() != cudaSuccess) return SBP_ERR_CUDA;
  set_launch_count(1);
  return SBP_OK;
}

size_t sbp_rmsnorm_backward_workspace_bytes(int64_t T, int64_t d, int dtype) {
  BwdLayout L;
  return bwd_layout(T, d, dtype, &L) ? L.total : 0;
}

int sbp_rmsnorm_backward(const void* dY, const void* R, const void* gamma, const void* dR, int64_t T, int64_t d,
                         float eps, int dtype, void* dX, float* dgamma, int accumulate, void* workspace,
                         size_t ws_bytes, int32_t* dev_status, void* stream) {
  const int rc = norm_check(T, d, dtype);
  if (rc != SBP_OK) return rc;
  BwdLayout L;
  if (!bwd_layout(T, d, dtype, &L)) return SBP_ERR_UNSUPPORTED;
  if (!(eps >= 0.f) || std::isinf(eps) || !dgamma || !dev_status) return SBP_ERR_INVALID_ARG;
  if (T > 0 && (!dY || !R || !gamma || !dX)) return SBP_ERR_INVALID_ARG;
  for (const void* q : {dY, R, gamma, dR, (const void*)dX, (const void*)dgamma})
    if (!aligned16(q)) return SBP_ERR_ALIGNMENT;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || ws_bytes < L.total) return SBP_ERR_WORKSPACE;
  NvtxRange nv("sbp_rmsnorm_backward");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) != cudaSuccess) return SBP_ERR_CUDA;
  if (T == 0) {
    set_launch_count(0);
    if (!accumulate && cudaMemsetAsync(dgamma, 0, (size_t)d * sizeof(float), s) != cudaSuccess) return SBP_ERR_CUDA;
    return SBP_OK;
  }
  char* w = static_cast<char*>(workspace);
  int launches = 2;
  int st = workspace_guards(w, L.guards, 0, dev_status, s, &launches);
  if (st != SBP_OK) return st;
  const Shape sh = shape_of(d);
  float* part = reinterpret_cast<float*>(w + L.off_part);
  BwdP p{dY, R, gamma, dR, T, (int)d, (int)(d / 8), sh.wpr, sh.rpb, eps, dX, part};
  const cudaError_t e = dtype == SBP_BF16 ? launch_bwd<__nv_bfloat16>(p, sh, (unsigned)L.blocks, s)
                                          : launch_bwd<float>(p, sh, (unsigned)L.blocks, s);
  if (e != cudaSuccess) return SBP_ERR_CUDA;
  k_dgamma<<<(unsigned)((d + 31) / 32), 1024, 0, s>>>(part, (int)(L.blocks * sh.rpb), (int)d, accumulate ? 1 : 0,
                                                      dgamma);
  if (cudaGetLastError() != cudaSuccess) return SBP_ERR_CUDA;
  st = workspace_guards(w, L.guards, 1, dev_status, s, &launches);
  if (st == SBP_OK) set_launch_count(launches);
  return st;
}

}  // extern "C"
