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

#include "sbp_tc_common.cuh"

namespace sbp {
namespace {

constexpr int MAXW = 32;            // warps of a block
constexpr int64_t MAX_D = 16384;    // 32 warps x 32 lanes x 2 vectors x 8 elements

// Eight elements of a row: as they lie in memory (16 or 32 bytes) and in fp32.
struct F8 { float v[8]; };
template <typename E> struct Raw;
template <> struct Raw<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ F8 f() const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    F8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f.v[2 * i] = __uint_as_float(w[i] << 16);
      f.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    return f;
  }
};
template <> struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ F8 f() const { return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}}; }
};
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

// Sums of two values over the lanes of this row: lpr lanes of one warp, or wpr whole warps.
// Every warp of the block calls it; two calls in a row use different slots (flip), so one
// barrier a call is enough.
__device__ __forceinline__ float2 row_sums(float2 v, float2 (*red)[MAXW], int flip, int lpr, int wpr) {
  for (int o = lpr / 2; o; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if (wpr == 1) return v;
  const int warp = threadIdx.x / 32;
  if (threadIdx.x % 32 == 0) red[flip][warp] = v;
  __syncthreads();
  const int w0 = warp / wpr * wpr;
  float2 s = make_float2(0.f, 0.f);
  for (int i = 0; i < wpr; ++i) {
    s.x += red[flip][w0 + i].x;
    s.y += red[flip][w0 + i].y;
  }
  return s;
}

struct FwdP {
  const void *X, *res, *gamma;
  int64_t T;
  int d, nvec, lpr, wpr, rpb;   // 8-element vectors, lanes and warps of a row, rows of a block
  float eps;
  void *R, *Y;
  float* scales;   // 8-bit output: [T, nblk]
  int nblk;
};

// E: bf16 or fp32.  NV vectors a thread.  Q8: Y in e4m3 with a scale for each 128 columns,
// the 128 columns of a block being 16 neighbouring lanes (or all the row's, if it is
// narrower) of one warp and vector.
// Blocks walk the rows; the next row's loads are issued before this row's sum, so that a block
// always has a row in flight, and the grid is what the SMs hold at once (T = 16384, d = 4096:
// 79 us, 6840 GB/s; with a third more blocks than that 91 us).
template <typename E, int NV, bool Q8, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k_rmsnorm_fwd(const FwdP p) {
  __shared__ float2 red[2][MAXW];
  const int step = p.lpr * p.wpr;               // threads of a row
  const int sub = threadIdx.x / step;           // row of the block
  const int t0 = threadIdx.x - sub * step;      // thread of the row
  const float inv_d = 1.f / (float)p.d;
  Raw<E> x[NV], q[NV], g[NV];
  auto fetch = [&](int64_t row) {
    const int nvec = row < p.T ? p.nvec : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t0 + i * step;
      x[i].zero();
      q[i].zero();
      if (v < nvec) {
        const int64_t at = row * p.d + 8 * v;
        x[i].load(static_cast<const E*>(p.X) + at);
        if (p.res) q[i].load(static_cast<const E*>(p.res) + at);
      }
    }
  };
  fetch((int64_t)blockIdx.x * p.rpb + sub);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t0 + i * step;
    if (v < p.nvec) g[i].load(static_cast<const E*>(p.gamma) + 8 * v);
    else g[i].zero();
  }
  int flip = 0;
  const int64_t stride = (int64_t)gridDim.x * p.rpb;
  for (int64_t r0 = (int64_t)blockIdx.x * p.rpb; r0 < p.T; r0 += stride) {
    const int64_t row = r0 + sub;
    const int nvec = row < p.T ? p.nvec : 0;
    const int64_t at = row * p.d;
    F8 r[NV];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      r[i] = x[i].f();
      const F8 a = q[i].f();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        r[i].v[k] += a.v[k];
        ss = fmaf(r[i].v[k], r[i].v[k], ss);
      }
    }
    fetch(row + stride);
    if (p.R) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = t0 + i * step;
        if (v < nvec) store8(static_cast<E*>(p.R) + at + 8 * v, r[i]);
      }
    }
    const float rstd = rsqrtf(row_sums(make_float2(ss, 0.f), red, flip, p.lpr, p.wpr).x * inv_d + p.eps);
    flip ^= 1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t0 + i * step;
      const F8 w = g[i].f();
#pragma unroll
      for (int k = 0; k < 8; ++k) r[i].v[k] = r[i].v[k] * rstd * w.v[k];
      if constexpr (!Q8) {
        if (v < nvec) store8(static_cast<E*>(p.Y) + at + 8 * v, r[i]);
      } else {
        float a = 0.f;
        if (v < nvec) {
#pragma unroll
          for (int k = 0; k < 8; ++k) a = fmaxf(a, fabsf(r[i].v[k]));
        }
        for (int o = min(8, p.lpr / 2); o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        // 448: e4m3's largest value.  A block of zeros keeps the scale 1; a scale that is not
        // normal would have no inverse.  One division a
        // block and products instead of a division an element (132 us against 87).
        const float s = a > 0.f ? fmaxf(a / 448.f, 1.17549435e-38f) : 1.f, inv = 1.f / s;
        if (v < nvec) {
          uint32_t w2[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(r[i].v[4 * k] * inv, r[i].v[4 * k + 1] * inv),
                                                         __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(r[i].v[4 * k + 2] * inv, r[i].v[4 * k + 3] * inv),
                                                         __NV_SATFINITE, __NV_E4M3);
            w2[k] = lo | (hi << 16);
          }
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.Y) + at + 8 * v) = make_uint2(w2[0], w2[1]);
          if (v % 16 == 0) p.scales[row * p.nblk + v / 16] = s;
        }
      }
    }
  }
}

struct BwdP {
  const void *dY, *R, *gamma, *dR;
  int64_t T;
  int d, nvec, lpr, wpr, rpb;
  float eps;
  void* dX;
  float* part;   // [gridDim.x, d]: each block's share of dgamma
};

// A block walks rows blockIdx.x * rpb + k gridDim.x * rpb, keeps its share of dgamma in
// registers and leaves it in `part` (summed in a fixed order by k_dgamma).  The
// next row's loads are issued before this row's sums, which hide them: without that a block
// waited for memory and for its barriers in turn (T = 16384, d = 4096: 235 us, 92 with).
// MAXT: the most threads of a block, MINB: how many blocks of it an SM should hold, which set
// the registers a thread may have.
template <typename E, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k_rmsnorm_bwd(const BwdP p) {
  constexpr bool AHEAD = MAXT <= 512;   // a block of 1024 threads has no registers for it
  __shared__ float2 red[2][MAXW];
  const int step = p.lpr * p.wpr;               // threads of a row
  const int sub = threadIdx.x / step;           // row of the block
  const int t0 = threadIdx.x - sub * step;      // thread of the row
  const float inv_d = 1.f / (float)p.d;
  F8 dg[NV];
  Raw<E> g[NV], r[NV], y[NV], q[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t0 + i * step;
    if (v < p.nvec) g[i].load(static_cast<const E*>(p.gamma) + 8 * v);
    else g[i].zero();
#pragma unroll
    for (int k = 0; k < 8; ++k) dg[i].v[k] = 0.f;
  }
  auto fetch = [&](int64_t row) {
    const int nvec = row < p.T ? p.nvec : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t0 + i * step;
      r[i].zero();
      y[i].zero();
      q[i].zero();
      if (v < nvec) {
        const int64_t at = row * p.d + 8 * v;
        r[i].load(static_cast<const E*>(p.R) + at);
        y[i].load(static_cast<const E*>(p.dY) + at);
        if (p.dR) q[i].load(static_cast<const E*>(p.dR) + at);
      }
    }
  };
  int flip = 0;
  const int64_t stride = (int64_t)gridDim.x * p.rpb;
  if (AHEAD) fetch((int64_t)blockIdx.x * p.rpb + sub);
  for (int64_t r0 = (int64_t)blockIdx.x * p.rpb; r0 < p.T; r0 += stride) {
    const int64_t row = r0 + sub;
    const int nvec = row < p.T ? p.nvec : 0;
    if (!AHEAD) fetch(row);
    Raw<E> cr[NV], cy[NV], cq[NV];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      cr[i] = r[i];
      cy[i] = y[i];
      cq[i] = q[i];
      const F8 a = cr[i].f(), b = cy[i].f(), c = g[i].f();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s.x = fmaf(a.v[k], a.v[k], s.x);
        s.y = fmaf(b.v[k] * c.v[k], a.v[k], s.y);
      }
    }
    if (AHEAD) fetch(row + stride);
    s = row_sums(s, red, flip, p.lpr, p.wpr);
    flip ^= 1;
    // a row past the last one is zeros: 0 times the infinite root of eps = 0 must not reach dgamma
    const float rstd = row < p.T ? rsqrtf(s.x * inv_d + p.eps) : 0.f;
    const float c = rstd * rstd * (s.y * inv_d);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t0 + i * step;
      const F8 a = cr[i].f(), b = cy[i].f(), e = g[i].f(), f = cq[i].f();
      F8 o;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        dg[i].v[k] = fmaf(b.v[k], a.v[k] * rstd, dg[i].v[k]);
        o.v[k] = fmaf(rstd, b.v[k] * e.v[k] - a.v[k] * c, f.v[k]);
      }
      if (v < nvec) store8(static_cast<E*>(p.dX) + row * p.d + 8 * v, o);
    }
  }
  // the block's row groups together, in their order: rows that share a warp by shuffles, then
  // one group after the other through shared memory (groups are 256 threads at most, so
  // 256 * NV * 8 columns)
  float* part = p.part + (int64_t)blockIdx.x * p.d;
  if (p.rpb == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t0 + i * step;
      if (v < p.nvec) store8(part + 8 * v, dg[i]);
    }
    return;
  }
  __shared__ float acc[MAXT <= 256 ? 256 * NV * 8 : 8];
  for (int o = p.lpr; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) dg[i].v[k] += __shfl_xor_sync(0xffffffffu, dg[i].v[k], o);
  const bool shared_warp = p.lpr < 32;
  const int group = shared_warp ? threadIdx.x / 32 : sub, groups = shared_warp ? blockDim.x / 32 : p.rpb;
  const bool mine = !shared_warp || (int)(threadIdx.x % 32) < p.lpr;
  for (int n = 0; n < groups; ++n) {
    if (group == n && mine) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = t0 + i * step;
        if (v < p.nvec) {
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[8 * v + k] = n ? acc[8 * v + k] + dg[i].v[k] : dg[i].v[k];
        }
      }
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < p.d; i += blockDim.x) part[i] = acc[i];
}

// The same where a block works on one row (d > 2048), whose R, dY and dR come by bulk copies into a
// ring of `stages` rows in shared memory: whole rows stay in flight however many registers their
// threads have.  A row's place is filled again behind the next row's barrier.  bf16, from
// registers and from the ring: 16384 x 2560 63 and 60 us, 16384 x 4096 92 and 88 (6120 GB/s),
// 8190 x 5120 74 and 67, 8190 x 8192 95 and 87 (6190 GB/s); 4096 x 16384, two rows of 1024
// threads, 151 and 146.
struct RingP {
  BwdP b;
  int stages;
  int stall;   // test hook: a block's second row is never loaded, so that the wait for it runs out
  int32_t* status;
  uint64_t limit_ns;
};
constexpr int MAX_STAGES = 4;
constexpr int RING_BYTES = 208 * 1024;   // of an SM
template <typename E, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k_rmsnorm_bwd_ring(const RingP a) {
  constexpr int NV = 2;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 red[2][MAXW];
  __shared__ uint64_t full[MAX_STAGES];
  // A wait of this row (two rows in turn) ran out.  Set before the row's barrier and read behind
  // it, so that every thread leaves at the same row: one flag for all rows could be set by a
  // thread a row ahead, and threads would stop at different barriers.
  __shared__ int late[2];
  const BwdP& p = a.b;
  const int step = blockDim.x, t0 = threadIdx.x;
  const uint32_t bytes = (uint32_t)(p.d * sizeof(E));   // of an operand's row
  const float inv_d = 1.f / (float)p.d;
  const int64_t stride = gridDim.x;
  auto load = [&](int64_t row, int slot) {   // by one thread
    if (row >= p.T || (a.stall && row == blockIdx.x + stride)) return;
    uint8_t* dst = ring + (size_t)slot * 3 * bytes;
    tc::mbar_expect_tx(&full[slot], (p.dR ? 3u : 2u) * bytes);
    tc::bulk_load(tc::saddr(dst), static_cast<const E*>(p.R) + row * p.d, bytes, &full[slot]);
    tc::bulk_load(tc::saddr(dst + bytes), static_cast<const E*>(p.dY) + row * p.d, bytes, &full[slot]);
    if (p.dR) tc::bulk_load(tc::saddr(dst + 2 * bytes), static_cast<const E*>(p.dR) + row * p.d, bytes, &full[slot]);
  };
  if (t0 == 0) {
    late[0] = late[1] = 0;
    for (int i = 0; i < a.stages; ++i) tc::mbar_init(&full[i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (int i = 0; i < a.stages; ++i) load(blockIdx.x + i * stride, i);
  }
  F8 dg[NV];
  Raw<E> g[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t0 + i * step;
    if (v < p.nvec) g[i].load(static_cast<const E*>(p.gamma) + 8 * v);
    else g[i].zero();
#pragma unroll
    for (int k = 0; k < 8; ++k) dg[i].v[k] = 0.f;
  }
  __syncthreads();
  int flip = 0, slot = 0;
  uint32_t phase = 0;
  bool out = false;
  for (int64_t row = blockIdx.x; row < p.T; row += stride) {
    const E* r = reinterpret_cast<const E*>(ring + (size_t)slot * 3 * bytes);
    const E *y = r + p.d, *q = y + p.d;
    volatile int* mark = &late[flip];
    if (!tc::wait_inl<false>(&full[slot], phase, mark, a.limit_ns)) *mark = 1;
    Raw<E> cr[NV], cy[NV];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t0 + i * step;
      cr[i].zero();
      cy[i].zero();
      if (v < p.nvec) {
        cr[i].load(r + 8 * v);
        cy[i].load(y + 8 * v);
      }
      const F8 x = cr[i].f(), b = cy[i].f(), c = g[i].f();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s.x = fmaf(x.v[k], x.v[k], s.x);
        s.y = fmaf(b.v[k] * c.v[k], x.v[k], s.y);
      }
    }
    s = row_sums(s, red, flip, 32, step / 32);
    flip ^= 1;
    out = *mark != 0;
    if (out) break;
    // the row before this one has been read by all
    if (t0 == 0 && row != blockIdx.x) load(row + (a.stages - 1) * stride, slot ? slot - 1 : a.stages - 1);
    const float rstd = rsqrtf(s.x * inv_d + p.eps);
    const float c = rstd * rstd * (s.y * inv_d);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t0 + i * step;
      if (v < p.nvec) {
        Raw<E> cq;
        cq.zero();
        if (p.dR) cq.load(q + 8 * v);
        const F8 x = cr[i].f(), b = cy[i].f(), e = g[i].f(), f = cq.f();
        F8 o;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          dg[i].v[k] = fmaf(b.v[k], x.v[k] * rstd, dg[i].v[k]);
          o.v[k] = fmaf(rstd, b.v[k] * e.v[k] - x.v[k] * c, f.v[k]);
        }
        store8(static_cast<E*>(p.dX) + row * p.d + 8 * v, o);
      }
    }
    if (++slot == a.stages) {
      slot = 0;
      phase ^= 1;
    }
  }
  if (out) {   // the copies in flight come to rest before the block ends
    if (t0 == 0) {
      atomicCAS(a.status, 0, SBP_ERR_TIMEOUT);
      for (int i = 0; i < a.stages; ++i) tc::wait_inl<false>(&full[i], phase ^ (i < slot ? 1u : 0u), nullptr, 200000000ull);
    }
    __syncthreads();
  }
  float* part = p.part + (int64_t)blockIdx.x * p.d;
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

// Up to 256 elements a row: one vector a thread, a power of two lanes a row, several rows a
// warp.  Else two vectors a thread (twice the loads in flight of one: T = 16384, d = 4096 forward,
// a row a block then, 85 us against 89) and whole warps a row; up to 256 threads' worth of rows a block.
struct Shape { int nv, lpr, wpr, rpb, threads; };
Shape shape_of(int64_t d) {
  const int nvec = (int)(d / 8);
  Shape s;
  s.nv = nvec <= 32 ? 1 : 2;
  s.lpr = 32;
  while (s.lpr > 1 && s.lpr / 2 >= nvec) s.lpr /= 2;
  s.wpr = std::max(1, (nvec + 32 * s.nv - 1) / (32 * s.nv));
  s.rpb = std::max(1, 256 / (s.lpr * s.wpr));
  s.threads = s.lpr * s.wpr * s.rpb;
  return s;
}
// Blocks of a launch: what the SMs hold at once of a kernel built for `minb` blocks of `maxt`
// threads, and no more than there are rows.
int64_t blocks_of(int64_t T, const Shape& s, int maxt, int minb) {
  return std::max<int64_t>(1, std::min<int64_t>((T + s.rpb - 1) / s.rpb,
                                                (int64_t)num_sms() * std::max(1, maxt * minb / s.threads)));
}

int norm_check(int64_t T, int64_t d, int dtype) {
  if (T < 0 || d < 1 || (dtype != SBP_BF16 && dtype != SBP_FP32)) return SBP_ERR_INVALID_ARG;
  if (d % 8 != 0 || d > MAX_D || T > (int64_t)1 << 31) return SBP_ERR_UNSUPPORTED;
  return SBP_OK;
}

template <typename E, int NV, bool Q8, int MAXT, int MINB>
cudaError_t launch_fwd1(const FwdP& p, const Shape& s, cudaStream_t st) {
  k_rmsnorm_fwd<E, NV, Q8, MAXT, MINB><<<(unsigned)blocks_of(p.T, s, MAXT, MINB), s.threads, 0, st>>>(p);
  return cudaGetLastError();
}
template <typename E, bool Q8>
cudaError_t launch_fwd(const FwdP& p, const Shape& s, cudaStream_t st) {
  if (s.nv == 1) return launch_fwd1<E, 1, Q8, 256, 4>(p, s, st);
  if (s.threads <= 256) return launch_fwd1<E, 2, Q8, 256, 3>(p, s, st);
  if (s.threads <= 512) return launch_fwd1<E, 2, Q8, 512, 2>(p, s, st);
  return launch_fwd1<E, 2, Q8, 1024, 1>(p, s, st);
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
  FwdP p{X, res, gamma, T, (int)d, (int)(d / 8), sh.lpr, sh.wpr, sh.rpb, eps, R, Y, scales, (int)((d + 127) / 128)};
  cudaError_t e;
  if (dtype == SBP_BF16)
    e = q8 ? launch_fwd<__nv_bfloat16, true>(p, sh, s) : launch_fwd<__nv_bfloat16, false>(p, sh, s);
  else
    e = q8 ? launch_fwd<float, true>(p, sh, s) : launch_fwd<float, false>(p, sh, s);
  if (e != cudaSuccess) return SBP_ERR_CUDA;
  set_launch_count(1);
  return SBP_OK;
}

// The register builds: threads and blocks an SM, which set the registers of a thread (128; 64 at
// more than 512 threads, which leaves none for the loads ahead).
void bwd_build(const Shape& s, int* maxt, int* minb) {
  if (s.nv == 1) { *maxt = 256; *minb = 3; }
  else if (s.threads <= 256) { *maxt = 256; *minb = 2; }
  else if (s.threads <= 512) { *maxt = 512; *minb = 1; }
  else { *maxt = 1024; *minb = 1; }
}

// The ring's rows and its blocks an SM; no rows where several rows share a block or fewer than
// three fit (fp32, 8190 x 8192: 221 us with two, 186 from registers; two are kept where the
// registers hold no row ahead).
int ring_stages(const Shape& s, int64_t d, int dtype, int* per_sm) {
  *per_sm = std::max(1, 512 / s.threads);
  if (s.rpb > 1) return 0;
  const int64_t n = RING_BYTES / *per_sm / (3 * d * (dtype == SBP_BF16 ? 2 : 4));
  return n < (s.threads <= 512 ? 3 : 2) ? 0 : (int)std::min<int64_t>(n, MAX_STAGES);
}

struct BwdLayout {
  size_t off_part = 0, total = 0;
  int64_t blocks = 0;
  int stages = 0;
  Guards guards;   // checked build only
};
bool bwd_layout(int64_t T, int64_t d, int dtype, BwdLayout* L) {
  if (norm_check(T, d, dtype) != SBP_OK) return false;
  BwdLayout l;
  const Shape s = shape_of(d);
  int maxt, minb;
  bwd_build(s, &maxt, &minb);
  int per_sm;
  l.stages = ring_stages(s, d, dtype, &per_sm);
  l.blocks = l.stages ? std::max<int64_t>(1, std::min<int64_t>(T, (int64_t)num_sms() * per_sm)) : blocks_of(T, s, maxt, minb);
  size_t o = 0;
  l.off_part = take_region(o, (size_t)l.blocks * d * sizeof(float), l.guards);
  l.total = o;
  *L = l;
  return true;
}

template <typename E>
cudaError_t launch_bwd(const BwdP& p, const Shape& s, unsigned grid, cudaStream_t st) {
  if (s.nv == 1) k_rmsnorm_bwd<E, 1, 256, 3><<<grid, s.threads, 0, st>>>(p);
  else if (s.threads <= 256) k_rmsnorm_bwd<E, 2, 256, 2><<<grid, s.threads, 0, st>>>(p);
  else if (s.threads <= 512) k_rmsnorm_bwd<E, 2, 512, 1><<<grid, s.threads, 0, st>>>(p);
  else k_rmsnorm_bwd<E, 2, 1024, 1><<<grid, s.threads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename E, int MAXT, int MINB>
cudaError_t launch_ring1(const RingP& r, const Shape& s, unsigned grid, cudaStream_t st) {
  static int attr_state[64] = {};
  static std::mutex mu;
  if (!tc::once_per_device(attr_state, mu, [] {
        return cudaFuncSetAttribute(k_rmsnorm_bwd_ring<E, MAXT, MINB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    RING_BYTES / MINB) == cudaSuccess;
      }))
    return cudaErrorInvalidConfiguration;
  k_rmsnorm_bwd_ring<E, MAXT, MINB><<<grid, s.threads, (size_t)r.stages * 3 * r.b.d * sizeof(E), st>>>(r);
  return cudaGetLastError();
}
template <typename E>
cudaError_t launch_ring(const RingP& r, const Shape& s, unsigned grid, cudaStream_t st) {
  if (s.threads <= 256) return launch_ring1<E, 256, 2>(r, s, grid, st);
  if (s.threads <= 512) return launch_ring1<E, 512, 1>(r, s, grid, st);
  return launch_ring1<E, 1024, 1>(r, s, grid, st);
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
  BwdP p{dY, R, gamma, dR, T, (int)d, (int)(d / 8), sh.lpr, sh.wpr, sh.rpb, eps, dX, part};
  cudaError_t e;
  if (L.stages) {
    const RingP r{p, L.stages, tc::fault_stall_requested(), dev_status, tc::wait_limit_ns()};
    e = dtype == SBP_BF16 ? launch_ring<__nv_bfloat16>(r, sh, (unsigned)L.blocks, s)
                          : launch_ring<float>(r, sh, (unsigned)L.blocks, s);
  } else {
    e = dtype == SBP_BF16 ? launch_bwd<__nv_bfloat16>(p, sh, (unsigned)L.blocks, s)
                          : launch_bwd<float>(p, sh, (unsigned)L.blocks, s);
  }
  if (e != cudaSuccess) return SBP_ERR_CUDA;
  k_dgamma<<<(unsigned)((d + 31) / 32), 1024, 0, s>>>(part, (int)L.blocks, (int)d, accumulate ? 1 : 0, dgamma);
  if (cudaGetLastError() != cudaSuccess) return SBP_ERR_CUDA;
  st = workspace_guards(w, L.guards, 1, dev_status, s, &launches);
  if (st == SBP_OK) set_launch_count(launches);
  return st;
}

}  // extern "C"
