// Quantisers to 8 bits (e4m3) with one scale for each block of 128 (sm_103a): what the block-scaled
// product takes.
//
//   s = max(max|x| * fl(1 / 448), 2^-126) over the block (1 for a block of zeros),  q = e4m3(x * fl(1 / s))
//
//   rows      blocks of 128 columns of a row
//   columns   blocks of 128 tokens of one column, or tiles of 128 tokens x 128 columns, written
//             transposed (the tokens run along the rows, as a product that sums over tokens wants
//             them), each expert's tokens from a multiple of 128 on
//   weight    tiles of 128 x 128, written in both orders
//
// All are bound by device memory.
#include <algorithm>

#include "sbp_groups.cuh"
#include "sbp_rows.cuh"
#include "sbp_tc_common.cuh"

namespace sbp {
namespace {

constexpr int64_t MAX_D = 1 << 20;

// The scale of a block whose largest magnitude is `a`.  448: e4m3's largest value.  A block of zeros
// keeps the scale 1; a scale that is not normal would have no inverse.
__device__ __forceinline__ float block_scale(float a) {
  return a > 0.f ? fmaxf(a * (1.f / 448.f), 1.17549435e-38f) : 1.f;
}

template <typename E>
__device__ __forceinline__ float amax8(const Raw<E>& r) {
  const F8 f = r.f();
  float a = fabsf(f.v[0]);
#pragma unroll
  for (int k = 1; k < 8; ++k) a = fmaxf(a, fabsf(f.v[k]));
  return a;
}

// Largest magnitudes of two pairs of bf16 values at a time (a NaN is passed over, as by fmaxf).
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}
__device__ __forceinline__ uint32_t abs2(uint32_t a) { return a & 0x7fff7fffu; }
__device__ __forceinline__ uint32_t amax2(const Raw<__nv_bfloat16>& r) {
  return max2(max2(abs2(r.u.x), abs2(r.u.y)), max2(abs2(r.u.z), abs2(r.u.w)));
}
__device__ __forceinline__ float low2(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high2(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
// The largest magnitude of each of eight rows over the 16 lanes that share them: in lane c that of
// row c % 8.
__device__ __forceinline__ float row_amax(const Raw<__nv_bfloat16> (&x)[8], int c) {
  uint32_t m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {   // rows 2i and 2i + 1 in one word
    const uint32_t a = amax2(x[2 * i]), b = amax2(x[2 * i + 1]);
    m[i] = max2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
  }
#pragma unroll
  for (int o = 8; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = max2(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
  const uint32_t v = c & 4 ? (c & 2 ? m[3] : m[2]) : (c & 2 ? m[1] : m[0]);
  return c & 1 ? high2(v) : low2(v);
}
__device__ __forceinline__ float row_amax(const Raw<float> (&x)[8], int c) {
  float m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = amax8(x[i]);
#pragma unroll
  for (int o = 8; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
  float v = m[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) v = (c & 7) == i ? m[i] : v;
  return v;
}
// The largest magnitude of each of eight columns over the eight rows of this thread and those of
// the other half of the warp.
__device__ __forceinline__ F8 col_amax(const Raw<__nv_bfloat16> (&x)[8]) {
  uint32_t m[4] = {abs2(x[0].u.x), abs2(x[0].u.y), abs2(x[0].u.z), abs2(x[0].u.w)};
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    m[0] = max2(m[0], abs2(x[i].u.x));
    m[1] = max2(m[1], abs2(x[i].u.y));
    m[2] = max2(m[2], abs2(x[i].u.z));
    m[3] = max2(m[3], abs2(x[i].u.w));
  }
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = max2(m[i], __shfl_xor_sync(0xffffffffu, m[i], 16));
    f.v[2 * i] = low2(m[i]);
    f.v[2 * i + 1] = high2(m[i]);
  }
  return f;
}
__device__ __forceinline__ F8 col_amax(const Raw<float> (&x)[8]) {
  F8 m = x[0].f();
#pragma unroll
  for (int j = 0; j < 8; ++j) m.v[j] = fabsf(m.v[j]);
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    const F8 v = x[i].f();
#pragma unroll
    for (int j = 0; j < 8; ++j) m.v[j] = fmaxf(m.v[j], fabsf(v.v[j]));
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) m.v[j] = fmaxf(m.v[j], __shfl_xor_sync(0xffffffffu, m.v[j], 16));
  return m;
}
__device__ __forceinline__ float all_amax(const Raw<__nv_bfloat16> (&x)[8]) {
  uint32_t m = amax2(x[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max2(m, amax2(x[i]));
  return fmaxf(low2(m), high2(m));
}
__device__ __forceinline__ float all_amax(const Raw<float> (&x)[8]) {
  float a = amax8(x[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) a = fmaxf(a, amax8(x[i]));
  return a;
}

struct RowsP {
  const void* X;
  uint32_t units;       // blocks of 128 columns of all rows
  uint32_t nblk, d;
  uint8_t* Y8;
  float* scales;
};

constexpr int ROW_UNITS = 2;   // blocks of 16 lanes, all loads in flight (16384 x 4096: 34 us; 35 with four, 41 with one)

// 16 lanes a block of 128 columns, 8 columns a lane.
template <typename E>
__global__ void __launch_bounds__(256) k_quant_rows(const RowsP p) {
  const uint32_t lane = threadIdx.x % 16;
  const uint64_t u0 = (uint64_t)blockIdx.x * (16 * ROW_UNITS) + threadIdx.x / 16;
  Raw<E> x[ROW_UNITS];
  int64_t at[ROW_UNITS];
#pragma unroll
  for (int i = 0; i < ROW_UNITS; ++i) {
    const uint64_t u = u0 + 16 * i;
    x[i].zero();
    at[i] = -1;
    if (u < p.units) {
      const uint32_t row = (uint32_t)u / p.nblk, c = ((uint32_t)u - row * p.nblk) * 128 + 8 * lane;
      if (c < p.d) {
        at[i] = (int64_t)row * p.d + c;
        x[i].load(static_cast<const E*>(p.X) + at[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < ROW_UNITS; ++i) {
    float a = amax8(x[i]);
#pragma unroll
    for (int o = 8; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    const float s = block_scale(a), inv = 1.f / s;
    if (at[i] < 0) continue;
    const F8 f = x[i].f();
    *reinterpret_cast<uint2*>(p.Y8 + at[i]) =
        make_uint2(e4m3_pack(f.v[0], f.v[1], f.v[2], f.v[3], inv), e4m3_pack(f.v[4], f.v[5], f.v[6], f.v[7], inv));
    if (lane == 0) p.scales[u0 + 16 * i] = s;
  }
}

struct TileP {
  const void* X;            // [rows, d]
  const int32_t* offsets;   // columns: the experts' rows (null: one expert)
  int64_t T;
  int E, d, nf;             // nf: blocks of 128 columns
  int wrows, wblocks;       // weight: rows and row blocks of an expert (0: columns)
  uint8_t* Y8;              // row order
  float* scales;
  uint8_t* Yt8;             // transposed
  int64_t pitch;
  float* scales_t;
  int nbt;                  // scales of a transposed row
  int32_t* status;
};

// One CTA a tile of 128 tokens x 128 columns, held in registers: thread (g, c) has 8 columns of
// 8 neighbouring tokens, so that its 64 values make 8 transposed words of 8 bytes.  They are
// exchanged through 16 KB of shared memory (the 8-byte chunk of a token group xored with the column
// group, both ways without bank conflicts) and leave as rows of 128 bytes.
// ROWS: 0 none, 1 blocks of 128 columns of a row, 2 tiles.  COLS: 1 blocks of 128 tokens of a
// column, 2 tiles.
// Blocks an SM (16384 x 4096 in bf16, 3, 4, 5 and 6 of them): columns 42, 38, 36 and 50 us, tiles 41, 37,
// 35 and 45, columns and rows 55, 50, 61 and 68; in fp32 the tile takes the registers of two.
template <typename E, int ROWS, int COLS>
__global__ void __launch_bounds__(256, sizeof(E) == 4 ? 2 : ROWS == 0 ? 5 : 4) k_quant_tile(const TileP p) {
  __shared__ uint2 tile[128 * 16];
  __shared__ float cmax[8][128];
  __shared__ float sinv[128];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, c8 = tid % 16, g8 = tid / 16;
  const int b = (int)(blockIdx.x / p.nf), f = (int)(blockIdx.x - (unsigned)b * p.nf), f0 = f * 128;
  int64_t row0;
  int rows, e = 0, ib = b;
  if (p.wblocks) {
    e = b / p.wblocks;
    ib = b - e * p.wblocks;
    row0 = (int64_t)e * p.wrows + ib * 128;
    rows = min(128, p.wrows - ib * 128);
  } else {
    const Group g = find_unit_of_block(p.offsets, p.E, p.T, 128, b);
    if (blockIdx.x == 0 && tid == 0 && p.status) *p.status = g.bad ? SBP_ERR_SEQLENS : SBP_OK;
    if (g.bad || !g.found) return;
    row0 = (int64_t)g.row0 + g.i * 128;
    rows = min(128, g.rows - g.i * 128);
  }
  const int col = f0 + 8 * c8;
  Raw<E> x[8];
  const E* in = static_cast<const E*>(p.X) + (row0 + g8 * 8) * p.d + col;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = g8 * 8 + i;
    x[i].zero();
    if (r < rows && col < p.d) x[i].load(in + (int64_t)i * p.d);
  }
  float tinv = 1.f;
  if (COLS == 1) {
    const F8 m = col_amax(x);
    if (lane < 16) {
      float4* q = reinterpret_cast<float4*>(&cmax[warp][8 * c8]);
      q[0] = make_float4(m.v[0], m.v[1], m.v[2], m.v[3]);
      q[1] = make_float4(m.v[4], m.v[5], m.v[6], m.v[7]);
    }
    __syncthreads();
    if (tid < 128) {
      float a = cmax[0][tid];
#pragma unroll
      for (int w = 1; w < 8; ++w) a = fmaxf(a, cmax[w][tid]);
      const float s = block_scale(a);
      sinv[tid] = 1.f / s;
      if (f0 + tid < p.d) p.scales_t[(int64_t)(f0 + tid) * p.nbt + b] = s;
    }
    __syncthreads();
  } else {
    float a = all_amax(x);
#pragma unroll
    for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (lane == 0) cmax[0][warp] = a;
    __syncthreads();
    a = cmax[0][0];
#pragma unroll
    for (int w = 1; w < 8; ++w) a = fmaxf(a, cmax[0][w]);
    const float s = block_scale(a);
    tinv = 1.f / s;
    if (tid == 0) {
      if (p.wblocks) {
        p.scales[((int64_t)e * p.wblocks + ib) * p.nf + f] = s;
        p.scales_t[((int64_t)e * p.nf + f) * p.wblocks + ib] = s;
      } else {
        p.scales_t[(int64_t)f * p.nbt + b] = s;
      }
    }
  }
  if (ROWS != 0) {
    float rinv = tinv;
    if (ROWS == 1) {   // each lane one row's scale: a division costs more than a shuffle
      const float s = block_scale(row_amax(x, c8));
      rinv = 1.f / s;
      if (c8 < 8 && g8 * 8 + c8 < rows) p.scales[(row0 + g8 * 8 + c8) * p.nf + f] = s;
    }
    uint8_t* out = p.Y8 + (row0 + g8 * 8) * p.d + col;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float inv = ROWS == 1 ? __shfl_sync(0xffffffffu, rinv, i, 16) : tinv;
      if (g8 * 8 + i < rows && col < p.d) {
        const F8 v = x[i].f();
        *reinterpret_cast<uint2*>(out + (int64_t)i * p.d) =
            make_uint2(e4m3_pack(v.v[0], v.v[1], v.v[2], v.v[3], inv), e4m3_pack(v.v[4], v.v[5], v.v[6], v.v[7], inv));
      }
    }
  }
  float ci[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) ci[j] = COLS == 1 ? sinv[8 * c8 + j] : tinv;
  {
    F8 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x[i].f();
#pragma unroll
    for (int j = 0; j < 8; ++j)
      tile[(8 * c8 + j) * 16 + (g8 ^ c8)] =
          make_uint2(e4m3_pack(v[0].v[j], v[1].v[j], v[2].v[j], v[3].v[j], ci[j]),
                     e4m3_pack(v[4].v[j], v[5].v[j], v[6].v[j], v[7].v[j], ci[j]));
  }
  __syncthreads();
  // transposed rows: 128 bytes each (an expert's padding is zeros), in pieces of 16
  uint8_t* out = p.Yt8 + (p.wblocks ? (int64_t)e * p.d * p.pitch + ib * 128 : (int64_t)b * 128);
  const int wide = p.wblocks ? rows : 128;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int q = k * 256 + tid, r = q / 8, m = q % 8, sw = r / 8;
    if (f0 + r < p.d && 16 * m < wide) {
      const uint2 lo = tile[r * 16 + ((2 * m) ^ sw)], hi = tile[r * 16 + ((2 * m + 1) ^ sw)];
      *reinterpret_cast<uint4*>(out + (int64_t)(f0 + r) * p.pitch + 16 * m) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  }
}

// Y = q * scale: blocks of 2^shift rows x 128 columns, 8 elements a thread (n8 of them a row) twice,
// so that a warp's loads and stores are whole lines.
template <typename O, typename I>
__global__ void __launch_bounds__(256) k_quant_expand(const uint8_t* __restrict__ q, const float* __restrict__ scales,
                                                      I n, uint32_t n8, int shift, int nblk, O* __restrict__ out) {
  uint2 u[2];
  float s[2];
  const I i0 = (I)blockIdx.x * 512 + threadIdx.x;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const I i = i0 + 256 * k;
    if (i < n) {
      const I row = i / n8;
      u[k] = *reinterpret_cast<const uint2*>(q + (int64_t)i * 8);
      s[k] = scales[(int64_t)(row >> shift) * nblk + (uint32_t)(i - row * n8) / 16];
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const I i = i0 + 256 * k;
    const uint32_t w[2] = {u[k].x, u[k].y};
    F8 f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j / 2] >> (16 * (j % 2))), __NV_E4M3);
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&r));
      f.v[2 * j] = x.x * s[k];
      f.v[2 * j + 1] = x.y * s[k];
    }
    if (i < n) store8(out + (int64_t)i * 8, f);
  }
}

// ------------------------------------------------------------------------------ host side

int quant_check(int64_t T, int64_t d, int dtype) {
  if (T < 0 || d < 1 || (dtype != SBP_BF16 && dtype != SBP_FP32)) return SBP_ERR_INVALID_ARG;
  if (d % 8 != 0 || d > MAX_D || T > (int64_t(1) << 30)) return SBP_ERR_UNSUPPORTED;
  return SBP_OK;
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int launched() {
  if (cudaGetLastError() != cudaSuccess) return SBP_ERR_CUDA;
  set_launch_count(1);
  return SBP_OK;
}

template <int ROWS, int COLS>
int launch_tile(const TileP& p, int64_t blocks, int dtype, cudaStream_t s) {
  if (blocks > INT32_MAX) return SBP_ERR_UNSUPPORTED;
  if (dtype == SBP_BF16) k_quant_tile<__nv_bfloat16, ROWS, COLS><<<(unsigned)blocks, 256, 0, s>>>(p);
  else k_quant_tile<float, ROWS, COLS><<<(unsigned)blocks, 256, 0, s>>>(p);
  return launched();
}

}  // namespace
}  // namespace sbp

using namespace sbp;

extern "C" {

int64_t sbp_token_blocks(int64_t T, int64_t E) {
  return T < 0 || E < 1 || T > (int64_t(1) << 30) || E > MAX_GROUPS ? -1 : max_units(T, E, 128);
}

int sbp_quant_e4m3_rows(const void* X, int64_t T, int64_t d, int dtype, void* Y8, float* scales, void* stream) {
  const int rc = quant_check(T, d, dtype);
  if (rc != SBP_OK) return rc;
  const int64_t nblk = (d + 127) / 128;
  if (T * nblk > INT32_MAX) return SBP_ERR_UNSUPPORTED;
  if (T > 0 && (!X || !Y8 || !scales)) return SBP_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(Y8) || !aligned4(scales)) return SBP_ERR_ALIGNMENT;
  NvtxRange nv("sbp_quant_e4m3_rows");
  set_launch_count(0);
  if (T == 0) return SBP_OK;
  const RowsP p{X, (uint32_t)(T * nblk), (uint32_t)nblk, (uint32_t)d, static_cast<uint8_t*>(Y8), scales};
  const unsigned grid = (unsigned)((T * nblk + 16 * ROW_UNITS - 1) / (16 * ROW_UNITS));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == SBP_BF16) k_quant_rows<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
  else k_quant_rows<float><<<grid, 256, 0, s>>>(p);
  return launched();
}

int sbp_quant_e4m3_expand(const void* Y8, const float* scales, int64_t T, int64_t d, int tiles, int dtype, void* Y,
                          void* stream) {
  const int rc = quant_check(T, d, dtype);
  if (rc != SBP_OK) return rc;
  if ((tiles != 0 && tiles != 1) || (T > 0 && (!Y8 || !scales || !Y))) return SBP_ERR_INVALID_ARG;
  const int64_t n = T * (d / 8), blocks = (n + 511) / 512;
  if (blocks > INT32_MAX) return SBP_ERR_UNSUPPORTED;
  if (!aligned16(Y8) || !aligned16(Y) || !aligned4(scales)) return SBP_ERR_ALIGNMENT;
  NvtxRange nv("sbp_quant_e4m3_expand");
  set_launch_count(0);
  if (T == 0) return SBP_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const uint8_t* q = static_cast<const uint8_t*>(Y8);
  const int shift = tiles ? 7 : 0, nblk = (int)((d + 127) / 128);
  auto go = [&](auto* y) {   // 32-bit indices where they do
    if (n < (int64_t(1) << 31))
      k_quant_expand<<<(unsigned)blocks, 256, 0, s>>>(q, scales, (uint32_t)n, (uint32_t)(d / 8), shift, nblk, y);
    else
      k_quant_expand<<<(unsigned)blocks, 256, 0, s>>>(q, scales, n, (uint32_t)(d / 8), shift, nblk, y);
  };
  if (dtype == SBP_BF16) go(static_cast<__nv_bfloat16*>(Y));
  else go(static_cast<float*>(Y));
  return launched();
}

int sbp_quant_e4m3_columns(const void* X, const int32_t* offsets, int64_t E, int64_t T, int64_t d, int dtype,
                           int tiles, void* Y8, float* scales, void* Yt8, float* scales_t, int32_t* dev_status,
                           void* stream) {
  const int rc = quant_check(T, d, dtype);
  if (rc != SBP_OK) return rc;
  if (E < 1 || (!offsets && E != 1) || (tiles != 0 && tiles != 1)) return SBP_ERR_INVALID_ARG;
  if (E > MAX_GROUPS) return SBP_ERR_UNSUPPORTED;
  if ((Y8 == nullptr) != (scales == nullptr) || !dev_status || (T > 0 && (!X || !Yt8 || !scales_t)))
    return SBP_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(Y8) || !aligned16(Yt8)) return SBP_ERR_ALIGNMENT;
  for (const void* q : {(const void*)offsets, (const void*)scales, (const void*)scales_t, (const void*)dev_status})
    if (!aligned4(q)) return SBP_ERR_ALIGNMENT;
  NvtxRange nv("sbp_quant_e4m3_columns");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  set_launch_count(0);
  if (T == 0) return no_rows(offsets, E, nullptr, 0, dev_status, s);
  const int64_t nb = max_units(T, E, 128), nf = (d + 127) / 128;
  TileP p{X, offsets, T, (int)E, (int)d, (int)nf, 0, 0, static_cast<uint8_t*>(Y8), scales,
          static_cast<uint8_t*>(Yt8), nb * 128, scales_t, (int)nb, dev_status};
  if (Y8) return tiles ? launch_tile<1, 2>(p, nb * nf, dtype, s) : launch_tile<1, 1>(p, nb * nf, dtype, s);
  return tiles ? launch_tile<0, 2>(p, nb * nf, dtype, s) : launch_tile<0, 1>(p, nb * nf, dtype, s);
}

int sbp_quant_e4m3_weight(const void* W, int64_t E, int64_t N, int64_t K, int dtype, void* W8, float* scales,
                          void* Wt8, float* scales_t, void* stream) {
  if (E < 1 || N < 1 || K < 1 || (dtype != SBP_BF16 && dtype != SBP_FP32)) return SBP_ERR_INVALID_ARG;
  if (E > MAX_GROUPS || N % 16 != 0 || K % 16 != 0 || N > MAX_D || K > MAX_D) return SBP_ERR_UNSUPPORTED;
  if (!W || !W8 || !scales || !Wt8 || !scales_t) return SBP_ERR_INVALID_ARG;
  if (!aligned16(W) || !aligned16(W8) || !aligned16(Wt8) || !aligned4(scales) || !aligned4(scales_t))
    return SBP_ERR_ALIGNMENT;
  NvtxRange nv("sbp_quant_e4m3_weight");
  set_launch_count(0);
  const int64_t nn = (N + 127) / 128, nk = (K + 127) / 128;
  TileP p{W, nullptr, E * N, (int)E, (int)K, (int)nk, (int)N, (int)nn, static_cast<uint8_t*>(W8), scales,
          static_cast<uint8_t*>(Wt8), N, scales_t, (int)nn, nullptr};
  return launch_tile<2, 2>(p, E * nn * nk, dtype, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
