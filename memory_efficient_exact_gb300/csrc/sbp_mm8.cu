// Matrix products in 8 bits (e4m3) with a scale for each block of 128 (sm_103a).
//
//   rows     C[i, n] = sum_b sa[i, b] sb[e, n / 128, b] sum_{k in block b} A[i, k] B[e, n, k]
//            for the rows i of expert e (one expert: a linear layer; its dX with B transposed)
//   columns  dW[e, m, n] (+)= the same sum over the blocks b of expert e's tokens, A and B being
//            what the column quantiser leaves
//
// A has a scale for each row and block of 128, B one for each 128 x 128 tile.  Each product of two
// values is exact in fp32; the tensor cores add a block's up in fp32 (and may cut a sum off instead of
// rounding it); a block's sum is scaled and added in fp32, rounded.
#include <algorithm>

#include "sbp_groups.cuh"
#include "sbp_mm8.cuh"
#include "sbp_tc_common.cuh"

namespace sbp {
namespace mm8 {

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weights are read once: past the L1 cache, which keeps A and the scales.
__device__ __forceinline__ uint4 load_once(const uint8_t* q) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(q));
  return v;
}
constexpr int FEW_WARPS = 8;

// Few rows: what bounds the call is reading B once.  A block has 16 rows of B against 8 NT rows of
// A, its warps sharing out the blocks of 128; they go straight from device memory into the
// operands' registers.  (The order of k within a block of 128 is that of the 32 bytes a thread
// loads, the same for A and B.)  8 rows x 24576 x 4096: 22 us, 4.6 TB/s, with the matrix from memory;
// 19.6 with the same one throughout, part of it in L2.  Several blocks of 128 in flight a warp, at the
// price of blocks an SM, were slower than those 19.6 (28 us with two, 31 with four).
// MINB blocks are resident an SM, and so many are launched.
template <int NT, int MINB>
__global__ void __launch_bounds__(32 * FEW_WARPS, MINB) k_mm8_few(const P p) {
  __shared__ float red[FEW_WARPS][8 * NT][17];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int strips = (p.nb + 15) / 16;
  bool bad = false;
  int total;
  if (p.columns) {
    const Group u = find_unit(p.offsets, p.E, p.T, 128, 0);
    bad = u.bad;
    total = p.E * ((p.na + 8 * NT - 1) / (8 * NT));
  } else {
    const Group u = find_unit(p.offsets, p.E, p.T, 8 * NT, 0);
    bad = u.bad;
    total = u.total;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = bad ? SBP_ERR_SEQLENS : SBP_OK;
  if (bad) return;
  const int64_t items = (int64_t)total * strips;
  const int64_t i0 = items * blockIdx.x / gridDim.x, i1 = items * (blockIdx.x + 1) / gridDim.x;
  int have = -1;
  Unit w{};
  for (int64_t item = i0; item < i1; ++item) {
    const int u = (int)(item / strips), strip = (int)(item - (int64_t)u * strips);
    if (u != have) {
      w = unit_of(p, 8 * NT, u);
      have = u;
    }
    const int n0 = strip * 16;
    const int64_t first = (int64_t)(w.kb0 + warp) * 128 + 32 * t;
    const uint8_t* b0 = p.B + (int64_t)w.e * p.b_stride + (int64_t)min(n0 + g, p.nb - 1) * p.ldb + first;
    const int64_t to1 = (int64_t)(min(n0 + g + 8, p.nb - 1) - min(n0 + g, p.nb - 1)) * p.ldb;
    const uint8_t* a[NT];
    const float* sa[NT];
    int64_t to_next[NT];   // from the scale of the first of this thread's two columns to the second's
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      a[i] = p.A + (int64_t)(w.row0 + min(8 * i + g, w.rows - 1)) * p.lda + first;
      const int r = min(8 * i + 2 * t, w.rows - 1);
      sa[i] = p.sa + (int64_t)(w.row0 + r) * p.sa_pitch + w.kb0 + warp;
      to_next[i] = min(8 * i + 2 * t + 1, w.rows - 1) == r ? 0 : p.sa_pitch;
    }
    const float* sb = p.sb + (int64_t)w.e * p.sb_stride + (int64_t)(n0 / 128) * p.sb_pitch + w.kb0 + warp;
    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    auto block = [&](bool in0, bool in1) {   // which 16 bytes of this thread's 32 are inside the row
      const uint4 z = make_uint4(0u, 0u, 0u, 0u);
      uint4 x[4];
      x[0] = in0 ? load_once(b0) : z;
      x[1] = in1 ? load_once(b0 + 16) : z;
      x[2] = in0 ? load_once(b0 + to1) : z;
      x[3] = in1 ? load_once(b0 + to1 + 16) : z;
      const float s = *sb;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (i && 8 * i >= w.rows) break;
        const uint4 y0 = in0 ? *reinterpret_cast<const uint4*>(a[i]) : z;
        const uint4 y1 = in1 ? *reinterpret_cast<const uint4*>(a[i] + 16) : z;
        const float s0 = s * sa[i][0], s1 = s * sa[i][to_next[i]];
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        mma_e4m3(c, x[0].x, x[2].x, x[0].y, x[2].y, y0.x, y0.y);
        mma_e4m3(c, x[0].z, x[2].z, x[0].w, x[2].w, y0.z, y0.w);
        mma_e4m3(c, x[1].x, x[3].x, x[1].y, x[3].y, y1.x, y1.y);
        mma_e4m3(c, x[1].z, x[3].z, x[1].w, x[3].w, y1.z, y1.w);
        acc[i][0] = fmaf(c[0], s0, acc[i][0]);
        acc[i][1] = fmaf(c[1], s1, acc[i][1]);
        acc[i][2] = fmaf(c[2], s0, acc[i][2]);
        acc[i][3] = fmaf(c[3], s1, acc[i][3]);
        a[i] += FEW_WARPS * 128;
        sa[i] += FEW_WARPS;
      }
      b0 += FEW_WARPS * 128;
      sb += FEW_WARPS;
    };
    const int whole = min(w.kb1, (int)(p.K / 128));
    int kb = w.kb0 + warp;
#pragma unroll 1
    for (; kb < whole; kb += FEW_WARPS) block(true, true);
    if (kb < w.kb1) {
      const int64_t left = p.K - (int64_t)kb * 128 - 32 * t;
      block(left > 0, left > 16);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      red[warp][8 * i + 2 * t][g] = acc[i][0];
      red[warp][8 * i + 2 * t + 1][g] = acc[i][1];
      red[warp][8 * i + 2 * t][g + 8] = acc[i][2];
      red[warp][8 * i + 2 * t + 1][g + 8] = acc[i][3];
    }
    __syncthreads();
    for (int o = threadIdx.x; o < 128 * NT; o += 32 * FEW_WARPS) {
      const int r = o / 16, n = o % 16;
      if (r < w.rows && n0 + n < p.nb) {
        float v = red[0][r][n];
#pragma unroll
        for (int i = 1; i < FEW_WARPS; ++i) v += red[i][r][n];
        const int64_t at = (int64_t)w.e * p.c_stride + (int64_t)(w.row0 + r) * p.nb + n0 + n;
        if (p.out == SBP_BF16) {
          static_cast<__nv_bfloat16*>(p.C)[at] = __float2bfloat16_rn(v);
        } else {
          float* c = static_cast<float*>(p.C) + at;
          *c = p.accumulate ? *c + v : v;
        }
      }
    }
    __syncthreads();
  }
}

thread_local int g_ran = SBP_PRODUCT_NONE;
void ran(int kernel) { g_ran = kernel; }

// Blocks an SM, with the registers that leaves: 5 and 3 and 3 instead take 21.7 against 19.6 us for 8
// rows and 16.2 against 10.9 for 32, N = 24576 and 4096, K = 4096, the same inputs throughout.
constexpr int few_blocks(int nt) { return nt == 1 ? 4 : 2; }

template <int NT>
cudaError_t launch_few(const P& p, int64_t units, cudaStream_t s) {
  const int64_t items = units * ((p.nb + 15) / 16);
  const int64_t most = (int64_t)num_sms() * few_blocks(NT);
  k_mm8_few<NT, few_blocks(NT)><<<(unsigned)std::max<int64_t>(1, std::min(items, most)), 32 * FEW_WARPS, 0, s>>>(p);
  ran(SBP_PRODUCT_FEW);
  return cudaGetLastError();
}

// Rows of A that one block takes: as many as an expert has on average, in tiles of 8.
int few_tiles(const P& p) {
  const int64_t rows = p.columns ? p.na : (p.T + p.E - 1) / p.E;
  return rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
}
cudaError_t few(const P& p, cudaStream_t s) {
  const int nt = few_tiles(p);
  const int64_t units = p.columns ? (int64_t)p.E * ((p.na + 8 * nt - 1) / (8 * nt)) : max_units(p.T, p.E, 8 * nt);
  if (nt == 1) return launch_few<1>(p, units, s);
  if (nt == 2) return launch_few<2>(p, units, s);
  return launch_few<4>(p, units, s);
}

// k_mm8_few reads each unit's matrix at 5.5 TB/s behind a start of 4 us (8 rows x 24576 x 4096: 22
// us), and takes 1.5 and 2.65 times as long for units of 16 and 32 rows, whose values are converted
// for every strip.  Short sums are bound by the 2.1 us that a block takes for a strip of a unit at least
// (1000 rows x 512 x 512: 10.5 us).
int64_t few_ns(const P& p) {
  const int nt = few_tiles(p);
  const int64_t units = about_units(p, 8 * nt), blocks = (int64_t)num_sms() * few_blocks(nt);
  const int64_t bytes = (int64_t)p.nb * about_blocks(p) * 128, items = units * ((p.nb + 15) / 16);
  return std::max(4000 + units * bytes / 5500 * (nt == 1 ? 100 : nt == 2 ? 150 : 265) / 100,
                  1600 + (items + blocks - 1) / blocks * 2100);
}

// The kernel that takes the least time by the three rules.  Measured, few / many / swap, in us, with
// other inputs from call to call, so that matrices come from memory (the kernel taken is within 5% of
// the fastest in all of these and in 40 sizes more):
//   4096 x 4096, rows 1, 32, 48, 64, 128:       6.7 19 15,  11.4 16.5 17.5,  17 16.5 18,  20 16.6 17.8,  35 17 18
//   24576 x 4096, rows 8, 16, 32, 48, 64:       22 46 29,  32 42 31,  53 35 33,  81 35 39,  96 36 39
//   4096 x 12288, rows 32, 64:                  28 31 37,  54 31 37
//   512 x 512, rows 300, 1000:                  6.3 10.3 8.3,  10.5 10.3 8.3
//   64 experts, 4096 x 2560, rows 1, 2, 4, 8, 16 of as many:  6.8 17 14,  7.9 19 14,  12.5 22 17,  22 32 23,  35 78 38
//   the same, rows 64, 192, 400, 1000, 2000 of all:  123 144 107,  123 145 110,  125 147 111,  199 150 115,  352 155 122
//   256 experts, 2048 x 2048, rows 1, 4, 16, 64 of as many:   5.7 16 12,  8.6 19 14,  19 31 21,  54 74 51
//   8 experts, 4096 x 4096, rows 1, 4, 8, 16, 64, 128, 256:  7.7 20 16,  16 27 20,  28 44 31,  28 43 31,  30 40 31,  41 41 33,  65 42 35
//   columns, 1024 x 1024 of 128 tokens, 512 x 512 of 1000, 128 x 256 of 1000 of 32 experts:  15 10 -,  7.6 11 -,  17 11 -
int run(const P& p, cudaStream_t s) {
  const int64_t f = few_ns(p), m = many_ns(p), w = p.columns ? INT64_MAX : swap_ns(p);
  if ((f <= m && f <= w ? few(p, s) : m <= w ? many(p, s) : swap(p, s)) != cudaSuccess) return SBP_ERR_CUDA;
  set_launch_count(1);
  return SBP_OK;
}

__global__ void __launch_bounds__(256) k_no_rows(const int32_t* off, int E, float4* zeros, int64_t n, int32_t* status) {
  const bool bad = find_unit(off, E, 0, 1, 0).bad;
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = bad ? SBP_ERR_SEQLENS : SBP_OK;
  if (bad) return;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    zeros[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

int check_common(int64_t E, int64_t T, int64_t N, int64_t K, const void* A8, const void* sa, const void* B8,
                 const void* sb, const int32_t* offsets, const void* C, const int32_t* status) {
  for (const void* q : {A8, B8, C})
    if (!aligned16(q)) return SBP_ERR_ALIGNMENT;
  for (const void* q : {sa, sb, (const void*)offsets, (const void*)status})
    if (reinterpret_cast<uintptr_t>(q) & 3u) return SBP_ERR_ALIGNMENT;
  return SBP_OK;
}

}  // namespace mm8

int no_rows(const int32_t* offsets, int64_t E, float* zeros, int64_t n, int32_t* status, cudaStream_t s) {
  const int64_t n4 = zeros ? n / 4 : 0;
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>((n4 + 255) / 256, (int64_t)num_sms() * 8));
  mm8::k_no_rows<<<grid, 256, 0, s>>>(offsets, (int)E, reinterpret_cast<float4*>(zeros), n4, status);
  if (cudaGetLastError() != cudaSuccess) return SBP_ERR_CUDA;
  set_launch_count(1);
  return SBP_OK;
}

}  // namespace sbp

using namespace sbp;

extern "C" {

int sbp_matmul_e4m3(const void* A8, const float* sa, const void* B8, const float* sb, const int32_t* offsets,
                    int64_t E, int64_t T, int64_t N, int64_t K, int out_dtype, void* C, int32_t* dev_status,
                    void* stream) {
  if (E < 1 || T < 0 || N < 1 || K < 1 || (!offsets && E != 1) || (out_dtype != SBP_BF16 && out_dtype != SBP_FP32))
    return SBP_ERR_INVALID_ARG;
  if (E > MAX_GROUPS || K % 16 != 0 || N % 8 != 0 || T > (int64_t(1) << 30) || N > mm8::MAX_SIDE || K > mm8::MAX_SIDE)
    return SBP_ERR_UNSUPPORTED;
  if (!dev_status || (T > 0 && (!A8 || !sa || !B8 || !sb || !C))) return SBP_ERR_INVALID_ARG;
  const int rc = mm8::check_common(E, T, N, K, A8, sa, B8, sb, offsets, C, dev_status);
  if (rc != SBP_OK) return rc;
  NvtxRange nv("sbp_matmul_e4m3");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  set_launch_count(0);
  mm8::ran(SBP_PRODUCT_NONE);
  if (T == 0) return no_rows(offsets, E, nullptr, 0, dev_status, s);
  mm8::P p{};
  const int64_t kb = (K + 127) / 128, nb = (N + 127) / 128;
  p.A = static_cast<const uint8_t*>(A8); p.sa = sa; p.lda = K; p.sa_pitch = kb;
  p.B = static_cast<const uint8_t*>(B8); p.sb = sb; p.ldb = K; p.sb_pitch = kb;
  p.b_stride = N * K; p.sb_stride = nb * kb; p.c_stride = 0;
  p.offsets = offsets; p.E = (int)E; p.T = T; p.na = 0; p.nb = (int)N; p.K = K; p.kblocks = (int)kb;
  p.columns = 0; p.out = out_dtype; p.accumulate = 0; p.C = C; p.status = dev_status;
  return mm8::run(p, s);
}

int sbp_matmul_e4m3_columns(const void* At8, const float* sat, const void* Bt8, const float* sbt,
                            const int32_t* offsets, int64_t E, int64_t T, int64_t N, int64_t K, float* dW,
                            int accumulate, int32_t* dev_status, void* stream) {
  if (E < 1 || T < 0 || N < 1 || K < 1 || (!offsets && E != 1)) return SBP_ERR_INVALID_ARG;
  if (E > MAX_GROUPS || K % 8 != 0 || N % 8 != 0 || T > (int64_t(1) << 30) || N > mm8::MAX_SIDE || K > mm8::MAX_SIDE)
    return SBP_ERR_UNSUPPORTED;
  if (!dev_status || !dW || (T > 0 && (!At8 || !sat || !Bt8 || !sbt))) return SBP_ERR_INVALID_ARG;
  const int rc = mm8::check_common(E, T, N, K, At8, sat, Bt8, sbt, offsets, dW, dev_status);
  if (rc != SBP_OK) return rc;
  NvtxRange nv("sbp_matmul_e4m3_columns");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  set_launch_count(0);
  mm8::ran(SBP_PRODUCT_NONE);
  if (T == 0) return no_rows(offsets, E, accumulate ? nullptr : dW, E * N * K, dev_status, s);
  mm8::P p{};
  const int64_t blocks = max_units(T, E, 128);
  p.A = static_cast<const uint8_t*>(At8); p.sa = sat; p.lda = blocks * 128; p.sa_pitch = blocks;
  p.B = static_cast<const uint8_t*>(Bt8); p.sb = sbt; p.ldb = blocks * 128; p.sb_pitch = blocks;
  p.b_stride = 0; p.sb_stride = 0; p.c_stride = N * K;
  p.offsets = offsets; p.E = (int)E; p.T = T; p.na = (int)N; p.nb = (int)K; p.K = blocks * 128; p.kblocks = (int)blocks;
  p.columns = 1; p.out = SBP_FP32; p.accumulate = accumulate ? 1 : 0; p.C = dW; p.status = dev_status;
  return mm8::run(p, s);
}

int sbp_last_product_kernel(void) { return mm8::g_ran; }

}  // extern "C"
