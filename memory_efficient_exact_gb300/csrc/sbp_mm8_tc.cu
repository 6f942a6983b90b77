// The block-scaled 8-bit product on tcgen05 (sm_103a): many rows.
//
// SM pairs compute 256 x 256 tiles of C; one stage of the operand ring is one block of 128 of the
// sum, which is also one 128-byte swizzled row.  Tensor memory holds one block's sum at a time, in
// two buffers: the epilogue warps read each block's 128 x 256 accumulators out, scale them by
// sa[row] sb[column block] and add them to the tile's sums, which stay in their registers (128 a
// thread), while the next block is multiplied.  Roles, pair protocol and bounded waits are those
// of the LM-head kernels.
#include "sbp_mm8.cuh"
#include "sbp_rows.cuh"
#include "sbp_tc_common.cuh"

namespace sbp {
namespace tc {

// Instruction descriptor of tcgen05.mma kind::f8f6f4: D fp32 (bits 4-5 = 1), A and B e4m3 (bits
// 7-9 and 10-12 = 0), both K-major, N >> 3 at bit 17, M >> 4 at bit 24.
constexpr uint32_t IDESC_E4M3 = (1u << 4) | (uint32_t(256 >> 3) << 17) | (uint32_t(256 >> 4) << 24);

__device__ __forceinline__ void mma2_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(
          d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// Warp 0 loads, warp 1 multiplies, warps 4 to 19 are the epilogue's: 32 rows x 64 columns each, so
// that a thread's 64 sums fit into the 96 registers that 640 threads may have.
constexpr int MM8_EPI = 16, MM8_THREADS = 128 + 32 * MM8_EPI;

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

constexpr uint32_t STG_MM8 = 32 * 64;   // a warp's staging block: 32 rows of 64 bytes
constexpr size_t SMEM_MM8 = STAGES * STAGE_BYTES + MM8_EPI * STG_MM8 + sizeof(Ctrl) + 1024;
static_assert(SMEM_MM8 <= 232448, "shared memory budget of one CTA");
// Tiles are walked in bands of this many units of 256 rows, all columns of a band before the next:
// the 76 pairs' tiles then share 8 blocks of A's rows and 9 or 10 of B's.
constexpr int BAND = 8;

struct Tile {
  mm8::Unit w;
  int n0;
};
__device__ __forceinline__ Tile tile_of(const mm8::P& p, int units, int ntn, int t) {
  const int band = t / (BAND * ntn), r = t - band * BAND * ntn;
  const int high = min(BAND, units - band * BAND);
  Tile o;
  o.w = mm8::unit_of(p, 256, band * BAND + r % high);
  o.n0 = r / high * BN;
  return o;
}

template <int OUT, bool ACC>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(MM8_THREADS, 1)
    k_mm8(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const mm8::P p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stg_base = base + STAGES * STAGE_BYTES;
  Ctrl* c = reinterpret_cast<Ctrl*>(stg_base + MM8_EPI * STG_MM8);
  const int warp = uniform_warp(), lane = threadIdx.x % 32;
  const uint32_t rank = ctarank();
  const Group first = find_unit(p.offsets, p.E, p.T, p.columns ? 128 : 256, 0);
  if (first.bad) {   // the same in every thread of the grid
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = SBP_ERR_SEQLENS;
    return;
  }
  const int units = p.columns ? p.E * ((p.na + 255) / 256) : first.total;
  const int ntn = (p.nb + BN - 1) / BN;
  const int total = units * ntn;
  const int pid = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  prologue(c, warp, MM8_EPI);
  const uint32_t tmem = c->tmem_base;

  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0, issued = 0, last = 0;   // stages in use, the parity of each one's last use
    if (lane == 0) {
      prefetch_map(&tmA);
      prefetch_map(&tmB);
    }
    for (int t = pid; t < total; t += npairs) {
      const Tile o = tile_of(p, units, ntn, t);
      bool ok = true;
      if (lane == 0) {
        const int arow = o.w.row0 + (int)rank * 128;
        const int brow = (p.columns ? 0 : o.w.e * p.nb) + o.n0 + (int)rank * 128;
        for (int kb = o.w.kb0; kb < o.w.kb1; ++kb) {
          if (!wait_inl<false>(&c->empty[stage], phase ^ 1u, &c->abort, p.limit_ns)) { ok = false; break; }
          const uint32_t sa = saddr(base + stage * STAGE_BYTES), sb = sa + A_BYTES;
          const uint32_t fb = mapa(saddr(&c->full[stage]), 0);
          if (rank == 0) mbar_expect_tx(&c->full[stage], PAIR_TX);
          tma_load_2d_pair(sa, &tmA, fb, kb * 128, arow);
          tma_load_2d_pair(sb, &tmB, fb, kb * 128, brow);
          issued |= 1u << stage;
          last = (last & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) {
          fail(c, p.status);
          if (rank == 0) {   // no copy may be in flight when the block ends
#pragma unroll
            for (int i = 0; i < STAGES; ++i)
              if (issued & (1u << i)) wait_inl<false>(&c->full[i], (last >> i) & 1u, nullptr, 200000000ull);
          }
        }
      }
      if (!__shfl_sync(0xffffffffu, (int)ok, 0)) break;
    }
  } else if (warp == 1) {
    if (rank == 0) {
      int stage = 0;
      uint32_t phase = 0, it = 0;   // it: blocks multiplied so far
      bool ok = true;
      for (int t = pid; t < total && ok; t += npairs) {
        const Tile o = tile_of(p, units, ntn, t);
        for (int kb = o.w.kb0; kb < o.w.kb1; ++kb, ++it) {
          const int buf = it & 1;
          ok = wait_inl<true>(&c->tempty[buf], ((it >> 1) & 1u) ^ 1u, &c->abort, p.limit_ns) &&
               wait_inl<false>(&c->full[stage], phase, &c->abort, p.limit_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (lane == 0) {
            const uint32_t sa = saddr(base + stage * STAGE_BYTES), sb = sa + A_BYTES;
            const uint32_t dt = tmem + (uint32_t)(buf * BN);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma2_e4m3(dt, sw128_desc(sa + k * 32, 16, 1024), sw128_desc(sb + k * 32, 16, 1024), IDESC_E4M3, k != 0);
            commit2_mc(&c->empty[stage], 3);
            commit2_mc(&c->tfull[buf], 3);
          }
          __syncwarp();
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (lane == 0) {
        if (!ok) fail(c, p.status);
        commit2_mc(&c->mdone, 1);
        wait_inl<false>(&c->mdone, 0, nullptr, 200000000ull);
      }
      __syncwarp();
    }
  } else if (warp >= 4) {
    const int q = warp & 3, h = (warp - 4) >> 2;
    const uint32_t stg = saddr(stg_base + (warp - 4) * STG_MM8);
    const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(h * 64);
    const uint32_t te0 = mapa(saddr(&c->tempty[0]), 0), te1 = mapa(saddr(&c->tempty[1]), 0);
    uint32_t it = 0;
    bool ok = true;
    for (int t = pid; t < total && ok; t += npairs) {
      const Tile o = tile_of(p, units, ntn, t);
      const int r0 = (int)rank * 128 + q * 32;            // this warp's first row of the unit
      const int rows = min(32, o.w.rows - r0);            // how many of them are (may be none)
      const float* sa = p.sa + (int64_t)(o.w.row0 + min(r0 + lane, o.w.rows - 1)) * p.sa_pitch;
      const int nb128 = min(o.n0 / 128 + h / 2, (p.nb - 1) / 128);
      const float* sb = p.sb + (int64_t)o.w.e * p.sb_stride + (int64_t)nb128 * p.sb_pitch;
      float2 acc[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) acc[i] = make_float2(0.f, 0.f);
      // scales two blocks ahead
      const int k0 = o.w.kb0, k1 = o.w.kb1;
      float s0 = k0 < k1 ? sa[k0] * sb[k0] : 0.f;
      float a1 = k0 + 1 < k1 ? sa[k0 + 1] : 0.f, b1 = k0 + 1 < k1 ? sb[k0 + 1] : 0.f;
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const float s = s0;
        s0 = a1 * b1;
        if (kb + 2 < k1) {
          a1 = sa[kb + 2];
          b1 = sb[kb + 2];
        }
        const int buf = it & 1;
        ok = __all_sync(0xffffffffu, wait_inl<true>(&c->tfull[buf], (it >> 1) & 1u, &c->abort, p.limit_ns));
        if (!ok) break;
        tc_fence_after();
        const float2 s2 = make_float2(s, s);
        const uint32_t tc = tb + (uint32_t)(buf * BN);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t r[16];
          tmem_ld16(tc + (uint32_t)(16 * j), r);
          tmem_ld_wait();
          if (j == 3) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_remote(buf ? te1 : te0);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            acc[8 * j + i] = fma2(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), s2, acc[8 * j + i]);
        }
      }
      if (!ok) {
        if (lane == 0) fail(c, p.status);
        break;
      }
      // the tile's sums leave through the staging block, so that a warp writes 64-byte pieces of
      // eight rows at a time (rows past the unit's last are masked); 16-byte chunk k of row r lies
      // at chunk k ^ (r / 2 % 4), without bank conflicts either way
      constexpr int ES = OUT == SBP_BF16 ? 2 : 4, PASS = 64 / ES;   // columns a pass
#pragma unroll
      for (int g = 0; g < 64 / PASS; ++g) {
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (OUT == SBP_BF16) {
              const float2 f = acc[g * PASS / 2 + 4 * k + i];
              v[i] = pack_bf16(f.x, f.y);
            } else {
              const float2 f = acc[g * PASS / 2 + 2 * k + i / 2];
              v[i] = __float_as_uint(i & 1 ? f.y : f.x);
            }
          }
          sts128(stg + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4), v[0], v[1], v[2], v[3]);
        }
        __syncwarp();
        const int col = o.n0 + h * 64 + g * PASS + (lane % 4) * (16 / ES);
        uint8_t* out = static_cast<uint8_t*>(p.C) +
                       ((int64_t)o.w.e * p.c_stride + (int64_t)(o.w.row0 + r0 + lane / 4) * p.nb + col) * ES;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 8 + lane / 4;
          uint32_t v[4];
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                       : "r"(stg + r * 64 + (((lane % 4) ^ ((r >> 1) & 3)) << 4))
                       : "memory");
          if (r < rows && col < p.nb) {
            if (ACC) {
              const float4 old = *reinterpret_cast<const float4*>(out);
              *reinterpret_cast<float4*>(out) = make_float4(old.x + __uint_as_float(v[0]), old.y + __uint_as_float(v[1]),
                                                            old.z + __uint_as_float(v[2]), old.w + __uint_as_float(v[3]));
            } else {
              *reinterpret_cast<uint4*>(out) = make_uint4(v[0], v[1], v[2], v[3]);
            }
          }
          out += (int64_t)8 * p.nb * ES;
        }
      }
    }
  }
  teardown(c, warp);
}

// Map over a row-major array of bytes, 128 x 128 boxes, 128-byte swizzle, zeros outside.
inline bool make_map_u8(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer, uint64_t pitch) {
  auto enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {pitch};
  cuuint32_t box[2] = {128, 128};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc

namespace mm8 {

cudaError_t many(const P& p, cudaStream_t s) {
  using namespace tc;
  static int attr_state[64] = {};
  static std::mutex mu;
  if (!once_per_device(attr_state, mu, [] {
        const void* ks[] = {(const void*)k_mm8<SBP_BF16, false>, (const void*)k_mm8<SBP_FP32, false>,
                            (const void*)k_mm8<SBP_FP32, true>};
        for (const void* k : ks)
          if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_MM8) != cudaSuccess)
            return false;
        return true;
      }))
    return cudaErrorInvalidConfiguration;
  CUtensorMap mA, mB;
  if (!make_map_u8(&mA, p.A, (uint64_t)p.K, (uint64_t)(p.columns ? p.na : p.T), (uint64_t)p.lda) ||
      !make_map_u8(&mB, p.B, (uint64_t)p.K, p.columns ? (uint64_t)p.nb : (uint64_t)p.E * p.nb, (uint64_t)p.ldb))
    return cudaErrorInvalidValue;
  if (cudaMemsetAsync(p.status, 0, sizeof(int32_t), s) != cudaSuccess) return cudaErrorUnknown;
  P q = p;
  q.limit_ns = wait_limit_ns();
  const void* kern = p.out == SBP_BF16 ? (const void*)k_mm8<SBP_BF16, false>
                     : p.accumulate    ? (const void*)k_mm8<SBP_FP32, true>
                                       : (const void*)k_mm8<SBP_FP32, false>;
  const int64_t units = p.columns ? (int64_t)p.E * ((p.na + 255) / 256) : max_units(p.T, p.E, 256);
  const int64_t tiles = units * ((p.nb + BN - 1) / BN);
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  int pairs = max_pairs(kern, SMEM_MM8, MM8_THREADS);
  if (pairs > tiles) pairs = (int)tiles;
  if (p.out == SBP_BF16) k_mm8<SBP_BF16, false><<<2 * pairs, MM8_THREADS, SMEM_MM8, s>>>(mA, mB, q);
  else if (p.accumulate) k_mm8<SBP_FP32, true><<<2 * pairs, MM8_THREADS, SMEM_MM8, s>>>(mA, mB, q);
  else k_mm8<SBP_FP32, false><<<2 * pairs, MM8_THREADS, SMEM_MM8, s>>>(mA, mB, q);
  return cudaGetLastError();
}

}  // namespace mm8
}  // namespace sbp
