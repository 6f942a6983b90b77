// The block-scaled 8-bit product on tcgen05 (sm_103a) with the operands' parts exchanged: few rows
// an expert, many experts.
//
// What bounds such a call is reading each expert's matrix once.  An SM pair takes 256 rows of B as
// the 256 rows of its products, 32 rows of A as their columns: per block of 128 it brings in 32 KB
// of B and 4 KB of A through a ring of eleven stages, and its accumulators are 32 columns wide, so
// that sixteen blocks are in flight in tensor memory and the exchange with the epilogue warps (one
// row of B a thread, 32 sums in registers) never shows.  64 experts of 4096 x 2560, three rows each, all
// 671 MB from memory: 110 us, 6.1 TB/s; 123 with mma.sync, 145 with 256 rows of A a tile.
#include <algorithm>

#include "sbp_mm8_tc.cuh"

namespace sbp {
namespace tc {

constexpr int SW_ROWS = 32;                        // rows of A of a unit
constexpr int SW_EPI = 4, SW_THREADS = 128 + 32 * SW_EPI;
constexpr int SW_STAGES = 11, SW_BUFS = 16;
constexpr uint32_t SW_B_BYTES = 128 * 128, SW_A_BYTES = SW_ROWS / 2 * 128, SW_STAGE = SW_B_BYTES + SW_A_BYTES;
constexpr int SW_SC = 4, SW_KB = 4;                // stages of the scales' ring, blocks of each
constexpr uint32_t SW_IDESC = idesc_e4m3(256, SW_ROWS);
static_assert(SW_STAGE % 1024 == 0 && SW_BUFS * SW_ROWS <= (int)TMEM_COLS, "swizzled tiles, tensor memory");

struct SwapCtrl {
  uint64_t full[SW_STAGES], empty[SW_STAGES];
  uint64_t tfull[SW_BUFS], tempty_l[SW_BUFS], tempty_r[SW_BUFS];
  uint64_t sfull[SW_SC], sempty[SW_SC];
  uint64_t mdone;
  uint32_t tmem_base;
  int abort;
  int4 tile[SW_SC];                                // with a tile's first stage: expert, rows of A, rows of B
  float4 scale[SW_SC][SW_KB][SW_ROWS / 4];         // sa sb for each row of A
};
constexpr size_t SMEM_SWAP = SW_STAGES * SW_STAGE + sizeof(SwapCtrl) + 1024;
static_assert(SMEM_SWAP <= 232448, "shared memory budget of one CTA");

template <int OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(SW_THREADS, 1)
    k_mm8_swap(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const mm8::P p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  SwapCtrl* c = reinterpret_cast<SwapCtrl*>(base + SW_STAGES * SW_STAGE);
  const int warp = uniform_warp(), lane = threadIdx.x % 32;
  const uint32_t rank = ctarank();
  const Group first = find_unit(p.offsets, p.E, p.T, SW_ROWS, 0);
  if (first.bad) {   // the same in every thread of the grid
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = SBP_ERR_SEQLENS;
    return;
  }
  const int units = first.total, ntn = (p.nb + 255) / 256, total = units * ntn, nkb = p.kblocks;
  const int pid = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < SW_STAGES; ++i) {
      mbar_init(&c->full[i], 1);
      mbar_init(&c->empty[i], 1);
    }
    for (int i = 0; i < SW_BUFS; ++i) {
      mbar_init(&c->tfull[i], 1);
      mbar_init(&c->tempty_l[i], SW_EPI);
      mbar_init(&c->tempty_r[i], SW_EPI);
    }
    for (int i = 0; i < SW_SC; ++i) {
      mbar_init(&c->sfull[i], 1);
      mbar_init(&c->sempty[i], SW_EPI);
    }
    mbar_init(&c->mdone, 1);
    c->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&c->tmem_base)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = c->tmem_base;

  if (warp == 0) {
    uint32_t stage = 0, phase = 0, issued = 0, last = 0;   // stages in use, the parity of each one's last use
    bool ok = true;
    if (lane == 0) {
      prefetch_map(&tmA);
      prefetch_map(&tmB);
    }
    const uint32_t ring = saddr(base), fb = mapa(saddr(&c->full[0]), 0);
    for (int t = pid; t < total && ok; t += npairs) {
      const Tile o = tile_of(p, SW_ROWS, units, ntn, 256, t);
      const int arow = __shfl_sync(0xffffffffu, o.w.row0 + (int)rank * (SW_ROWS / 2), 0);
      const int brow = __shfl_sync(0xffffffffu, o.w.e * p.nb + o.n0 + (int)rank * 128, 0);
      for (int kb = 0; kb < nkb; ++kb) {
        ok = warp_wait<false>(&c->empty[stage], phase ^ 1u, c, p.limit_ns);
        if (!ok) break;
        if (elect_one()) {
          const uint32_t sb = ring + stage * SW_STAGE, bar = fb + stage * (uint32_t)sizeof(uint64_t);
          if (rank == 0) mbar_expect_tx(&c->full[stage], 2 * SW_STAGE);
          tma_load_2d_pair(sb, &tmB, bar, kb * 128, brow);
          tma_load_2d_pair(sb + SW_B_BYTES, &tmA, bar, kb * 128, arow);
        }
        issued |= 1u << stage;
        last = (last & ~(1u << stage)) | (phase << stage);
        if (++stage == SW_STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    if (!ok) {
      if (lane == 0) fail_mm8(c, p.status);
      if (rank == 0) {   // no copy may be in flight when the block ends
        for (int i = 0; i < SW_STAGES; ++i)
          if (issued & (1u << i)) wait_inl<false>(&c->full[i], (last >> i) & 1u, nullptr, 200000000ull);
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    if (rank == 0) {
      uint32_t stage = 0, phase = 0, it = 0;   // it: blocks multiplied so far
      bool ok = !p.stall || warp_wait<false>(&c->mdone, 0, c, p.limit_ns);
      for (int t = pid; t < total && ok; t += npairs) {
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const uint32_t buf = it % SW_BUFS, ep = ((it / SW_BUFS) & 1u) ^ 1u;
          // the tests go out together; only what is not there yet is waited for
          const bool tl = mbar_test<false>(&c->tempty_l[buf], ep), tr = mbar_test<true>(&c->tempty_r[buf], ep);
          const bool tf = mbar_test<false>(&c->full[stage], phase);
          if (!__all_sync(0xffffffffu, tl && tr && tf))
            ok = warp_wait<false>(&c->tempty_l[buf], ep, c, p.limit_ns) &&
                 warp_wait<true>(&c->tempty_r[buf], ep, c, p.limit_ns) &&
                 warp_wait<false>(&c->full[stage], phase, c, p.limit_ns);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t sb = saddr(base) + stage * SW_STAGE, sa = sb + SW_B_BYTES;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma2_e4m3(tmem + buf * SW_ROWS, sw128_desc(sb + k * 32, 16, 1024), sw128_desc(sa + k * 32, 16, 1024),
                        SW_IDESC, k != 0);
            commit2_mc(&c->tfull[buf], 3);
            commit2_mc(&c->empty[stage], 3);
          }
          __syncwarp();
          if (++stage == SW_STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (lane == 0 && !ok) fail_mm8(c, p.status);
      __syncwarp();
      if (elect_one()) commit2_mc(&c->mdone, 1);
      wait_inl<false>(&c->mdone, 0, nullptr, 200000000ull);
      __syncwarp();
    }
  } else if (warp == 2) {
    // scales: a row of A a lane, times that of this CTA's 128 rows of B
    uint32_t n = 0;
    bool ok = true;
    for (int t = pid; t < total && ok; t += npairs) {
      const Tile o = tile_of(p, SW_ROWS, units, ntn, 256, t);
      const float* sa = p.sa + (int64_t)(o.w.row0 + min(lane, o.w.rows - 1)) * p.sa_pitch;
      const float* sb = p.sb + (int64_t)o.w.e * p.sb_stride +
                        (int64_t)min(o.n0 / 128 + (int)rank, (p.nb - 1) / 128) * p.sb_pitch;
      for (int kb = 0; kb < nkb; kb += SW_KB, ++n) {
        const uint32_t s = n % SW_SC;
        float v[SW_KB];
#pragma unroll
        for (int k = 0; k < SW_KB; ++k) v[k] = kb + k < nkb ? sa[kb + k] * sb[kb + k] : 0.f;
        ok = warp_wait<false>(&c->sempty[s], ((n / SW_SC) & 1u) ^ 1u, c, p.limit_ns);
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < SW_KB; ++k) reinterpret_cast<float*>(c->scale[s][k])[lane] = v[k];
        if (lane == 0 && kb == 0) c->tile[s] = make_int4(o.w.e, o.w.row0, o.w.rows, o.n0);
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->sfull[s]);
      }
    }
    if (!ok && lane == 0) fail_mm8(c, p.status);
  } else if (warp >= 4) {
    const int q = warp & 3;
    const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16);
    const bool p0 = lane == 0 && rank == 0, p1 = lane == 0 && rank != 0;
    const uint32_t rel_l = saddr(&c->tempty_l[0]), rel_r = mapa(saddr(&c->tempty_r[0]), 0);
    uint32_t it = 0, n = 0;   // blocks so far, stages of scales so far
    bool ok = true;
    for (int t = pid; t < total && ok; t += npairs) {
      float acc[SW_ROWS];
#pragma unroll
      for (int i = 0; i < SW_ROWS; ++i) acc[i] = 0.f;
      int4 tile;
      for (int kb = 0; kb < nkb; kb += SW_KB, ++n) {
        const uint32_t ss = n % SW_SC;
        ok = wait_inl<false>(&c->sfull[ss], (n / SW_SC) & 1u, &c->abort, p.limit_ns) && ok;
        if (kb == 0) {
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;   // (nothing came)
          tile = c->tile[ss];
        }
        __syncwarp();
        const int some = min(SW_KB, nkb - kb);
        for (int k = 0; k < some; ++k, ++it) {
          const uint32_t buf = it % SW_BUFS;
          ok = wait_inl<false>(&c->tfull[buf], (it / SW_BUFS) & 1u, &c->abort, p.limit_ns) && ok;
          __syncwarp();
          tc_fence_after();
          uint32_t r[SW_ROWS];
          tmem_ld32(tb + buf * SW_ROWS, r);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          arrive_if(p0, rel_l + buf * 8, p1, rel_r + buf * 8);
          const float4* sc = c->scale[ss][k];
#pragma unroll
          for (int i = 0; i < SW_ROWS / 4; ++i) {
            if (i % 2 == 0 && 4 * i >= tile.z) break;   // (no rows from here on)
            const float4 s = sc[i];
            acc[4 * i] = fmaf(__uint_as_float(r[4 * i]), s.x, acc[4 * i]);
            acc[4 * i + 1] = fmaf(__uint_as_float(r[4 * i + 1]), s.y, acc[4 * i + 1]);
            acc[4 * i + 2] = fmaf(__uint_as_float(r[4 * i + 2]), s.z, acc[4 * i + 2]);
            acc[4 * i + 3] = fmaf(__uint_as_float(r[4 * i + 3]), s.w, acc[4 * i + 3]);
          }
        }
        __syncwarp();
        arrive_if(lane == 0, saddr(&c->sempty[ss]), false, 0);
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) fail_mm8(c, p.status);
        break;
      }
      // a thread has one column of C: a warp writes 32 neighbouring ones of each row
      const int col = tile.w + (int)rank * 128 + q * 32 + lane;
      if (col < p.nb) {
        const int64_t at = (int64_t)tile.y * p.nb + col;
#pragma unroll
        for (int i = 0; i < SW_ROWS; ++i) {
          if (i >= tile.z) break;
          if (OUT == SBP_BF16) static_cast<__nv_bfloat16*>(p.C)[at + (int64_t)i * p.nb] = __float2bfloat16_rn(acc[i]);
          else static_cast<float*>(p.C)[at + (int64_t)i * p.nb] = acc[i];
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(c->tmem_base), "r"(TMEM_COLS)
                 : "memory");
  }
}

}  // namespace tc

namespace mm8 {

template <int OUT>
cudaError_t launch_swap(const P& p, cudaStream_t s) {
  using namespace tc;
  static int attr_state[64] = {};
  static std::mutex mu;
  const auto kern = k_mm8_swap<OUT>;
  if (!once_per_device(attr_state, mu, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_SWAP) == cudaSuccess;
      }))
    return cudaErrorInvalidConfiguration;
  CUtensorMap mA, mB;
  if (!make_map_u8(&mA, p.A, (uint64_t)p.K, (uint64_t)p.T, (uint64_t)p.lda, SW_ROWS / 2) ||
      !make_map_u8(&mB, p.B, (uint64_t)p.K, (uint64_t)p.E * p.nb, (uint64_t)p.ldb, 128))
    return cudaErrorInvalidValue;
  if (cudaMemsetAsync(p.status, 0, sizeof(int32_t), s) != cudaSuccess) return cudaErrorUnknown;
  P q = p;
  q.limit_ns = wait_limit_ns();
  q.stall = fault_stall_requested();
  const int64_t tiles = max_units(p.T, p.E, SW_ROWS) * ((p.nb + 255) / 256);
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  const int pairs = (int)std::min<int64_t>(max_pairs((const void*)kern, SMEM_SWAP, SW_THREADS), tiles);
  kern<<<2 * pairs, SW_THREADS, SMEM_SWAP, s>>>(mA, mB, q);
  ran(SBP_PRODUCT_SWAP);
  return cudaGetLastError();
}

// A pair takes 310 ns for a block of 128 of its 256 rows of B where memory keeps up (32 rows x 4096 x
// 12288: 36.7 us), and memory gives 6.0 TB/s, uneven last rounds included (8 experts of 4096 x 4096:
// 30.7 us, 64 of 4096 x 2560: 107).
int64_t swap_ns(const P& p) {
  const int64_t tiles = about_units(p, 32) * ((p.nb + 255) / 256), pairs = num_sms() / 2;
  const int64_t bytes = std::min<int64_t>(p.E, p.T) * p.nb * p.K;
  return 7400 + std::max((tiles + pairs - 1) / pairs * about_blocks(p) * 310, bytes / 6000);
}

cudaError_t swap(const P& p, cudaStream_t s) {
  return p.out == SBP_BF16 ? launch_swap<SBP_BF16>(p, s) : launch_swap<SBP_FP32>(p, s);
}

}  // namespace mm8
}  // namespace sbp
