// The block-scaled 8-bit product on tcgen05 (sm_103a): many rows.
//
// SM pairs compute tiles of 256 rows x 128 HALVES columns of C; one stage of the operand ring is one
// block of 128 of the sum, which is also one 128-byte swizzled row.  Tensor memory holds sums of
// single blocks, four accumulators of 128 columns in turn: the epilogue warps read each out, give
// it back, and add it, times sa[row] sb[column block], to the tile's sums in their registers.
//
// What bounds it is not the products (512 cycles a block of a 256 x 256 tile) but this exchange:
// 512 columns of tensor memory are in flight, and an accumulator takes some 2000 cycles from the
// products' issue over the commit, the read and the arrival of both CTAs' warps to the next issue,
// so 1000 a block.  Hence the shape of the loops: two warps issue, so that one tests its barriers
// while the other's products run; with tiles of 256 columns the two epilogue warps of a scheduler
// take different accumulators, so that one adds while the other waits and loads; an epilogue warp
// asks for 64 columns at once and releases an accumulator before it adds its last ones up; its loop
// is unrolled over the accumulators with no branches but the waits'; the scales are multiplied and
// put in place by a warp of their own.  16384 x 24576 x 4096: 4130 us with two accumulators of 256
// columns, 16 epilogue warps that loaded 16 columns at a time and scales read by each; 1785 with
// four accumulators of 128 and the scales' warp; 1717 with two issuing warps; 1383 with eight
// epilogue warps of 224 registers and the unrolled loop; 1350 with the scales multiplied in advance;
// 1285 with accumulators of their own (2570 TFLOP/s).  All of these with the same inputs throughout; with
// other inputs from call to call, at the power cap, the last form takes 1300 to 1420 (2540 to 2320
// TFLOP/s).  Not faster: packed additions of two values (1599 against 1620 TFLOP/s in an earlier form), 16
// epilogue warps (1405 against 1355), the next columns' load before these are added (1352 against 1290).
#include <algorithm>

#include "sbp_mm8_tc.cuh"

namespace sbp {
namespace tc {

// Warp 0 loads the operands, warps 1 and 2 multiply, warp 3 loads the scales, warps 4 to 11 are the
// epilogue's: 32 rows x 64 columns of each accumulator, or x 128 of every other one.  The block's
// 12 x 32 threads are launched with 168 registers each; the epilogue's 128 sums and 64 values in
// flight need more, so the first four warps hand theirs over.  (Waits are inlined: a call would not
// know of the split.)  The split leaves the first four warps short: the compiler spills 104 bytes a
// thread and loads 152 back in the forms of 256 columns, 304 in those of 128.
constexpr int MM8_EPI = 8, MM8_THREADS = 128 + 32 * MM8_EPI;
constexpr int REGS_LAUNCH = 168, REGS_FEW = 56, REGS_MANY = 224;
static_assert(128 * REGS_FEW + 32 * MM8_EPI * REGS_MANY <= MM8_THREADS * REGS_LAUNCH, "no more than the block has");

// blocks of 128 of both operands in shared memory: 32 KB each, or 24 KB with half the columns
constexpr int mm8_stages(int halves) { return halves == 2 ? 6 : 8; }
constexpr uint32_t mm8_stage_bytes(int halves) { return A_BYTES + halves * B_BYTES / 2; }
constexpr int BUFS = 4, BUF_N = 128;     // accumulators of one block: 128 columns each
constexpr int SC_KB = 4;                 // blocks of a stage of the scales' ring
constexpr uint32_t STG_MM8 = 16 * 128;   // a warp's staging block: 16 rows of 128 bytes
constexpr uint32_t IDESC_E4M3 = idesc_e4m3(256, BUF_N);

struct Mm8Ctrl {
  uint64_t full[8], empty[8];
  uint64_t tfull[BUFS], tempty_l[BUFS], tempty_r[BUFS];   // released by the leader's own warps, by the other CTA's
  uint64_t sfull[2], sempty[2];
  uint64_t mdone[2];
  uint32_t tmem_base;
  int abort;
  float4 scale[2][2][128];   // [stage][column block][row]: SC_KB blocks
  int4 tile[2][2];           // with a tile's first stage: its expert, rows, columns and blocks
};
constexpr size_t SMEM_MM8 = 6 * STAGE_BYTES + MM8_EPI * STG_MM8 + sizeof(Mm8Ctrl) + 1024;
static_assert(mm8_stages(1) * mm8_stage_bytes(1) == 6 * STAGE_BYTES && mm8_stages(2) * mm8_stage_bytes(2) == 6 * STAGE_BYTES &&
                  SMEM_MM8 <= 232448,
              "shared memory budget of one CTA");

template <int HALVES, int OUT, bool ACC>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(MM8_THREADS, 1)
    k_mm8(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const mm8::P p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int MM8_STAGES = mm8_stages(HALVES);
  constexpr uint32_t STAGE = mm8_stage_bytes(HALVES);
  uint8_t* stg_base = base + MM8_STAGES * STAGE;
  Mm8Ctrl* c = reinterpret_cast<Mm8Ctrl*>(stg_base + MM8_EPI * STG_MM8);
  const int warp = uniform_warp(), lane = threadIdx.x % 32;
  const uint32_t rank = ctarank();
  const Group first = find_unit(p.offsets, p.E, p.T, p.columns ? 128 : 256, 0);
  if (first.bad) {   // the same in every thread of the grid
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = SBP_ERR_SEQLENS;
    return;
  }
  const int units = p.columns ? p.E * ((p.na + 255) / 256) : first.total;
  const int ntn = (p.nb + 128 * HALVES - 1) / (128 * HALVES);
  const int total = units * ntn;
  const int pid = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < MM8_STAGES; ++i) {
      mbar_init(&c->full[i], 1);
      mbar_init(&c->empty[i], HALVES);
    }
    for (int i = 0; i < BUFS; ++i) {
      mbar_init(&c->tfull[i], 1);
      mbar_init(&c->tempty_l[i], MM8_EPI / HALVES);
      mbar_init(&c->tempty_r[i], MM8_EPI / HALVES);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c->sfull[i], 1);
      mbar_init(&c->mdone[i], 1);
      mbar_init(&c->sempty[i], MM8_EPI);
    }
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

  // The accumulators a block uses: buffers HALVES g and on, group g counting from 0 with each tile.
  constexpr int GROUPS = BUFS / HALVES;
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_FEW));
    if (warp == 0) {
      // (the warp stays converged and one elected lane issues, with operands that the compiler can
      // keep uniform)
      uint32_t stage = 0, phase = 0, issued = 0, last = 0;   // stages in use, the parity of each one's last use
      bool ok = true;
      if (lane == 0) {
        prefetch_map(&tmA);
        prefetch_map(&tmB);
      }
      const uint32_t ring = saddr(base), fb = mapa(saddr(&c->full[0]), 0);
      for (int t = pid; t < total && ok; t += npairs) {
        const Tile o = tile_of(p, 256, units, ntn, 128 * HALVES, t);
        const int arow = __shfl_sync(0xffffffffu, o.w.row0 + (int)rank * 128, 0);
        // of each 128 of the tile's columns, this CTA's 64 rows of B
        const int brow = __shfl_sync(0xffffffffu, (p.columns ? 0 : o.w.e * p.nb) + o.n0 + (int)rank * 64, 0);
        const int kb1 = __shfl_sync(0xffffffffu, o.w.kb1, 0);
        for (int kb = __shfl_sync(0xffffffffu, o.w.kb0, 0); kb < kb1; ++kb) {
          ok = warp_wait<false>(&c->empty[stage], phase ^ 1u, c, p.limit_ns);
          if (!ok) break;
          if (elect_one()) {
            const uint32_t sa = ring + stage * STAGE, sb = sa + A_BYTES, bar = fb + stage * (uint32_t)sizeof(uint64_t);
            if (rank == 0) mbar_expect_tx(&c->full[stage], 2 * STAGE);
            tma_load_2d_pair(sa, &tmA, bar, kb * 128, arow);
            tma_load_2d_pair(sb, &tmB, bar, kb * 128, brow);
            if (HALVES == 2) tma_load_2d_pair(sb + B_BYTES / 2, &tmB, bar, kb * 128, brow + 128);
          }
          issued |= 1u << stage;
          last = (last & ~(1u << stage)) | (phase << stage);
          if (++stage == MM8_STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {
        if (lane == 0) fail_mm8(c, p.status);
        if (rank == 0) {   // no copy may be in flight when the block ends
          for (int i = 0; i < MM8_STAGES; ++i)
            if (issued & (1u << i)) wait_inl<false>(&c->full[i], (last >> i) & 1u, nullptr, 200000000ull);
        }
        __syncwarp();
      }
    } else if (warp < 3) {
      // Two warps issue: one the first 128 columns of each tile and the other the second, or, with
      // one accumulator a block, every other block.  While one's products run, the other tests its
      // barriers.
      if (rank == 0) {
        const int j = warp - 1;
        uint32_t done = 0, use = 15;   // blocks of the tiles before; the parity of each group's last release
        bool ok = !p.stall || warp_wait<false>(&c->mdone[j], 0, c, p.limit_ns);
        for (int t = pid; t < total && ok; t += npairs) {
          const Tile o = tile_of(p, 256, units, ntn, 128 * HALVES, t);
          const int nkb = o.w.kb1 - o.w.kb0;
          for (int kb = HALVES == 2 ? 0 : j; kb < nkb; kb += HALVES == 2 ? 1 : 2) {
            const uint32_t n = done + kb, stage = n % MM8_STAGES, phase = (n / MM8_STAGES) & 1u;
            const uint32_t sa = saddr(base + stage * STAGE), sb = sa + A_BYTES + (HALVES == 2 ? j * (B_BYTES / 2) : 0);
            const uint32_t g = (uint32_t)kb % GROUPS, buf = HALVES == 2 ? HALVES * g + j : g, ep = (use >> g) & 1u;
            use ^= 1u << g;
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
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma2_e4m3(tmem + buf * BUF_N, sw128_desc(sa + k * 32, 16, 1024), sw128_desc(sb + k * 32, 16, 1024),
                          IDESC_E4M3, k != 0);
              commit2_mc(&c->tfull[buf], 3);
              commit2_mc(&c->empty[stage], 3);
            }
            __syncwarp();
          }
          done += (uint32_t)nkb;
        }
        if (lane == 0 && !ok) fail_mm8(c, p.status);
        __syncwarp();
        if (elect_one()) commit2_mc(&c->mdone[j], 1);
        wait_inl<false>(&c->mdone[j], 0, nullptr, 200000000ull);
        __syncwarp();
      }
    } else {
      // scales: SC_KB blocks of this CTA's 128 rows at a time, four rows a lane, times those of the
      // tile's column blocks.  All loads of a stage are in flight together, before its place is
      // waited for: with a row after the other they took 1000 cycles a block and set the pace.
      uint32_t n = 0;
      bool ok = true;
      const bool quads = p.sa_pitch % SC_KB == 0 && reinterpret_cast<uintptr_t>(p.sa) % 16 == 0;
      for (int t = pid; t < total && ok; t += npairs) {
        const Tile o = tile_of(p, 256, units, ntn, 128 * HALVES, t);
        const float* sa[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sa[i] = p.sa + (int64_t)(o.w.row0 + min((int)rank * 128 + lane + 32 * i, o.w.rows - 1)) * p.sa_pitch;
        const float* sb0 = p.sb + (int64_t)o.w.e * p.sb_stride + (int64_t)(o.n0 / 128) * p.sb_pitch;
        const float* sb1 = HALVES == 2 && o.n0 + 128 < p.nb ? sb0 + p.sb_pitch : sb0;
        // (a tile without blocks has a stage too, which says so)
        for (int kb = o.w.kb0; kb < o.w.kb1 || kb == o.w.kb0; kb += SC_KB, ++n) {
          const uint32_t s = n & 1u;
          const int left = o.w.kb1 - kb;
          auto four = [&](const float* q) {
            return make_float4(left > 0 ? q[0] : 0.f, left > 1 ? q[1] : 0.f, left > 2 ? q[2] : 0.f, left > 3 ? q[3] : 0.f);
          };
          float4 x[4];
          if (quads && kb % SC_KB == 0 && left >= SC_KB) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(sa[i] + kb);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = four(sa[i] + kb);
          }
          const float4 b0 = four(sb0 + kb), b1 = HALVES == 2 ? four(sb1 + kb) : b0;
          ok = warp_wait<false>(&c->sempty[s], ((n >> 1) & 1u) ^ 1u, c, p.limit_ns);
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            c->scale[s][0][lane + 32 * i] = make_float4(x[i].x * b0.x, x[i].y * b0.y, x[i].z * b0.z, x[i].w * b0.w);
            if (HALVES == 2)
              c->scale[s][1][lane + 32 * i] = make_float4(x[i].x * b1.x, x[i].y * b1.y, x[i].z * b1.z, x[i].w * b1.w);
          }
          if (lane == 0 && kb == o.w.kb0) {
            c->tile[s][0] = make_int4(o.w.e, o.w.row0, o.w.rows, o.n0);
            c->tile[s][1] = make_int4(o.w.kb1 - o.w.kb0, 0, 0, 0);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&c->sfull[s]);
        }
      }
      if (!ok && lane == 0) fail_mm8(c, p.status);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_MANY));
    // warps 4 to 7: the first 128 columns of the tile (the first 64, where there are 128), warps 8 to
    // 11: the second
    const int q = warp & 3, h = (warp - 4) >> 2;
    const uint32_t stg = saddr(stg_base + (warp - 4) * STG_MM8);
    const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(HALVES == 2 ? 0 : h * 64);
    // where this warp's lane 0 says that it has read an accumulator: on the leader's barrier for its
    // own warps or for the other CTA's
    const bool p0 = lane == 0 && rank == 0, p1 = lane == 0 && rank != 0;
    const uint32_t rel_l = saddr(&c->tempty_l[0]), rel_r = mapa(saddr(&c->tempty_r[0]), 0);
    uint32_t n = 0, use = 0;   // stages of scales so far; the parity of each group's next accumulators
    bool ok = true;
    for (int t = pid; t < total && ok; t += npairs) {
      float acc[HALVES][64];
#pragma unroll
      for (int j = 0; j < HALVES; ++j)
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[j][i] = 0.f;
      int4 tile;
      int nkb = 1;
      for (int kb = 0; kb < nkb; kb += SC_KB, ++n) {
        const uint32_t ss = n & 1u;
        ok = wait_inl<false>(&c->sfull[ss], (n >> 1) & 1u, &c->abort, p.limit_ns) && ok;
        if (kb == 0) {   // what the tile is comes with its first scales, not from the table again
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;   // (nothing came)
          tile = c->tile[ss][0];
          nkb = c->tile[ss][1].x;
        }
        const float4 sv = c->scale[ss][HALVES == 2 ? h : 0][q * 32 + lane];
        const float sk[SC_KB] = {sv.x, sv.y, sv.z, sv.w};
        __syncwarp();
        arrive_if(lane == 0, saddr(&c->sempty[ss]), false, 0);
#pragma unroll
        for (int k = 0; k < SC_KB; ++k) {
          if (kb + k >= nkb) break;
          constexpr uint32_t S = sizeof(uint64_t);
          const uint32_t g = k % GROUPS, buf = HALVES == 2 ? 2 * g + h : g;
          ok = wait_inl<false>(&c->tfull[buf], (use >> g) & 1u, &c->abort, p.limit_ns) && ok;
          __syncwarp();
          tc_fence_after();
#pragma unroll
          for (int j = 0; j < HALVES; ++j) {
            uint32_t r[2][32];
            tmem_ld32(tb + buf * BUF_N + 64 * j, r[0]);
            tmem_ld32(tb + buf * BUF_N + 64 * j + 32, r[1]);
            tmem_ld_wait();
            if (j == HALVES - 1) {
              tc_fence_before();
              __syncwarp();
              arrive_if(p0, rel_l + buf * S, p1, rel_r + buf * S);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                acc[j][32 * x + i] = fmaf(__uint_as_float(r[x][i]), sk[k], acc[j][32 * x + i]);
          }
          use ^= 1u << g;
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) fail_mm8(c, p.status);
        break;
      }
      // the tile's sums leave through the staging block, 16 rows of 128 bytes at a time, so that a
      // warp writes whole lines (rows past the unit's last are masked); 16-byte chunk k of row r lies
      // at chunk k ^ r % 8, without bank conflicts either way.  (dW of 16 experts, 2560 x 4096 in fp32
      // from 16384 tokens: 258 us, 279 with 32 rows of 64 bytes, 190 without stores.)
      constexpr int ES = OUT == SBP_BF16 ? 2 : 4, PASS = 128 / ES;   // columns a pass
      const int r0 = (int)rank * 128 + q * 32;            // this warp's first row of the unit
      const int rows = tile.z - r0 - lane / 8;            // how many there are from this lane's first on
      const int col0 = tile.w + h * (HALVES == 2 ? 128 : 64) + (lane % 8) * (16 / ES);
      uint8_t* out = static_cast<uint8_t*>(p.C) +
                     ((int64_t)tile.x * p.c_stride + (int64_t)(tile.y + r0 + lane / 8) * p.nb + col0) * ES;
      const int64_t down = (int64_t)4 * p.nb * ES;
#pragma unroll
      for (int gg = 0; gg < HALVES * 64 / PASS; ++gg) {
        const int cc = gg * PASS, j = cc / 64, g0 = cc % 64;
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          __syncwarp();
          if (lane / 16 == hr) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              uint32_t v[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (OUT == SBP_BF16) {
                  v[i] = pack_bf16(acc[j][g0 + 8 * k + 2 * i], acc[j][g0 + 8 * k + 2 * i + 1]);
                } else {
                  v[i] = __float_as_uint(acc[j][g0 + 4 * k + i]);
                }
              }
              sts128(stg + (lane & 15) * 128 + ((k ^ (lane & 7)) << 4), v[0], v[1], v[2], v[3]);
            }
          }
          __syncwarp();
          uint32_t v[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i * 4 + lane / 8;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[i][0]), "=r"(v[i][1]), "=r"(v[i][2]), "=r"(v[i][3])
                         : "r"(stg + r * 128 + (((lane % 8) ^ (r & 7)) << 4))
                         : "memory");
          }
          if (col0 + cc < p.nb) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (16 * hr + 4 * i >= rows) break;
              uint8_t* at = out + cc * ES + (4 * hr + i) * down;
              if (ACC) {
                const float4 old = *reinterpret_cast<const float4*>(at);
                *reinterpret_cast<float4*>(at) =
                    make_float4(old.x + __uint_as_float(v[i][0]), old.y + __uint_as_float(v[i][1]),
                                old.z + __uint_as_float(v[i][2]), old.w + __uint_as_float(v[i][3]));
              } else {
                *reinterpret_cast<uint4*>(at) = make_uint4(v[i][0], v[i][1], v[i][2], v[i][3]);
              }
            }
          }
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

// Units of 256 rows of A: the most there can be.
int64_t units_many(const P& p) {
  return p.columns ? (int64_t)p.E * ((p.na + 255) / 256) : max_units(p.T, p.E, 256);
}

template <int HALVES, int OUT, bool ACC>
cudaError_t launch_many(const P& p, cudaStream_t s) {
  using namespace tc;
  static int attr_state[64] = {};
  static std::mutex mu;
  const auto kern = k_mm8<HALVES, OUT, ACC>;
  if (!once_per_device(attr_state, mu, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_MM8) == cudaSuccess;
      }))
    return cudaErrorInvalidConfiguration;
  CUtensorMap mA, mB;
  if (!make_map_u8(&mA, p.A, (uint64_t)p.K, (uint64_t)(p.columns ? p.na : p.T), (uint64_t)p.lda, 128) ||
      !make_map_u8(&mB, p.B, (uint64_t)p.K, p.columns ? (uint64_t)p.nb : (uint64_t)p.E * p.nb, (uint64_t)p.ldb, 64))
    return cudaErrorInvalidValue;
  if (cudaMemsetAsync(p.status, 0, sizeof(int32_t), s) != cudaSuccess) return cudaErrorUnknown;
  P q = p;
  q.limit_ns = wait_limit_ns();
  q.stall = fault_stall_requested();
  const int64_t tiles = units_many(p) * ((p.nb + 128 * HALVES - 1) / (128 * HALVES));
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  const int pairs = (int)std::min<int64_t>(max_pairs((const void*)kern, SMEM_MM8, MM8_THREADS), tiles);
  kern<<<2 * pairs, MM8_THREADS, SMEM_MM8, s>>>(mA, mB, q);
  ran(HALVES == 2 ? SBP_PRODUCT_MANY_256 : SBP_PRODUCT_MANY_128);
  return cudaGetLastError();
}
template <int HALVES>
cudaError_t launch_many(const P& p, cudaStream_t s) {
  if (p.out == SBP_BF16) return launch_many<HALVES, SBP_BF16, false>(p, s);
  return p.accumulate ? launch_many<HALVES, SBP_FP32, true>(p, s) : launch_many<HALVES, SBP_FP32, false>(p, s);
}

// Tiles of 256 columns take 496 ns a block on all pairs at once, tiles of 128 columns 281 (16384 x
// 24576 x 4096, the same inputs throughout: 1285 and 1453 us), where all eight epilogue warps take every
// accumulator; the narrow ones leave fewer pairs idle (501 x 4096 x 12288: 53 and 33 us).  The shorter of
// the two sums of rounds is taken.
int64_t rounds_ns(const P& p, int halves) {
  const int64_t bn = 128 * halves, pairs = num_sms() / 2;
  return (about_units(p, 256) * ((p.nb + bn - 1) / bn) + pairs - 1) / pairs * about_blocks(p) * (halves == 2 ? 496 : 281);
}
int64_t many_ns(const P& p) { return 8000 + std::min(rounds_ns(p, 1), rounds_ns(p, 2)); }

cudaError_t many(const P& p, cudaStream_t s) {
  return rounds_ns(p, 2) <= rounds_ns(p, 1) ? launch_many<2>(p, s) : launch_many<1>(p, s);
}

}  // namespace mm8
}  // namespace sbp
