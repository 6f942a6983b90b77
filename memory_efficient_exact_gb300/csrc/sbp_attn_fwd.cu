// Forward of the attention over packed documents (bf16 operands, fp32 softmax, sm_103a).
//
// k_attn_o  unit = (query head, 256 queries), 128 queries in each CTA of an SM pair, the
// longest units first.  O stays in tensor memory while the unit walks its blocks of 128 keys:
//   S = Q K^T            (tensor memory, two buffers)
//   P = 2^(x - m)        (softmax warps; bf16, two buffers in tensor memory)
//   O += P V             (tensor memory; P is the A operand from tensor memory)
// so nothing of size (queries x keys) leaves the SM.  With two S buffers the next block's S
// is ready before the softmax warps have finished a block, and O += P V of the block before
// runs behind it, so that the softmax warps never wait for the tensor pipe.
// The running maximum m is only raised when a block exceeds it by more than 2^8 (P and its
// sum stay far from overflow below that), and O is rescaled in tensor memory only then.  The
// sum l adds the fp32 probabilities; P is rounded to bf16 for the product, the operand type
// of the tensor pipe at full rate: at most 2^-9 of each probability.
//
// Pair protocol and bounded waits as in the backward kernels (sbp_attn_fused.cuh).
#include <algorithm>

#include "sbp_attn_fused.cuh"
#include "sbp_attn_packed.cuh"

namespace sbp {
namespace tc {
namespace fo {

using fa::dplus;
using fa::mma2_bf16_ts;
using fa::tmem_st_wait;

// Warps: 0 TMA producers, 1 MMA issuer, 2-9 softmax (lane quadrant warp % 4, 64 of the 128
// columns each), 10 forwarder (turns the CTA's local arrivals into one arrival at the
// leader), 11 idle: 12 warps, so 168 registers a thread.
constexpr int EPI = 8;
constexpr int FWD_WARP = 2 + EPI;
constexpr int THREADS = 384;

// Shared memory, bytes from the 1024-aligned base; tiles are 128-byte swizzled
// [64-element block][rows][128 B].
constexpr int KV_STAGES = 4;
constexpr uint32_t O_Q = 0;                              // 2 units: this CTA's 128 queries
constexpr uint32_t O_K = 65536;                          // this CTA's 64 keys of the block
constexpr uint32_t O_V = O_K + KV_STAGES * 16384;        // 128 keys x this CTA's 64 of hd
constexpr uint32_t O_MX = O_V + KV_STAGES * 16384;       // [2][2 halves][128 rows] fp32
constexpr uint32_t O_CTRL = O_MX + 2048;
// Tensor memory: S buffers at 0 and 128, O at T_O, P buffers of 64 columns at T_P.
constexpr uint32_t T_O = 256, T_P = 384;
constexpr uint32_t IDESC_KK = idesc_bf16(256, 128, false, false);  // A, B K-major
constexpr uint32_t IDESC_KM = idesc_bf16(256, 128, false, true);   // A K-major, B MN-major

struct Ctrl {
  uint64_t kfull[KV_STAGES], kempty[KV_STAGES], vfull[KV_STAGES], vempty[KV_STAGES];
  uint64_t qfull[2], qempty[2];
  uint64_t sfull[2];             // S buffer is ready (both CTAs)
  uint64_t sempty[2];            // leader: both CTAs have read the S buffer
  uint64_t pready[2];            // leader: both CTAs' P buffer is written
  uint64_t pfree[2];             // O += P V of the P buffer is done (both CTAs)
  uint64_t sempty_l[2], pready_l[2];   // the CTA's softmax warps, forwarded
  uint64_t accempty;             // leader: the unit's O has been read out
  uint64_t mx[4];                // per lane quadrant: its two warps have left their row values
  uint64_t mdone;
  uint32_t tmem_base;
  int abort;
};
constexpr size_t SMEM = O_CTRL + sizeof(Ctrl) + 1024;
static_assert(SMEM <= 232448, "shared memory of the attention forward");

struct Params {
  int H, T, hd, group, n_units;
  pk::Scale sc;
  const float* slopes;
  const PackedQUnit* units;
  const int32_t *lo, *hi, *tail;
  __nv_bfloat16* O;
  float* lse;
  int32_t* status;
  uint64_t limit_ns;
};

// Unit u: head z, queries [256 qp, +256), key blocks [j0, j0 + nj).
__device__ __forceinline__ void unit_of(const Params& p, int u, int& z, int& qp, int& j0, int& nj) {
  const int i = u / p.H;
  z = u - i * p.H;
  const int4* s = reinterpret_cast<const int4*>(p.units + i);
  const int4 a = s[0];
  qp = a.x;
  j0 = a.y;
  nj = max(a.z, s[1].x) - a.y;
}

__device__ __forceinline__ void fail_o(Ctrl* c, int32_t* status) {
  *(volatile int*)&c->abort = 1;
  if (status) atomicCAS(status, 0, SBP_ERR_TIMEOUT);
}
__device__ __forceinline__ bool wait1(uint64_t* b, uint32_t parity, Ctrl* c, uint64_t limit) {
  return wait_inl<true>(b, parity & 1u, &c->abort, limit);
}
__device__ __forceinline__ bool warp_wait(uint64_t* b, uint32_t parity, Ctrl* c, uint64_t limit) {
  return __all_sync(0xffffffffu, wait_inl<true>(b, parity & 1u, &c->abort, limit));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// tmVt: the last block's V with zeroed padding (PackedWork::tail)
template <bool CAP, bool BIAS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    k_attn_o(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
             const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmVt, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctrl* c = reinterpret_cast<Ctrl*>(base + O_CTRL);
  const uint32_t sb = saddr(base);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = ctarank();
  if (threadIdx.x == 0) {
    for (int i = 0; i < KV_STAGES; ++i) {
      mbar_init(&c->kfull[i], 1);
      mbar_init(&c->kempty[i], 1);
      mbar_init(&c->vfull[i], 1);
      mbar_init(&c->vempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c->qfull[i], 1);
      mbar_init(&c->qempty[i], 1);
      mbar_init(&c->sfull[i], 1);
      mbar_init(&c->sempty[i], 2);
      mbar_init(&c->pready[i], 2);
      mbar_init(&c->pfree[i], 1);
      mbar_init(&c->sempty_l[i], EPI);
      mbar_init(&c->pready_l[i], EPI);
    }
    mbar_init(&c->accempty, 2 * EPI);
    for (int i = 0; i < 4; ++i) mbar_init(&c->mx[i], 2);
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
  const int pid = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (warp == 0) {
    if (lane == 0) {
      // Q of the unit (this CTA's 128 queries), then K of each block (this CTA's 64 keys)
      prefetch_map(&tmQ);
      prefetch_map(&tmK);
      uint32_t g = 0, lu = 0;   // blocks and units so far
      bool ok = true;
      for (int u = pid; u < p.n_units && ok; u += npairs) {
        int z, qp, j0, nj;
        unit_of(p, u, z, qp, j0, nj);
        if (nj <= 0) continue;
        const uint32_t qs = lu & 1u;
        if (!wait1(&c->qempty[qs], (lu >> 1) ^ 1u, c, p.limit_ns)) { ok = false; break; }
        const uint32_t fq = mapa(saddr(&c->qfull[qs]), 0);
        if (rank == 0) mbar_expect_tx(&c->qfull[qs], 2u * 32768u);
        const int qrow = 256 * qp + 128 * (int)rank;
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
          tma_load_3d_pair(sb + O_Q + qs * 32768u + hb * 16384, &tmQ, fq, 64 * hb, qrow, z);
        ++lu;
        for (int j = 0; j < nj; ++j) {
          const uint32_t s = g % KV_STAGES;
          if (!wait1(&c->kempty[s], (g / KV_STAGES) ^ 1u, c, p.limit_ns)) { ok = false; break; }
          const uint32_t fk = mapa(saddr(&c->kfull[s]), 0);
          if (rank == 0) mbar_expect_tx(&c->kfull[s], 2u * 16384u);
          const int krow = 128 * (j0 + j) + 64 * (int)rank;
#pragma unroll
          for (int hb = 0; hb < 2; ++hb)
            tma_load_3d_pair(sb + O_K + s * 16384u + hb * 8192, &tmK, fk, 64 * hb, krow, z / p.group);
          ++g;
        }
      }
      if (!ok) {   // wait for the copies in flight
        fail_o(c, p.status);
        if (rank == 0) {
          for (uint32_t i = lu > 2 ? lu - 2 : 0; i < lu; ++i)
            wait_inl<false>(&c->qfull[i & 1u], (i >> 1) & 1u, nullptr, 200000000ull);
          for (uint32_t i = g > KV_STAGES ? g - KV_STAGES : 0; i < g; ++i)
            wait_inl<false>(&c->kfull[i % KV_STAGES], (i / KV_STAGES) & 1u, nullptr, 200000000ull);
        }
      }
    } else if (lane == 16) {
      // V of each block, 128 keys x this CTA's half of hd (B of O += P V)
      prefetch_map(&tmV);
      const int tail = *p.tail;
      uint32_t g = 0;
      bool ok = true;
      for (int u = pid; u < p.n_units && ok; u += npairs) {
        int z, qp, j0, nj;
        unit_of(p, u, z, qp, j0, nj);
        for (int j = 0; j < nj; ++j) {
          const uint32_t s = g % KV_STAGES;
          if (!wait1(&c->vempty[s], (g / KV_STAGES) ^ 1u, c, p.limit_ns)) { ok = false; break; }
          const uint32_t fv = mapa(saddr(&c->vfull[s]), 0);
          if (rank == 0) mbar_expect_tx(&c->vfull[s], 2u * 16384u);
          if (j0 + j == tail)
            tma_load_3d_pair(sb + O_V + s * 16384u, &tmVt, fv, 64 * (int)rank, 0, z / p.group);
          else
            tma_load_3d_pair(sb + O_V + s * 16384u, &tmV, fv, 64 * (int)rank, 128 * (j0 + j), z / p.group);
          ++g;
        }
      }
      if (!ok) {
        fail_o(c, p.status);
        if (rank == 0)
          for (uint32_t i = g > KV_STAGES ? g - KV_STAGES : 0; i < g; ++i)
            wait_inl<false>(&c->vfull[i % KV_STAGES], (i / KV_STAGES) & 1u, nullptr, 200000000ull);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint64_t dQ = sw128_desc(sb + O_Q, 16, 1024), dK = sw128_desc(sb + O_K, 16, 1024),
                     dV = sw128_desc(sb + O_V, 16384, 1024);
      uint32_t g = 0, lu = 0;
      bool ok = true;
      // O += P V of block gg (the first of its unit overwrites)
      auto accumulate = [&](uint32_t gg, bool first) -> bool {
        const uint32_t s = gg % KV_STAGES, b = gg & 1u;
        if (!wait1(&c->pready[b], gg >> 1, c, p.limit_ns)) return false;
        if (!wait1(&c->vfull[s], gg / KV_STAGES, c, p.limit_ns)) return false;
        if (first && !wait1(&c->accempty, lu ^ 1u, c, p.limit_ns)) return false;
        tc_fence_after();
        const uint64_t v0 = dplus(dV, s * 16384u);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma2_bf16_ts(tmem + T_O, tmem + T_P + 64 * b + 8 * k, dplus(v0, k * 2048), IDESC_KM,
                       (!first || k) ? 1u : 0u);
        commit2_mc(&c->vempty[s], 3);
        commit2_mc(&c->pfree[b], 3);
        return true;
      };
      for (int u = pid; u < p.n_units && ok; u += npairs) {
        int z, qp, j0, nj;
        unit_of(p, u, z, qp, j0, nj);
        if (nj <= 0) continue;
        const uint32_t qs = lu & 1u;
        if (!wait1(&c->qfull[qs], lu >> 1, c, p.limit_ns)) { ok = false; break; }
        for (int n = 0; n < nj; ++n, ++g) {
          const uint32_t s = g % KV_STAGES, b = g & 1u;
          if (!wait1(&c->sempty[b], (g >> 1) ^ 1u, c, p.limit_ns)) { ok = false; break; }
          if (!wait1(&c->kfull[s], g / KV_STAGES, c, p.limit_ns)) { ok = false; break; }
          tc_fence_after();
          const uint64_t q0 = dplus(dQ, qs * 32768u), k0 = dplus(dK, s * 16384u);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma2_bf16(tmem + 128 * b, dplus(q0, k * 32), dplus(k0, k * 32), IDESC_KK, k ? 1u : 0u);
          if (p.hd > 64) {   // the second 64 columns of a row (zero past hd)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma2_bf16(tmem + 128 * b, dplus(q0, 16384 + k * 32), dplus(k0, 8192 + k * 32), IDESC_KK, 1u);
          }
          commit2_mc(&c->kempty[s], 3);
          commit2_mc(&c->sfull[b], 3);
          if (n == nj - 1) commit2_mc(&c->qempty[qs], 3);
          if (n >= 1 && !accumulate(g - 1, n == 1)) { ok = false; break; }
        }
        if (!ok) break;
        if (!accumulate(g - 1, nj == 1)) { ok = false; break; }
        ++lu;
      }
      if (!ok) fail_o(c, p.status);
      commit2_mc(&c->mdone, 1);
      wait_inl<false>(&c->mdone, 0, nullptr, 200000000ull);
    }
    __syncwarp();
  } else if (warp == FWD_WARP) {
    if (lane == 0) {
      uint32_t g = 0;
      bool ok = true;
      for (int u = pid; u < p.n_units && ok; u += npairs) {
        int z, qp, j0, nj;
        unit_of(p, u, z, qp, j0, nj);
        for (int j = 0; j < nj; ++j, ++g) {
          const uint32_t b = g & 1u;
          if (!wait1(&c->sempty_l[b], g >> 1, c, p.limit_ns)) { ok = false; break; }
          arrive_remote(mapa(saddr(&c->sempty[b]), 0));
          if (!wait1(&c->pready_l[b], g >> 1, c, p.limit_ns)) { ok = false; break; }
          arrive_remote(mapa(saddr(&c->pready[b]), 0));
        }
      }
      if (!ok) fail_o(c, p.status);
    }
    __syncwarp();
  } else if (warp < FWD_WARP) {
    const int q = warp & 3, ch = (warp - 2) >> 2;   // lane quadrant; 64-column half
    const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16);
    float* mxp = reinterpret_cast<float*>(base + O_MX);
    const int lrow = 32 * q + lane;
    // scores stay raw when they only need the scale, which the exponent's FMA applies
    constexpr bool RAW = !CAP && !BIAS;
    const float mul = RAW ? p.sc.sl2 : 1.f;
    uint32_t g = 0, e = 0;   // blocks and row-value exchanges so far
    bool ok = true;
    // v of this row from the warp that has the other 64 columns
    auto other = [&](float v, float& o) -> bool {
      float* slot = mxp + (e & 1u) * 256;
      slot[ch * 128 + lrow] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->mx[q]);
      if (!warp_wait(&c->mx[q], e, c, p.limit_ns)) return false;
      o = slot[(ch ^ 1) * 128 + lrow];
      ++e;
      return true;
    };
    for (int u = pid; u < p.n_units && ok; u += npairs) {
      int z, qp, j0, nj;
      unit_of(p, u, z, qp, j0, nj);
      const int row = 256 * qp + 128 * (int)rank + lrow;
      const bool vrow = row < p.T;
      const int64_t ro = (int64_t)z * p.T + row;
      const int lo = vrow ? p.lo[row] : p.T, hi = vrow ? p.hi[row] : p.T;
      const int lo0 = __shfl_sync(0xffffffffu, lo, 0), lo1 = __shfl_sync(0xffffffffu, lo, 31);
      const int hi0 = __shfl_sync(0xffffffffu, hi, 0), hi1 = __shfl_sync(0xffffffffu, hi, 31);
      const pk::ScaleZ sc{p.sc.sl2, p.sc.c2, p.sc.k, BIAS ? p.slopes[z] * L2E : 0.f};
      float m = -INFINITY, l = 0.f;
      for (int n = 0; n < nj; ++n, ++g) {
        const uint32_t b = g & 1u;
        if (!warp_wait(&c->sfull[b], g >> 1, c, p.limit_ns)) { ok = false; break; }
        tc_fence_after();
        uint32_t r[2][32];
        tmem_ld32(trow + 128 * b + 64 * ch, r[0]);
        tmem_ld32(trow + 128 * b + 64 * ch + 32, r[1]);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->sempty_l[b]);   // S is in registers: its buffer may be refilled
        const int k0 = 128 * (j0 + n) + 64 * ch;       // this thread's first key
        if (!RAW) {
          const float fd = (float)(row - k0);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float dc;
              float x = pk::capped<CAP>(sc, __uint_as_float(r[h][i]), dc);
              if (BIAS) x = fmaf(-sc.slope2, fabsf(fd - (float)(32 * h + i)), x);
              r[h][i] = __float_as_uint(x);
            }
        }
        if (k0 < lo1 || k0 + 63 >= hi0) {   // some row of the warp does not see all 64 keys
          const int a = lo - k0, t = hi - k0;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * h + i < a || 32 * h + i >= t) r[h][i] = 0xff800000u;   // -inf
        }
        float mx[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          mx[h] = __uint_as_float(r[h >> 1][16 * (h & 1)]);
#pragma unroll
          for (int i = 1; i < 16; ++i) mx[h] = fmaxf(mx[h], __uint_as_float(r[h >> 1][16 * (h & 1) + i]));
        }
        float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), mo;
        if (!other(mb, mo)) { ok = false; break; }
        mb = fmaxf(mb, mo);
        float f = 1.f;
        if (mb > m && (m == -INFINITY || (mb - m) * mul > 8.f)) {
          f = ex2((m - mb) * mul);   // 0 from m = -inf
          m = mb;
        }
        // both warps of the row take the same decision; each rescales its 64 columns of O
        if (n > 0 && __any_sync(0xffffffffu, f != 1.f)) {
          if (!warp_wait(&c->pfree[b ^ 1u], (g - 1) >> 1, c, p.limit_ns)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int h = 0; h < 64; h += 32) {
            uint32_t o[32];
            tmem_ld32(trow + T_O + 64 * ch + h, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st32(trow + T_O + 64 * ch + h, o);
          }
        }
        l *= f;
        const float nm = m == -INFINITY ? 0.f : -m * mul;
        float ls[2] = {0.f, 0.f};
        uint32_t pw[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float e0 = ex2(fmaf(__uint_as_float(r[i >> 4][2 * i & 31]), mul, nm));
          const float e1 = ex2(fmaf(__uint_as_float(r[i >> 4][(2 * i & 31) + 1]), mul, nm));
          ls[0] += e0;
          ls[1] += e1;
          pw[i] = pack_bf16(e0, e1);
        }
        l += ls[0] + ls[1];
        // P into its buffer once the product of two blocks before has read it
        if (!warp_wait(&c->pfree[b], (g >> 1) ^ 1u, c, p.limit_ns)) { ok = false; break; }
        tmem_st32(trow + T_P + 64 * b + 32 * ch, pw);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->pready_l[b]);
      }
      if (!ok) break;
      if (nj > 0) {
        float lx;
        if (!other(l, lx)) { ok = false; break; }
        l = ch ? lx + l : l + lx;   // the same order in both warps
        // the last product covers all earlier ones
        if (!warp_wait(&c->pfree[(g - 1) & 1u], (g - 1) >> 1, c, p.limit_ns)) { ok = false; break; }
        tc_fence_after();
      }
      uint32_t o[2][32];
      __syncwarp();
      if (nj > 0) {
        tmem_ld32(trow + T_O + 64 * ch, o[0]);
        tmem_ld32(trow + T_O + 64 * ch + 32, o[1]);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_remote(mapa(saddr(&c->accempty), 0));
      }
      if (vrow) {
        // a row that sees nothing (padding): 0 and -inf
        const bool none = l == 0.f;
        const float inv = none ? 0.f : 1.f / l;
        if (ch == 0) p.lse[ro] = none ? -INFINITY : (m * mul + log2f(l)) * 0.6931471805599453f;
        uint4* dst = reinterpret_cast<uint4*>(p.O + ro * p.hd + 64 * ch);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = none ? 0u
                        : pack_bf16(__uint_as_float(o[k >> 2][8 * (k & 3) + 2 * i]) * inv,
                                    __uint_as_float(o[k >> 2][8 * (k & 3) + 2 * i + 1]) * inv);
          if (64 * ch + 8 * k < p.hd) dst[k] = make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
      __syncwarp();
    }
    if (!ok) fail_o(c, p.status);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
  }
}

}  // namespace fo
}  // namespace tc

namespace {

template <bool CAP, bool BIAS>
cudaError_t launch_o(const PackedArgs& a, const PackedWork& w, void* O, float* lse, cudaStream_t s) {
  using namespace tc::fo;
  static int attr_state[64] = {};
  static std::mutex mu;
  if (!tc::once_per_device(attr_state, mu, [] {
        return cudaFuncSetAttribute(k_attn_o<CAP, BIAS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM) ==
               cudaSuccess;
      }))
    return cudaErrorInvalidConfiguration;
  Params p;
  p.H = (int)a.H; p.T = (int)a.T; p.hd = (int)a.hd; p.group = (int)(a.H / a.Hkv);
  p.n_units = (int)((a.T + 255) / 256 * a.H);
  p.sc = tc::pk::make_scale(a.scale, a.softcap);
  p.slopes = a.slopes; p.units = w.qunits; p.lo = w.lo; p.hi = w.hi; p.tail = w.tail;
  p.O = static_cast<__nv_bfloat16*>(O); p.lse = lse; p.status = a.status; p.limit_ns = tc::wait_limit_ns();
  CUtensorMap mQ, mK, mV, mVt;
  if (!tc::make_map_heads(&mQ, a.Q, a.T, a.H, a.hd, 128) || !tc::make_map_heads(&mK, a.K, a.T, a.Hkv, a.hd, 64) ||
      !tc::make_map_heads(&mV, a.V, a.T, a.Hkv, a.hd, 128) ||
      !tc::make_map_heads(&mVt, w.tail_kv, 128, a.Hkv, a.hd, 128))
    return cudaErrorInvalidValue;
  const int pairs = std::min(tc::max_pairs((const void*)k_attn_o<CAP, BIAS>, SMEM, THREADS), p.n_units);
  k_attn_o<CAP, BIAS><<<2 * pairs, THREADS, SMEM, s>>>(mQ, mK, mV, mVt, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t packed_forward(const PackedArgs& a, const PackedWork& w, void* O, float* lse, cudaStream_t s) {
  if (a.softcap > 0.f)
    return a.slopes ? launch_o<true, true>(a, w, O, lse, s) : launch_o<true, false>(a, w, O, lse, s);
  return a.slopes ? launch_o<false, true>(a, w, O, lse, s) : launch_o<false, false>(a, w, O, lse, s);
}

}  // namespace sbp
