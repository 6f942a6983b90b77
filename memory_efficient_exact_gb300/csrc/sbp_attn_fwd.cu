// Forward of the attention over packed documents (bf16 operands, fp32 softmax, sm_103a).
//
// k_attn_o  unit = (query head, 256 queries), 128 queries in each CTA of an SM pair, the
// longest units first.  The unit walks its blocks of 128 keys; two groups of four softmax
// warps take the blocks in turn, each with its own S buffer, running maximum, sum and O
// accumulator in tensor memory, so that they exchange nothing until the unit's end (buffers and
// accumulator are shared where the maximum is known, see Tmem):
//   S = Q K^T            (tensor memory)
//   P = 2^(x - m)        (one query row a thread; bf16, written over S)
//   O += P V             (tensor memory; P is the A operand from tensor memory)
// While one group works on a block, the tensor pipe runs the other group's O += P V and its
// next S.  At the end the two accumulators are joined, O = (O0 2^(m0-m) + O1 2^(m1-m)) / l.
// Nothing of size (queries x keys) leaves the SM.
// The exponentials are taken from the maximum of earlier blocks, while the block's own is found
// beside them: any reference serves the quotient as long as neither overflows.  Only a block
// that exceeds it by 2^kLag or holds a row's first keys is read once more beforehand, to raise
// the maximum and rescale O and l.
// Scores capped at up to kStaticCap need no maximum (0, or the row's largest bias): 2^x neither
// overflows nor, for at least one key, underflows.  The sum l adds the fp32 probabilities; P is
// rounded to bf16 for the product, the operand type of the tensor pipe at full rate: at most
// 2^-8 of each probability.
// The end of a unit, the wait for its last products and the join, comes behind the next unit's
// first block.
// What bounds it: 32 / 8 heads of 128, 16384 tokens, take 1.49 ms (1475 TFLOP/s over the visible
// pairs); the tensor pipe is busy 1034 of about 1550 cycles a block, the rest is the handoff from
// P to O += P V to the group's next S, which the other group hides in part.  (l over the rounded
// probabilities would take their rounding out of rows that one key holds, 0.19% for 0.23% in norm
// with a cap of 50; two more operations a score, 1.68 ms for 1.49 and 241 us for 222.)  Documents of 1000 to
// 2500 tokens: 156 us (812 TFLOP/s; a quarter of the products lie outside the documents or
// behind the diagonal).  Capped at 50: 219 us; the special-function unit is the busiest, 55% of the
// cycles, the tensor pipe 35%, and 41% of the issue slots are taken: the softmax warps' waits for
// their scores and for each other's products are the rest, not any one unit.
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

// Warps: 0 TMA producers, 1 MMA issuer (leader), 2 and 3 idle, 4-7
// and 8-11 the softmax groups (lane quadrant warp % 4).
constexpr int SOFT_WARP = 4;
constexpr int THREADS = 384;
// The running maximum may lag behind the scores by this many powers of two.
constexpr float kLag = 16.f;

// Shared memory, bytes from the 1024-aligned base; tiles are 128-byte swizzled
// [64-element block][rows][128 B].
constexpr int KV_STAGES = 4;
constexpr uint32_t O_Q = 0;                              // 2 units: this CTA's 128 queries
constexpr uint32_t O_K = 65536;                          // this CTA's 64 keys of the block
constexpr uint32_t O_V = O_K + KV_STAGES * 16384;        // 128 keys x this CTA's 64 of hd
constexpr uint32_t O_ML = O_V + KV_STAGES * 16384;       // m, l: [2 units][2 groups][128 rows] float2
constexpr uint32_t O_CTRL = O_ML + 4096;
// Tensor memory: NB buffers of S (and P over it), block g's at 128 (g % NB), then O.  Two buffers,
// one a group, and an O each; or, where the maximum is known beforehand and both groups' P
// have the same reference, three and one O for both: a group's next S is then formed before its
// P is multiplied (cap 50, 8192 tokens: 222 us, 248 with two).
template <bool FIXED>
struct Tmem {
  static constexpr uint32_t NB = FIXED ? 3 : 2;
  static constexpr uint32_t O = 128 * NB;
};
constexpr uint32_t IDESC_KK = idesc_bf16(256, 128, false, false);  // A, B K-major
constexpr uint32_t IDESC_KM = idesc_bf16(256, 128, false, true);   // A K-major, B MN-major

struct Ctrl {
  uint64_t kfull[KV_STAGES], kempty[KV_STAGES], vfull[KV_STAGES], vempty[KV_STAGES];
  uint64_t qfull[2], qempty[2];   // Q of the unit; free: its products are done, and O has left
  uint64_t sfull[3];      // S of the buffer is ready, and the products before it are done
  uint64_t pready_l[3];   // P is written over it: the leader's four warps of the block's group
  uint64_t pready_r[3];   // the same of the other CTA (leader)
  uint64_t ofull;         // the unit's products are done (both CTAs)
  uint64_t accempty;      // leader: the unit's O has been read out
  uint64_t mlx;           // the CTA's eight softmax warps have left m and l
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

// Block n of a unit: behind to front with a distance bias, so that the maximum is found early (its
// slopes are positive as a rule).
template <bool BIAS>
__device__ __forceinline__ int block_at(int j0, int nj, int n) { return BIAS ? j0 + nj - 1 - n : j0 + n; }

// Unit u: head z, queries [256 qp, +256), key blocks [j0, j0 + nj); none past the last.
struct Unit { int z, qp, j0, nj; };
__device__ __forceinline__ Unit unit_of(const Params& p, int u) {
  if (u >= p.n_units) return Unit{0, 0, 0, 0};
  const int i = u / p.H;
  const int4* s = reinterpret_cast<const int4*>(p.units + i);
  const int4 a = s[0];
  return Unit{u - i * p.H, a.x, a.y, max(a.z, s[1].x) - a.y};
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

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A row's view of a block's keys k0 .., and what its warp's rows have in common.
struct Row {
  int a, b;           // the row sees the keys k0 + [a, b)
  int all_a, all_b;   // every row of the warp sees k0 + [all_a, all_b)
  int first;          // the warp's first query - k0
  float fd;           // the query - k0
  float top;          // the cap, less a fixed maximum
  __device__ __forceinline__ bool masked(int c, int n) const { return c < all_a || c + n > all_b; }   // keys c .. c + n - 1
  // some row does not see all 128 keys, or (BIAS) they lie on both sides of the warp's queries
  template <bool BIAS>
  __device__ __forceinline__ bool edge() const { return masked(0, 128) || (BIAS && first < 127 && first + 31 > 0); }
};
// The lowest n bits, n from 0 to 32 after clamping.
__device__ __forceinline__ uint32_t low_bits(int n) { return (uint32_t)((1ull << min(max(n, 0), 32)) - 1); }

// 32 scores (keys k0 + c ..) as they enter the exponential (left unscaled without cap and bias).
// EDGE: -inf where the row does not see the key, and the bias by each key's distance; else its
// products with the distance are linear in the key.
template <bool CAP, bool BIAS, bool EDGE>
__device__ __forceinline__ void scores32(uint32_t (&r)[32], int c, const Row& w, const pk::ScaleZ& sc) {
  auto f2 = [&](int i) { return make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])); };
  const float m = CAP ? -2.f * sc.c2 : sc.sl2, top = CAP ? w.top : 0.f;
  float fd = w.fd - (float)c;
  if (BIAS) asm volatile("" : "+f"(fd));   // 128 distances are not worth keeping for a second pass
  const float step = w.first > 0 ? sc.slope2 : -sc.slope2, at0 = fmaf(-step, fd, top);
  auto add = [&](int i) {   // the bias of key i
    if (!BIAS) return top;
    return EDGE ? fmaf(-sc.slope2, fabsf(fd - (float)i), top) : fmaf(step, (float)i, at0);
  };
  if (CAP || BIAS) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 v = fma2(CAP ? pk::cap_parts<EDGE>(sc, f2(i)) : f2(i), make_float2(m, m),
                            make_float2(add(2 * i), add(2 * i + 1)));
      r[2 * i] = __float_as_uint(v.x);
      r[2 * i + 1] = __float_as_uint(v.y);
    }
  }
  if (EDGE && w.masked(c, 32)) {
    const uint32_t see = low_bits(w.b - c) & ~low_bits(w.a - c);
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (!(see & (1u << i))) r[i] = 0xff800000u;
  }
}
__device__ __forceinline__ float max32(const uint32_t (&r)[32], float m0) {
  float m[4] = {m0, __uint_as_float(r[0]), __uint_as_float(r[1]), __uint_as_float(r[2])};
#pragma unroll
  for (int i = 3; i + 1 < 32; i += 2)
    m[(i >> 1) & 3] = max3(m[(i >> 1) & 3], __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
  return max3(fmaxf(m[0], m[1]), m[2], fmaxf(m[3], __uint_as_float(r[31])));
}
// 32 probabilities 2^(mul x + nm) (PLAIN: 2^x): packed to bf16, their sum added to l.
// (Keeping some of them off the special-function unit, by a polynomial, took longer at every
// share: a quarter 2.08 ms against 1.67 at 32 heads, 16384 tokens.)
template <bool PLAIN>
__device__ __forceinline__ void probs32(const uint32_t (&r)[32], float mul, float nm, uint32_t* pw, float2& l) {
  const float2 m2 = make_float2(mul, mul), nm2 = make_float2(nm, nm);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float2 x = make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
    if (!PLAIN) x = fma2(x, m2, nm2);
    const float2 e = make_float2(ex2(x.x), ex2(x.y));
    l = add2(l, e);
    pw[i] = pack_bf16(e.x, e.y);
  }
}

// A block of 128 scores of a row (tensor memory tS) into its probabilities there; m and l are the
// row's running maximum and sum, tO the group's accumulator, `fresh` while that holds nothing.
// `raise`: the maximum has to be found before the exponentials.
template <bool CAP, bool BIAS, bool FIXED, bool EDGE>
__device__ __forceinline__ void soft_block(uint32_t tS, uint32_t tO, bool fresh, bool raise, const Row& w,
                                           const pk::ScaleZ& sc, float mul, float& m, float2& l) {
  uint32_t ra[32], rb[32], pw[64];
  float2 lb;   // the block's sums
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    if (raise) {
      float mb = m;
#pragma unroll 1
      for (int h = 0; h < 128; h += 32) {
        __syncwarp();
        tmem_ld32(tS + h, ra);
        tmem_ld_wait();
        scores32<CAP, BIAS, true>(ra, h, w, sc);
        mb = max32(ra, mb);
      }
      const float f = mb > m ? ex2((m - mb) * mul) : 1.f;   // 0 from m = -inf
      if (mb > m) m = mb;
      l.x *= f;
      l.y *= f;
      if (!fresh && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
        for (int h = 0; h < 128; h += 16) {
          uint32_t o[16];
          fa::tmem_ld16(tO + h, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          fa::tmem_st16(tO + h, o);
        }
      }
    }
    const float nm = m == -INFINITY ? 0.f : -m * mul;
    float mb = -INFINITY;
    lb = make_float2(0.f, 0.f);
    auto part = [&](uint32_t (&r)[32], int c, uint32_t* out) {
      scores32<CAP, BIAS, EDGE>(r, c, w, sc);
      if (!FIXED) mb = max32(r, mb);
      probs32<FIXED>(r, mul, nm, out, lb);
    };
    __syncwarp();
    tmem_ld32(tS, ra);
    tmem_ld32(tS + 32, rb);
    tmem_ld_wait();
    part(ra, 0, pw);
    __syncwarp();
    tmem_ld32(tS + 64, ra);
    part(rb, 32, pw + 16);
    __syncwarp();
    tmem_ld32(tS + 96, rb);
    if (FIXED) tmem_st32(tS, pw);   // over scores that are in registers
    tmem_ld_wait();
    part(ra, 64, pw + 32);
    part(rb, 96, pw + 48);
    raise = !FIXED && __any_sync(0xffffffffu, (mb - m) * mul > kLag);
    if (!raise) break;   // always so after a pass that found the maximum
  }
  l = add2(l, lb);
  __syncwarp();
  if (!FIXED) tmem_st32(tS, pw);    // all the scores have been read
  tmem_st32(tS + 32, pw + 32);
  tmem_st_wait();
}

// tmVt: the last block's V with zeroed padding (PackedWork::tail)
// FIXED: scores capped low enough for a maximum that is known beforehand.
template <bool CAP, bool BIAS, bool FIXED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    k_attn_o(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
             const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmVt,
             const __grid_constant__ CUtensorMap tmO, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctrl* c = reinterpret_cast<Ctrl*>(base + O_CTRL);
  const uint32_t sb = saddr(base);
  const int warp = uniform_warp(), lane = threadIdx.x % 32;
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
      mbar_init(&c->qempty[i], 1 + 8);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&c->sfull[i], 1);
      mbar_init(&c->pready_r[i], 4);
      mbar_init(&c->pready_l[i], 4);
    }
    mbar_init(&c->ofull, 1);
    mbar_init(&c->accempty, 2 * 8);
    mbar_init(&c->mlx, 8);
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
  wait_for_primary();   // the preparing kernel
  const uint32_t tmem = c->tmem_base;
  const int pid = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (warp == 0) {
    if (lane == 0) {
      // Q of the unit (this CTA's 128 queries), then K of each block (this CTA's 64 keys)
      prefetch_map(&tmQ);
      prefetch_map(&tmK);
      uint32_t g = 0, lu = 0;   // blocks and units so far
      bool ok = true;
      Unit next = unit_of(p, pid);   // loaded a unit ahead
      for (int rnd = 0, u = pid; u < p.n_units && ok; u = pk::next_unit(++rnd, pid, npairs)) {
        const auto [z, qp, j0, nj] = next;
        next = unit_of(p, pk::next_unit(rnd + 1, pid, npairs));
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
          const int krow = 128 * block_at<BIAS>(j0, nj, j) + 64 * (int)rank;
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
      Unit next = unit_of(p, pid);   // loaded a unit ahead
      for (int rnd = 0, u = pid; u < p.n_units && ok; u = pk::next_unit(++rnd, pid, npairs)) {
        const auto [z, qp, j0, nj] = next;
        next = unit_of(p, pk::next_unit(rnd + 1, pid, npairs));
        for (int j = 0; j < nj; ++j) {
          const uint32_t s = g % KV_STAGES;
          if (!wait1(&c->vempty[s], (g / KV_STAGES) ^ 1u, c, p.limit_ns)) { ok = false; break; }
          const uint32_t fv = mapa(saddr(&c->vfull[s]), 0);
          if (rank == 0) mbar_expect_tx(&c->vfull[s], 2u * 16384u);
          const int blk = block_at<BIAS>(j0, nj, j);
          if (blk == tail)
            tma_load_3d_pair(sb + O_V + s * 16384u, &tmVt, fv, 64 * (int)rank, 0, z / p.group);
          else
            tma_load_3d_pair(sb + O_V + s * 16384u, &tmV, fv, 64 * (int)rank, 128 * blk, z / p.group);
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
    if (rank == 0) {
      const uint64_t dQ = sw128_desc(sb + O_Q, 16, 1024), dK = sw128_desc(sb + O_K, 16, 1024),
                     dV = sw128_desc(sb + O_V, 16384, 1024);
      uint32_t g = 0, lu = 0;
      bool ok = true;
      constexpr uint32_t NB = Tmem<FIXED>::NB;
      // S of block gg into its buffer: free, since the product that read the P in it was issued
      // before
      auto k_of = [&](uint32_t gg, bool need) {
        return fa::phase_f(&c->kfull[gg % KV_STAGES], gg / KV_STAGES, need);
      };
      auto scores = [&](uint32_t gg, uint32_t qs) {   // by the elected lane
        const uint32_t s = gg % KV_STAGES, b = gg % NB;
        const uint64_t q0 = dplus(dQ, qs * 32768u), k0 = dplus(dK, s * 16384u);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (k == 4 && p.hd <= 64) break;   // the other columns of a row are zero
          mma2_bf16(tmem + 128 * b, dplus(q0, (k >> 2) * 16384 + (k & 3) * 32),
                    dplus(k0, (k >> 2) * 8192 + (k & 3) * 32), IDESC_KK, k ? 1u : 0u);
        }
        commit2_mc(&c->kempty[s], 3);
        commit2_mc(&c->sfull[b], 3);
      };
      Unit next = unit_of(p, pid);   // loaded a unit ahead
      for (int rnd = 0, u = pid; u < p.n_units && ok; u = pk::next_unit(++rnd, pid, npairs)) {
        const auto [z, qp, j0, nj] = next;
        next = unit_of(p, pk::next_unit(rnd + 1, pid, npairs));
        if (nj <= 0) continue;
        const uint32_t qs = lu & 1u;
        if (!fa::warp_wait_all(c, p.limit_ns, fa::phase_f(&c->qfull[qs], lu >> 1), k_of(g, true), k_of(g + 1, nj > 1),
                               k_of(g + 2, NB > 2 && nj > 2))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          for (uint32_t i = 0; i < NB && (int)i < nj; ++i) scores(g + i, qs);
        }
        __syncwarp();
        for (int n = 0; n < nj; ++n, ++g) {
          const uint32_t s = g % KV_STAGES, b = g % NB;
          const bool more = n + (int)NB < nj;
          if (!fa::warp_wait_all(c, p.limit_ns, fa::phase_f(&c->pready_l[b], g / NB), fa::phase_c(&c->pready_r[b], g / NB),
                                 fa::phase_f(&c->vfull[s], g / KV_STAGES), k_of(g + NB, more),
                                 fa::phase_c(&c->accempty, lu ^ 1u, n == 0))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t v0 = dplus(dV, s * 16384u);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma2_bf16_ts(tmem + Tmem<FIXED>::O + (FIXED ? 0 : 128 * b), tmem + 128 * b + 8 * k, dplus(v0, k * 2048),
                           IDESC_KM, (n > (FIXED ? 0 : 1) || k) ? 1u : 0u);   // the accumulator's first block overwrites
            commit2_mc(&c->vempty[s], 3);
            if (more) scores(g + NB, qs);
            if (n == max(nj - (int)NB, 0)) commit2_mc(&c->qempty[qs], 3);   // every S of the unit is issued
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) commit2_mc(&c->ofull, 3);
        ++lu;
      }
      if (elect_one()) {
        if (!ok) fail_o(c, p.status);
        commit2_mc(&c->mdone, 1);
      }
      wait_inl<false>(&c->mdone, 0, nullptr, 200000000ull);
    }
    __syncwarp();
  } else if (warp >= SOFT_WARP) {
    const int q = warp & 3, grp = (warp - SOFT_WARP) >> 2;   // lane quadrant; softmax group
    const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16);
    constexpr uint32_t NB = Tmem<FIXED>::NB, T_O = Tmem<FIXED>::O;
    const int lrow = 32 * q + lane;
    // scores stay raw when they only need the scale, which the exponent's FMA applies
    constexpr bool RAW = !CAP && !BIAS;
    const float mul = RAW ? p.sc.sl2 : 1.f;
    uint32_t g = 0, lu = 0;
    bool ok = true;
    Unit next = unit_of(p, pid);   // the next unit's entry and this thread's row of it
    int nrow, nlo, nhi;
    auto row_ahead = [&]() {
      nrow = 256 * next.qp + 128 * (int)rank + lrow;
      nlo = nrow < p.T ? p.lo[nrow] : p.T;
      nhi = nrow < p.T ? p.hi[nrow] : p.T;
    };
    row_ahead();
    // The end of a unit waits until the group's first block of the next one is done: its products
    // then run meanwhile.  It joins the groups: m and l of the row's other group, then 64 columns
    // of both accumulators.
    uint32_t done = 0, left = 0;   // units joined; units whose O has left its staging block
    int zf = 0, rowf = 0;          // the unit's head, this thread's row
    auto finish = [&]() -> bool {
      if (done == lu) return true;
      const float2* ml = reinterpret_cast<const float2*>(base + O_ML) + (done & 1u) * 256;
      if (!warp_wait(&c->mlx, done, c, p.limit_ns) || !warp_wait(&c->ofull, done, c, p.limit_ns)) return false;
      tc_fence_after();
      __syncwarp();
      const float2 s0 = ml[lrow], s1 = ml[128 + lrow];
      const float mm = fmaxf(s0.x, s1.x);
      const float f0 = s0.y == 0.f ? 0.f : ex2((s0.x - mm) * mul), f1 = s1.y == 0.f ? 0.f : ex2((s1.x - mm) * mul);
      const float l = s0.y * f0 + s1.y * f1;
      const bool none = l == 0.f;   // a row that sees nothing (padding): 0 and -inf
      const float inv = none ? 0.f : 1.f / l;
      const float a0 = f0 * inv, a1 = f1 * inv;
      if (rowf < p.T && grp == 0) p.lse[(int64_t)zf * p.T + rowf] = none ? -INFINITY : (mm * mul + log2f(l)) * 0.6931471805599453f;
      // O leaves through the space of the unit's Q, which no product reads any more: two blocks
      // of 32 x 32 a warp
      const uint32_t stg = sb + O_Q + (done & 1u) * 32768u + (uint32_t)(warp - SOFT_WARP) * 4096u;
#pragma unroll
      for (int h = 0; h < 64; h += 32) {
        uint32_t ra[32], rb[32], v[16];
        __syncwarp();
        tmem_ld32(trow + T_O + 64 * grp + h, ra);
        if (!FIXED) tmem_ld32(trow + T_O + 128 + 64 * grp + h, rb);
        tmem_ld_wait();
        if (h == 32) {   // both accumulators have been read: the next unit may overwrite them
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_remote(mapa(saddr(&c->accempty), 0));
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (FIXED) {   // one accumulator, over one reference
            v[i] = none ? 0u : pack_bf16(__uint_as_float(ra[2 * i]) * inv, __uint_as_float(ra[2 * i + 1]) * inv);
            continue;
          }
          // a group without a block for the row leaves its accumulator unset: selected out
          const float x0 = f0 == 0.f ? 0.f : __uint_as_float(ra[2 * i]) * a0;
          const float x1 = f0 == 0.f ? 0.f : __uint_as_float(ra[2 * i + 1]) * a0;
          const float y0 = f1 == 0.f ? 0.f : __uint_as_float(rb[2 * i]) * a1;
          const float y1 = f1 == 0.f ? 0.f : __uint_as_float(rb[2 * i + 1]) * a1;
          v[i] = pack_bf16(x0 + y0, x1 + y1);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          sts128(stg + 64u * h + 64u * lane + 16u * k, v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0 && rowf < p.T) {
        const int col = 64 * grp;
        if (col < p.hd) tma_store_3d(&tmO, stg, col, rowf, zf);
        if (col + 32 < p.hd) tma_store_3d(&tmO, stg + 2048, col + 32, rowf, zf);
        bulk_commit();
      }
      ++done;
      return true;
    };
    auto release = [&]() {   // the Q buffer, once its O has left
      if (left == done) return;
      if (lane == 0) {
        bulk_wait_read();
        mbar_arrive(&c->qempty[left & 1u]);
      }
      ++left;
    };
    for (int rnd = 0, u = pid; ok; u = pk::next_unit(++rnd, pid, npairs)) {
      const bool end = u >= p.n_units;   // a last round joins the last unit
      const auto [z, qp, j0, nj] = next;
      const int row = nrow, lo = nlo, hi = nhi;   // the row sees the keys [lo, hi)
      const bool vrow = row < p.T;
      next = unit_of(p, pk::next_unit(rnd + 1, pid, npairs));
      const int lo1 = __shfl_sync(0xffffffffu, lo, 31), hi0 = __shfl_sync(0xffffffffu, hi, 0);
      const pk::ScaleZ sc = pk::scale_z(p.sc, BIAS ? p.slopes[z] : 0.f);
      // FIXED: the bias of the farthest key where the bias rises with the distance, else 0
      float m = FIXED ? (BIAS ? fmaxf(0.f, -sc.slope2 * (float)max(row - lo, hi - 1 - row)) : 0.f) : -INFINITY;
      const float top = sc.c2 - (FIXED ? m : 0.f);
      float2 l2 = make_float2(0.f, 0.f);
      for (int n = (int)((g ^ (uint32_t)grp) & 1u);; n += 2) {   // this group's blocks
        if (n < nj) {
          const int k0 = 128 * block_at<BIAS>(j0, nj, n);
          const Row w{lo - k0, hi - k0, lo1 - k0, hi0 - k0, row - lane - k0, (float)(row - k0), top};
          const bool edge = w.edge<BIAS>();
          // the row's first keys, or a bias that alone lifts the maximum from the group's block before
          bool raise = !FIXED && __any_sync(0xffffffffu, m == -INFINITY && w.a < 128 && w.b > 0);
          if (BIAS && !FIXED)
            raise = raise || (fabsf(sc.slope2) * 256.f > kLag && (sc.slope2 > 0.f ? w.first < 127 : w.first > -31));
          const uint32_t b = (g + n) % NB, tS = trow + 128 * b, tO = trow + T_O + 128 * grp;
          if (!warp_wait(&c->sfull[b], (g + n) / NB, c, p.limit_ns)) { ok = false; break; }
          tc_fence_after();
          __syncwarp();
          if (edge) soft_block<CAP, BIAS, FIXED, true>(tS, tO, n < 2, raise, w, sc, mul, m, l2);
          else soft_block<CAP, BIAS, FIXED, false>(tS, tO, n < 2, raise, w, sc, mul, m, l2);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) fa::arrive_leader(rank, &c->pready_l[b], &c->pready_r[b]);
        }
        release();
        if (!finish()) { ok = false; break; }
        if (n + 2 >= nj) break;
      }
      if (!ok || end) break;
      release();
      if (nj <= 0) {   // rows of padding alone
        if (vrow) {
          const int64_t ro = (int64_t)z * p.T + row;
          if (grp == 0) p.lse[ro] = -INFINITY;
          uint4* dst = reinterpret_cast<uint4*>(p.O + ro * p.hd + 64 * grp);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (64 * grp + 8 * k < p.hd) dst[k] = make_uint4(0u, 0u, 0u, 0u);
        }
        row_ahead();
        continue;
      }
      g += (uint32_t)nj;
      float2* ml = reinterpret_cast<float2*>(base + O_ML) + (lu & 1u) * 256;
      ml[grp * 128 + lrow] = make_float2(m, l2.x + l2.y);
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->mlx);
      ++lu;
      zf = z;
      rowf = row;
      row_ahead();
    }
    if (!ok) fail_o(c, p.status);
    if (lane == 0) bulk_wait_all();
    __syncwarp();
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

// Largest cap that needs no running maximum: 2^x of scores within 50 log2(e) = 72.1 lies in
// [2^-72.2, 2^72.2], which leaves 2^55 for the sums of |V| over a row's keys and 2^-53 for the
// smallest that counts (the header states both).  With a distance bias the scores less the row's largest bias take the place of x: none
// is above 72, and the key with that bias (the row's own, or the farthest) is not below -72.
// (8192 tokens in documents: cap 50 219 us, cap 50.5 314 us.)
constexpr float kStaticCap = 50.f;

template <bool CAP, bool BIAS, bool FIXED>
cudaError_t launch_o(const PackedArgs& a, const PackedWork& w, void* O, float* lse, cudaStream_t s) {
  using namespace tc::fo;
  static int attr_state[64] = {};
  static std::mutex mu;
  if (!tc::once_per_device(attr_state, mu, [] {
        return cudaFuncSetAttribute(k_attn_o<CAP, BIAS, FIXED>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM) ==
               cudaSuccess;
      }))
    return cudaErrorInvalidConfiguration;
  Params p;
  p.H = (int)a.H; p.T = (int)a.T; p.hd = (int)a.hd; p.group = (int)(a.H / a.Hkv);
  p.n_units = (int)((a.T + 255) / 256 * a.H);
  p.sc = tc::pk::make_scale(a.scale, a.softcap);
  p.slopes = a.slopes; p.units = w.qunits; p.lo = w.lo; p.hi = w.hi; p.tail = w.tail;
  p.O = static_cast<__nv_bfloat16*>(O); p.lse = lse; p.status = a.status; p.limit_ns = tc::wait_limit_ns();
  CUtensorMap mQ, mK, mV, mVt, mO;
  if (!tc::make_map_heads(&mQ, a.Q, a.T, a.H, a.hd, 128) || !tc::make_map_heads(&mK, a.K, a.T, a.Hkv, a.hd, 64) ||
      !tc::make_map_heads(&mV, a.V, a.T, a.Hkv, a.hd, 128) ||
      !tc::make_map_heads(&mVt, w.tail_kv, 128, a.Hkv, a.hd, 128) || !tc::make_map_out(&mO, O, a.T, a.T, a.H, a.hd, 2))
    return cudaErrorInvalidValue;
  const int pairs = std::min(tc::max_pairs((const void*)k_attn_o<CAP, BIAS, FIXED>, SMEM, THREADS), p.n_units);
  return tc::launch_early(k_attn_o<CAP, BIAS, FIXED>, 2 * pairs, THREADS, SMEM, s, mQ, mK, mV, mVt, mO, p);
}

}  // namespace

cudaError_t packed_forward(const PackedArgs& a, const PackedWork& w, void* O, float* lse, cudaStream_t s) {
  if (a.softcap > 0.f && a.softcap <= kStaticCap)
    return a.slopes ? launch_o<true, true, true>(a, w, O, lse, s) : launch_o<true, false, true>(a, w, O, lse, s);
  if (a.softcap > 0.f)
    return a.slopes ? launch_o<true, true, false>(a, w, O, lse, s) : launch_o<true, false, false>(a, w, O, lse, s);
  return a.slopes ? launch_o<false, true, false>(a, w, O, lse, s) : launch_o<false, false, false>(a, w, O, lse, s);
}

}  // namespace sbp
