// Fused tensor-core kernels of the chunked causal-attention backward at head dimension
// 128 (bf16 operands, fp32 accumulation, sm_103a).
//
// Per chunk of queries [c0, c1), which reads keys [0, c1) only (the causal structure
// StreamBP uses), two SM-pair kernels keep the chunk's probabilities and score gradients
// on chip: nothing of size (queries x keys) goes through HBM.
//
//   k_attn_kv  unit = (head, 256 keys).  dV and dK of those keys stay in tensor memory
//              while the unit walks the chunk's query blocks of 128:
//                S^T = K Q^T,  dP^T = V dO^T                      (tensor memory)
//                P^T = exp(s S^T - lse),  dS^T = P^T (dP^T - D)   (written over S^T and dP^T)
//                dV += P^T dO,  dK += dS^T Q                      (A from tensor memory)
//              then adds dV and s dK into the fp32 outputs (TMA reduce-add) or writes them.
//              The two streams S -> P -> dV and dP -> dS -> dK take turns: while the
//              epilogue works on one, the tensor pipe runs the other's products.  A block takes
//              about 3000 cycles, 2070 of them the tensor pipe's; the epilogue's work is as
//              long, and the handoffs between the two show (32 / 8 heads, 8192 tokens, one
//              document: tensor pipe 69% active, k_attn_q 80%).
//   k_attn_q   unit = (head, 256 queries of the chunk).  dQ stays in tensor memory while
//              the unit walks the key blocks of 128 up to its last query:
//                S = Q K^T,  dP = dO V^T,  dS = P (dP - D),  dQ += dS K
//              then stores s dQ in bf16.
// S and dP are formed in both kernels, so that no accumulator is shared between units:
// every output element is written by one unit in a fixed order (deterministic, no
// floating-point atomics).
//
// Both kernels are templates over a score policy, which says which (query, key) pairs a
// unit walks and sees, how a score becomes a logarithm of a probability, how dK and dV
// leave, and whether k_attn_q takes D from P and dP first: CausalScores (below, the chunked causal attention) and PackedScores
// (sbp_attn_packed.cu: packed documents, prefixes, capped and biased scores).
//
// Pair protocol as in the other tensor-core kernels: the leader CTA's thread issues
// tcgen05.mma cta_group::2 with M = 256 (128 rows in each CTA) and N = 128 (each CTA
// supplies half of B); TMA copies of both CTAs complete on the leader's barriers; the
// commits are multicast to both CTAs; every wait is bounded in time.
#pragma once

#include "sbp_tc_common.cuh"

namespace sbp {
namespace tc {
namespace fa {

// Warps: 0 TMA producers, 1 MMA issuer (leader CTA), then the epilogue warps (lane quadrant
// warp % 4, 32 of the 128 columns each), then (k_attn_kv) one warp that stages lse and D per
// block.  The epilogue warps arrive at the leader's barriers, one for its own warps and one
// for the other CTA's.  (One lane of that CTA turning local phases into one remote arrival
// each: causal benchmark 6.10M tokens/s, 6.25M without.)
constexpr int Q_EPI = 16, KV_EPI = 16;
constexpr int KV_LD_WARP = 2 + KV_EPI;
constexpr int KV_THREADS = 32 * (KV_LD_WARP + 1);   // five warps a scheduler: 96 registers a thread
constexpr int Q_THREADS = 32 * (2 + Q_EPI);
constexpr uint32_t IDESC_KK = idesc_bf16(256, 128, false, false);  // A, B K-major
constexpr uint32_t IDESC_KM = idesc_bf16(256, 128, false, true);   // A K-major, B MN-major

// Shared memory of k_attn_kv, bytes from the 1024-aligned base.  Tiles are 128-byte
// swizzled: [64-element block][rows][128 B].
constexpr uint32_t KV_K = 0;          // K rows of the unit (this CTA's 128 keys x 128)
constexpr uint32_t KV_V = 32768;      // V rows
constexpr uint32_t KV_AQ = 65536;     // 2 stages: Q of the block, this CTA's 64 queries x 128 (B of S^T)
constexpr uint32_t KV_AO = 98304;     // 2 stages: dO of the block, likewise (B of dP^T)
constexpr uint32_t KV_BQ = 131072;    // Q of the block, 128 queries x this CTA's 64 of hd (B of dK)
constexpr uint32_t KV_BO = 147456;    // dO of the block, likewise (B of dV)
constexpr uint32_t KV_STG = 163840;   // one 32 x 32 fp32 block of dV or dK an epilogue warp
constexpr uint32_t KV_LD = 229376;    // -lse * log2(e) [2 stages][128], then -D [128], of the block's queries
constexpr uint32_t KV_CTRL = 230912;
// Tensor memory of k_attn_kv: S^T (P^T over it), dP^T (dS^T over it), dV, dK.
constexpr uint32_t KT_DP = 128, KT_DV = 256, KT_DK = 384;

// Shared memory of k_attn_q: Q and dO of two units, two stages of each key-block operand.
constexpr uint32_t Q_R = 0;           // Q then dO rows of the unit (this CTA's 128 queries x 128 each)
constexpr uint32_t Q_K = 131072;      // K of the key block, this CTA's 64 keys x 128 (B of S)
constexpr uint32_t Q_V = 163840;      // V of the key block, likewise (B of dP)
constexpr uint32_t Q_Y = 196608;      // K of the key block, 128 keys x this CTA's 64 of hd (B of dQ)
constexpr uint32_t Q_CTRL = 229376;
// Tensor memory of k_attn_q: two S buffers (dS over them), dP, dQ.
constexpr uint32_t QT_DP = 256, QT_DQ = 384;

struct CtrlQ {
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2], yfull[2], yempty[2];
  uint64_t rfull[2], rempty[2];   // the unit's Q and dO; free: their products are done, and dQ has left
  uint64_t tfull;                 // S and dP of the block are ready
  // dP has been read, dS buffer is written: the leader's epilogue warps, and the other CTA's (leader)
  uint64_t tempty_l, oready_l[2], tempty_r, oready_r[2];
  uint64_t dqfull, accempty;      // the unit's dQ is complete; has been read out (leader)
  uint64_t sums[4];               // the four warps of a lane quadrant have left their rows' sums
  uint64_t mdone;
  uint32_t tmem_base;
  int abort;
};

struct CtrlF {
  uint64_t qfull[2], qempty[2], ofull[2], oempty[2];   // K-major Q and dO of the block
  uint64_t bqfull, bqempty, bofull, boempty;           // the same 128 queries x half of hd
  uint64_t rfull, rempty;        // the unit's K and V
  uint64_t sfull, dpfull;        // S^T / dP^T of the block is ready (both CTAs)
  // P^T / dS^T is written: the leader's epilogue warps, and the other CTA's (leader)
  uint64_t pready_l, dsready_l, pready_r, dsready_r;
  uint64_t accfull, accempty;    // the unit's dV and dK are complete; have been read out (leader)
  uint64_t lfull[2], lempty[2], dfull, dempty;   // lse (2 stages) and D of the block
  uint64_t mdone;
  uint32_t tmem_base;
  int abort;
};

constexpr size_t SMEM_KV = KV_CTRL + sizeof(CtrlF) + 1024;
constexpr size_t SMEM_Q = Q_CTRL + sizeof(CtrlQ) + 1024;
static_assert(SMEM_KV <= 232448 && SMEM_Q <= 232448, "shared memory of one CTA");

// Tensor memory and the barriers visible to the pair.
template <class C>
__device__ __forceinline__ void prologue_end(C* c, int warp) {
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
}
__device__ __forceinline__ void prologue_f(CtrlF* c, int warp) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c->qfull[i], 1);
      mbar_init(&c->qempty[i], 1);
      mbar_init(&c->ofull[i], 1);
      mbar_init(&c->oempty[i], 1);
      mbar_init(&c->lfull[i], 1);
      mbar_init(&c->lempty[i], KV_EPI);
    }
    mbar_init(&c->bqfull, 1);
    mbar_init(&c->bqempty, 1);
    mbar_init(&c->bofull, 1);
    mbar_init(&c->boempty, 1);
    mbar_init(&c->rfull, 1);
    mbar_init(&c->rempty, 1);
    mbar_init(&c->sfull, 1);
    mbar_init(&c->dpfull, 1);
    mbar_init(&c->pready_r, KV_EPI);
    mbar_init(&c->dsready_r, KV_EPI);
    mbar_init(&c->pready_l, KV_EPI);
    mbar_init(&c->dsready_l, KV_EPI);
    mbar_init(&c->accfull, 1);
    mbar_init(&c->accempty, 2 * KV_EPI);
    mbar_init(&c->dfull, 1);
    mbar_init(&c->dempty, KV_EPI);
    mbar_init(&c->mdone, 1);
    c->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  prologue_end(c, warp);
}
__device__ __forceinline__ void prologue_q(CtrlQ* c, int warp) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c->kfull[i], 1);
      mbar_init(&c->kempty[i], 1);
      mbar_init(&c->vfull[i], 1);
      mbar_init(&c->vempty[i], 1);
      mbar_init(&c->yfull[i], 1);
      mbar_init(&c->yempty[i], 1);
      mbar_init(&c->rfull[i], 1);
      mbar_init(&c->rempty[i], 1 + Q_EPI);
      mbar_init(&c->oready_r[i], Q_EPI);
      mbar_init(&c->oready_l[i], Q_EPI);
    }
    mbar_init(&c->tfull, 1);
    mbar_init(&c->tempty_r, Q_EPI);
    mbar_init(&c->tempty_l, Q_EPI);
    mbar_init(&c->dqfull, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&c->sums[i], Q_EPI / 4);
    mbar_init(&c->accempty, 2 * Q_EPI);
    mbar_init(&c->mdone, 1);
    c->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  prologue_end(c, warp);
}

template <class C>
__device__ __forceinline__ void teardown_f(C* c, int warp) {
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(c->tmem_base), "r"(TMEM_COLS)
                 : "memory");
  }
}

template <class C>
__device__ __forceinline__ void fail_f(C* c, int32_t* status) {
  *(volatile int*)&c->abort = 1;
  if (status) atomicCAS(status, 0, SBP_ERR_TIMEOUT);
}

// One phase, by its parity: of a barrier that only this CTA or the tensor pipe completes
// (_f), or that the pair's other CTA may complete (_c).
template <class C>
__device__ __forceinline__ bool warp_wait_f(uint64_t* b, uint32_t parity, C* c, uint64_t limit) {
  return __all_sync(0xffffffffu, wait_inl<false>(b, parity & 1u, &c->abort, limit));
}
template <class C>
__device__ __forceinline__ bool wait_c(uint64_t* b, uint32_t parity, C* c, uint64_t limit) {
  return wait_inl<true>(b, parity & 1u, &c->abort, limit);
}
template <class C>
__device__ __forceinline__ bool warp_wait_c(uint64_t* b, uint32_t parity, C* c, uint64_t limit) {
  return __all_sync(0xffffffffu, wait_c(b, parity, c, limit));
}
// An epilogue warp's arrival at the leader: on its barrier for its own warps or for the other CTA's.
__device__ __forceinline__ void arrive_leader(uint32_t rank, uint64_t* local, uint64_t* remote) {
  if (rank == 0) mbar_arrive(local);
  else arrive_remote(mapa(saddr(remote), 0));
}

// Several phases at once: a wait costs the MMA warp some 150 cycles even when its phase has
// completed, and with one wait for each operand that warp, not the tensor pipe, set the pace.
// The tests go out together; only what is not there yet is waited for.
template <bool CLUSTER>
struct Phase {
  uint64_t* b;
  uint32_t parity;
  bool need;   // false: passes
  __device__ __forceinline__ bool test() const {
    return !need || (CLUSTER ? mbar_test<true>(b, parity & 1u) : mbar_test<false>(b, parity & 1u));
  }
  __device__ __forceinline__ bool wait(const volatile int* abort_flag, uint64_t limit) const {
    return wait_inl<CLUSTER>(b, parity & 1u, abort_flag, limit);
  }
};
// (see warp_wait_f and warp_wait_c)
__device__ __forceinline__ Phase<false> phase_f(uint64_t* b, uint32_t parity, bool need = true) { return {b, parity, need}; }
__device__ __forceinline__ Phase<true> phase_c(uint64_t* b, uint32_t parity, bool need = true) { return {b, parity, need}; }
template <class C, class... P>
__device__ __forceinline__ bool warp_wait_all(C* c, uint64_t limit, const P&... ph) {
  bool there[] = {ph.test()...};
  int i = 0;
  bool all = true;
  ((all = all && there[i++], (void)ph), ...);
  if (__all_sync(0xffffffffu, all)) return true;
  i = 0;
  bool ok = true;
  ((ok = ok && (there[i++] || ph.wait(&c->abort, limit))), ...);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void tma_reduce_add_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}

// 2^a and 2^b (fp32 special-function unit; measured faster here than the packed
// half-precision form, whose conversions cost more than the halved exp count saves).
__device__ __forceinline__ float2 exp2_pair(float a, float b) { return make_float2(ex2(a), ex2(b)); }

// Descriptor d advanced by `bytes` (a multiple of 16 that keeps the start address inside
// its 14-bit field): one 32-bit add on the low word instead of rebuilding the descriptor
// for every operand and k-step.
__device__ __forceinline__ uint64_t dplus(uint64_t d, uint32_t bytes) {
  return (d & 0xFFFFFFFF00000000ull) | (uint64_t)((uint32_t)d + (bytes >> 4));
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// tcgen05.mma with A in tensor memory (each CTA's 128 rows in its lanes, two bf16 of
// consecutive K per 32-bit column, the lower K in the low half) and B in shared memory.
__device__ __forceinline__ void mma2_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                             uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(
          d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, uint32_t r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r) : "memory");
}
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t& r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 16 lanes (rows) x 32 columns as accumulator fragments: of column group g (8 columns) thread t
// holds row t / 4, columns 2 (t % 4) and + 1, in r[4 g] and r[4 g + 1], and row t / 4 + 8 in the
// next two.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// The same fragment packed to bf16 pairs, 16 columns: of group g row t / 4 in r[2 g], row
// t / 4 + 8 in r[2 g + 1], at column 4 g + t % 4.
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// ================================================================ k_attn_kv (dK, dV)

// k_attn_kv's epilogue, a warp's 32 keys x 32 queries.  First P^T = 2^(s S^T - lse log2 e), packed
// to bf16 pairs and kept in fp32 (over the scores, times the factors of the scores' gradients
// where a policy has them); then dS^T = P^T (dP^T - D).  The scores are held as accumulator
// fragments, [half of 16 keys][tmem_ld_frag], so that a thread meets 8 of the 32 queries
// only: their lse and D come from shared memory in 8 loads a block, where a key row a thread
// took 64 floats, a wavefront each, and the two kept the shared-memory pipe busy for
// half of the epilogue.
// MASK: some key of the warp is not seen by all 32 queries; the other blocks skip the
// per-element test (it costs more than the math it guards).
struct KvRows {
  int lo, hi;     // queries that see key kw + lane; fragment row 2 h + e is key kw + 16 h + 8 e + lane / 4
  int key;        // fragment row 0
};
template <class S, bool MASK>
__device__ __forceinline__ void kv_probs(uint32_t (&r)[16], int h, const float2 (&nlse)[4], const typename S::Scale& sc,
                                         int q0, const KvRows& w, uint32_t (&pw)[8]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int row = 16 * h + 8 * e;
    const float fd = (float)(q0 - (w.key + row));   // (past 2^24 the rows themselves are not fp32 values)
    int lo = 0, hi = 0;
    if (MASK) {
      lo = __shfl_sync(0xffffffffu, w.lo, row + (threadIdx.x & 31) / 4);
      hi = __shfl_sync(0xffffffffu, w.hi, row + (threadIdx.x & 31) / 4);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint32_t &r0 = r[4 * g + 2 * e], &r1 = r[4 * g + 2 * e + 1];
      float2 dc;
      const float2 x = S::template log2p2<MASK>(sc, make_float2(__uint_as_float(r0), __uint_as_float(r1)), nlse[g], fd, (float)(8 * g),
                                 (float)(8 * g + 1), dc);
      float2 pp = exp2_pair(x.x, x.y);
      const int q = q0 + 8 * g;
      if (MASK && (q < lo || q >= hi)) pp.x = 0.f;
      if (MASK && (q + 1 < lo || q + 1 >= hi)) pp.y = 0.f;
      pw[2 * g + e] = pack_bf16(pp.x, pp.y);
      pp = S::fold(pp, dc);
      r0 = __float_as_uint(pp.x);
      r1 = __float_as_uint(pp.y);
    }
  }
}
template <class S, bool MASK>
__device__ __forceinline__ void kv_grads(const uint32_t (&rp)[16], const uint32_t (&rd)[16], int h, const float2 (&nD)[4],
                                         int q0, const KvRows& w, uint32_t (&dw)[8]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int row = 16 * h + 8 * e;
    int lo = 0, hi = 0;
    if (S::kClearMasked && MASK) {
      lo = __shfl_sync(0xffffffffu, w.lo, row + (threadIdx.x & 31) / 4);
      hi = __shfl_sync(0xffffffffu, w.hi, row + (threadIdx.x & 31) / 4);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int i = 4 * g + 2 * e;
      float2 sv = mul2(make_float2(__uint_as_float(rp[i]), __uint_as_float(rp[i + 1])),
                       add2(make_float2(__uint_as_float(rd[i]), __uint_as_float(rd[i + 1])), nD[g]));
      const int q = q0 + 8 * g;
      if (S::kClearMasked && MASK && (q < lo || q >= hi)) sv.x = 0.f;
      if (S::kClearMasked && MASK && (q + 1 < lo || q + 1 >= hi)) sv.y = 0.f;
      dw[2 * g + e] = pack_bf16(sv.x, sv.y);
    }
  }
}

struct KvP {
  int H, T, c0, c1, nb, n_units;
  int Hkv, group;    // key / value heads; query heads per key / value head (H = Hkv * group)
  float scale;
  const float* lse;  // [H, T]
  const float* D;    // [H, T]
  int32_t* status;
  uint64_t limit_ns;
};

struct QP {
  int H, T, c0, c1, n_qp, n_units;
  int group;         // query heads per key / value head
  float scale;
  const float* lse;
  const float* D;
  int32_t* status;
  uint64_t limit_ns;
};

// Tensor maps of the kernels.  k_attn_kv: K, V (the unit's 128-key rows), Q, dO (64 queries
// of a block), Q, dO (128 queries x half of hd), and the fp32 outputs dK, dV;
// k_attn_q: Q, dO (128-query rows), K, V (64 keys of a block), K (128 keys x half of hd), and the
// output dQ.
// A policy with kTail names one block (tail_block) whose rows the accumulating products take from
// other maps (one block a head): Q, dO (in the place of the fp32 outputs) and K; it may have
// output maps of its own behind.
enum { KV_MK, KV_MV, KV_MQA, KV_MOA, KV_MQB, KV_MOB, KV_MDK, KV_MDV, KV_MAPS, KV_MQT = KV_MDK, KV_MOT = KV_MDV,
       KV_MOUTK = KV_MAPS, KV_MOUTV };
enum { Q_MQ, Q_MO, Q_MKA, Q_MVA, Q_MKB, Q_MOUT, Q_MAPS, Q_MKT = Q_MAPS };
template <int N>
struct MapArray {   // in the kernel's parameters
  CUtensorMap m[N];
  __device__ __forceinline__ const CUtensorMap* operator[](int i) const { return &m[i]; }
  template <int I>
  __device__ __forceinline__ const CUtensorMap* at() const {
    static_assert(I < N, "a map that this policy does not have");
    return &m[I];
  }
};

// Row `lane` of a warp's 32 x 32 staging block, times f: fp32 with the 128-byte swizzle, or
// bf16 rows of 64 bytes.
__device__ __forceinline__ void stage_f32(const uint32_t (&ra)[32], float f, uint32_t stg, int lane) {
  const uint32_t buf = stg + (uint32_t)lane * 128u;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    sts128(buf + ((uint32_t)(k ^ (lane & 7)) << 4), __float_as_uint(__uint_as_float(ra[4 * k]) * f),
           __float_as_uint(__uint_as_float(ra[4 * k + 1]) * f), __float_as_uint(__uint_as_float(ra[4 * k + 2]) * f),
           __float_as_uint(__uint_as_float(ra[4 * k + 3]) * f));
}
__device__ __forceinline__ void stage_bf16(const uint32_t (&ra)[32], float f, uint32_t stg, int lane) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = pack_bf16(__uint_as_float(ra[2 * i]) * f, __uint_as_float(ra[2 * i + 1]) * f);
  const uint32_t buf = stg + (uint32_t)lane * 64u;
#pragma unroll
  for (int k = 0; k < 4; ++k) sts128(buf + 16u * k, w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
}

// A unit of k_attn_kv: key / value head zk, keys [256 kp, +256), query blocks [b0, b0 + nbl) of
// each of the query heads [z0, z0 + nh); `plane` says where its dK and dV go.
struct KvUnit { int zk, kp, b0, nbl, z0, nh, plane; };

// The key blocks [j, j + n) that a unit of k_attn_q walks before its own, for the rows' sums of
// P (dP - D) alone.
struct SumBlocks { int j, n; };

// Chunked causal attention: query i of the chunk [c0, c1) sees the keys 0 .. i.
struct CausalScores {
  using Kv = KvP;
  using Q = QP;
  using KvMaps = MapArray<KV_MAPS>;
  using QMaps = MapArray<Q_MAPS>;
  static constexpr bool kClearMasked = false;
  static constexpr bool kAddOut = true;   // dK, dV are added into fp32 outputs
  using Scale = float;                    // scale * log2(e)

  // The unit of round t of SM pair pid.
  static __device__ __forceinline__ int next_unit(int t, int pid, int npairs) { return t * npairs + pid; }
  // Unit u: key / value head zk, keys [256 kp, 256 kp + 256); query blocks b0 .. nb-1 of
  // the chunk hold at least one query at or after the unit's first key.  The unit walks
  // those nbl blocks for each query head of zk's group, accumulating dV and dK of the
  // shared head.  Key pairs in ascending order, so the longest units start first.
  // (a policy whose units come from memory loads them ahead: kv_raw, q_raw)
  struct Raw {};
  static __device__ __forceinline__ Raw kv_raw(const KvP&, int) { return Raw{}; }
  static __device__ __forceinline__ Raw q_raw(const QP&, int) { return Raw{}; }
  static __device__ __forceinline__ void kv_unit(const KvP& p, int u, Raw, KvUnit& w) {
    w.kp = u / p.Hkv;
    w.zk = u - w.kp * p.Hkv;
    const int num = 256 * w.kp - p.c0 - 127;
    w.b0 = num <= 0 ? 0 : (num + 127) / 128;
    w.nbl = p.nb - w.b0;
    w.z0 = w.zk * p.group;
    w.nh = p.group;
    w.plane = w.zk;
  }
  // Queries [lo, hi) that see a key; both ends do not decrease with the key.  A warp's 32
  // keys from kw: lowest and highest of each end.
  static __device__ __forceinline__ void key_range(const KvP& p, int key, int& lo, int& hi) {
    lo = key;
    hi = p.c1;
  }
  static __device__ __forceinline__ void key_warp(const KvP& p, int kw, int, int, int& lo0, int& lo1, int& hi0,
                                                  int& hi1) {
    lo0 = kw;
    lo1 = kw + 31;
    hi0 = hi1 = p.c1;
  }

  // Unit u: head z, queries [c0 + 256 qp, +256) of the chunk, key blocks j0 .. j0+nj-1 (128
  // keys each) up to the unit's last query.  Later query pairs (more keys) first.
  static __device__ __forceinline__ void q_unit(const QP& p, int u, Raw, int& z, int& qp, int& j0, int& nj) {
    const int i = u / p.H;
    z = u - i * p.H;
    qp = p.n_qp - 1 - i;
    const int qend = min(p.c0 + 256 * qp + 256, p.c1);
    j0 = 0;
    nj = (qend + 127) / 128;
  }
  // Keys [lo, hi) that a query sees (a row past the chunk's end: none).
  static __device__ __forceinline__ void query_range(const QP& p, int q, int& lo, int& hi) {
    lo = 0;
    hi = q < p.c1 ? q + 1 : 0;
  }
  static __device__ __forceinline__ void query_warp(const QP& p, int qw, int, int, int& lo0, int& lo1, int& hi0,
                                                    int& hi1) {
    lo0 = lo1 = 0;
    hi0 = qw + 31 < p.c1 ? qw + 1 : 0;
    hi1 = qw < p.c1 ? qw + 32 : 0;
  }

  template <class P>
  static __device__ __forceinline__ Scale scale_of(const P& p, int) { return p.scale * L2E; }
  // log2 of the probabilities of two neighbouring pairs from their raw scores s, -lse in log2
  // units and their distances query - key, d + o0 and d + o1; dc: the factors of the scores'
  // gradients.  MASK: one of the two may be masked.
  template <bool>
  static __device__ __forceinline__ float2 log2p2(Scale sl2, float2 s, float2 nlz, float, float, float, float2& dc) {
    dc = make_float2(1.f, 1.f);
    return fma2(s, make_float2(sl2, sl2), nlz);
  }
  // A probability times the factor of its score's gradient.
  static __device__ __forceinline__ float2 fold(float2 p, float2) { return p; }
  static constexpr bool kTail = false;

  // How a warp's 32 x 32 block of dV (t = 0) or dK (t = 1) leaves: whether it does, one row of
  // it into the warp's staging block, and the copy out of that (fp32, 128-byte swizzle; added
  // into the outputs).  Rows past T are clipped by the tensor map, rows in [c1, T) add 0.
  static __device__ __forceinline__ bool kv_leaves(const KvP& p, int kw, int) { return kw < p.c1; }
  static __device__ __forceinline__ void kv_stage(const KvP& p, int t, const uint32_t (&ra)[32], uint32_t stg, int lane) {
    stage_f32(ra, t ? p.scale : 1.f, stg, lane);
  }
  static __device__ __forceinline__ void kv_copy(const KvMaps& maps, const KvP&, int t, uint32_t stg, int c, int kw,
                                                 const KvUnit& w) {
    tma_reduce_add_3d(maps[t ? KV_MDK : KV_MDV], stg, c, kw, w.zk);
  }
  static constexpr bool kSumFirst = false;
  struct Large {};
  static __device__ __forceinline__ Large q_large(const QP&, int, Raw) { return Large{}; }
  static __device__ __forceinline__ SumBlocks q_sums(Raw, Large) { return SumBlocks{0, 0}; }
  // Whether the products that sum over hd have columns past 64; hd.
  template <class P>
  static __device__ __forceinline__ bool wide(const P&) { return true; }
  static __device__ __forceinline__ int width(const QP&) { return 128; }
};

// A unit's blocks in order: query head z, query block b.  Returns whether z is another.
__device__ __forceinline__ bool kv_next(const KvUnit& w, int& z, int& b) {
  if (++b < w.b0 + w.nbl) return false;
  b = w.b0;
  ++z;
  return true;
}

template <class S>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(KV_THREADS, 1)
    k_attn_kv(const __grid_constant__ typename S::KvMaps maps, const typename S::Kv p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  CtrlF* c = reinterpret_cast<CtrlF*>(base + KV_CTRL);
  const uint32_t sb = saddr(base);
  const int warp = uniform_warp(), lane = threadIdx.x % 32;
  const uint32_t rank = ctarank();
  prologue_f(c, warp);
  wait_for_primary();
  const uint32_t tmem = c->tmem_base;
  const int pid = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (warp == 0) {
    if (lane == 0) {
      // the unit's K and V, then Q and dO of each block (this CTA's 64 queries)
      prefetch_map(maps[KV_MK]);
      prefetch_map(maps[KV_MV]);
      prefetch_map(maps[KV_MQA]);
      prefetch_map(maps[KV_MOA]);
      uint32_t g = 0, go = 0, lu = 0;   // blocks (Q; dO) and units loaded so far
      bool ok = true;
      typename S::Raw raw = S::kv_raw(p, pid);
      for (int rnd = 0, u = pid; u < p.n_units && ok; u = S::next_unit(++rnd, pid, npairs)) {
        KvUnit w;
        S::kv_unit(p, u, raw, w);
        raw = S::kv_raw(p, S::next_unit(rnd + 1, pid, npairs));
        const int nblk = w.nh * w.nbl;
        if (nblk == 0) continue;
        if (!wait_c(&c->rempty, lu ^ 1u, c, p.limit_ns)) { ok = false; break; }
        const uint32_t fr = mapa(saddr(&c->rfull), 0);
        if (rank == 0) mbar_expect_tx(&c->rfull, 4u * 32768u);
        const int krow = 256 * w.kp + 128 * (int)rank;
#pragma unroll
        for (int hb = 0; hb < 2; ++hb) {
          tma_load_3d_pair(sb + KV_K + hb * 16384, maps[KV_MK], fr, 64 * hb, krow, w.zk);
          tma_load_3d_pair(sb + KV_V + hb * 16384, maps[KV_MV], fr, 64 * hb, krow, w.zk);
        }
        ++lu;
        for (int n = 0, z = w.z0, b = w.b0; n < nblk; ++n, kv_next(w, z, b)) {
          const uint32_t s = g & 1u, ph = (g >> 1) ^ 1u;
          const int qrow = p.c0 + 128 * b + 64 * (int)rank;
          if (!wait_c(&c->qempty[s], ph, c, p.limit_ns)) { ok = false; break; }
          const uint32_t fq = mapa(saddr(&c->qfull[s]), 0), fo = mapa(saddr(&c->ofull[s]), 0);
          if (rank == 0) mbar_expect_tx(&c->qfull[s], 2u * 16384u);
#pragma unroll
          for (int hb = 0; hb < 2; ++hb)
            tma_load_3d_pair(sb + KV_AQ + s * 16384u + hb * 8192, maps[KV_MQA], fq, 64 * hb, qrow, z);
          ++g;
          if (!wait_c(&c->oempty[s], ph, c, p.limit_ns)) { ok = false; break; }
          if (rank == 0) mbar_expect_tx(&c->ofull[s], 2u * 16384u);
#pragma unroll
          for (int hb = 0; hb < 2; ++hb)
            tma_load_3d_pair(sb + KV_AO + s * 16384u + hb * 8192, maps[KV_MOA], fo, 64 * hb, qrow, z);
          ++go;
        }
      }
      if (!ok) {   // wait for the copies in flight
        fail_f(c, p.status);
        if (rank == 0) {
          if (lu) wait_inl<false>(&c->rfull, (lu - 1) & 1u, nullptr, 200000000ull);
          for (uint32_t i = g > 2 ? g - 2 : 0; i < g; ++i)
            wait_inl<false>(&c->qfull[i & 1u], (i >> 1) & 1u, nullptr, 200000000ull);
          for (uint32_t i = go > 2 ? go - 2 : 0; i < go; ++i)
            wait_inl<false>(&c->ofull[i & 1u], (i >> 1) & 1u, nullptr, 200000000ull);
        }
      }
    } else if (lane == 16) {
      // dO and Q of each block, 128 queries x this CTA's half of hd
      prefetch_map(maps[KV_MQB]);
      prefetch_map(maps[KV_MOB]);
      int tail = -1;
      if constexpr (S::kTail) tail = S::tail_block(p);
      uint32_t g = 0, gq = 0;
      bool ok = true;
      typename S::Raw raw = S::kv_raw(p, pid);
      for (int rnd = 0, u = pid; u < p.n_units && ok; u = S::next_unit(++rnd, pid, npairs)) {
        KvUnit w;
        S::kv_unit(p, u, raw, w);
        raw = S::kv_raw(p, S::next_unit(rnd + 1, pid, npairs));
        const int nblk = w.nh * w.nbl;
        for (int n = 0, z = w.z0, b = w.b0; n < nblk; ++n, kv_next(w, z, b)) {
          const int qrow = p.c0 + 128 * b;
          if (!wait_c(&c->boempty, g ^ 1u, c, p.limit_ns)) { ok = false; break; }
          const uint32_t fo = mapa(saddr(&c->bofull), 0), fq = mapa(saddr(&c->bqfull), 0);
          if (rank == 0) mbar_expect_tx(&c->bofull, 2u * 16384u);
          const CUtensorMap *mo = maps[KV_MOB], *mq = maps[KV_MQB];
          int row = qrow;
          if constexpr (S::kTail)
            if (b == tail) {
              mo = maps.template at<KV_MOT>();
              mq = maps.template at<KV_MQT>();
              row = 0;
            }
          tma_load_3d_pair(sb + KV_BO, mo, fo, 64 * (int)rank, row, z);
          ++g;
          if (!wait_c(&c->bqempty, gq ^ 1u, c, p.limit_ns)) { ok = false; break; }
          if (rank == 0) mbar_expect_tx(&c->bqfull, 2u * 16384u);
          tma_load_3d_pair(sb + KV_BQ, mq, fq, 64 * (int)rank, row, z);
          ++gq;
        }
      }
      if (!ok) {
        fail_f(c, p.status);
        if (rank == 0) {
          if (g) wait_inl<false>(&c->bofull, (g - 1) & 1u, nullptr, 200000000ull);
          if (gq) wait_inl<false>(&c->bqfull, (gq - 1) & 1u, nullptr, 200000000ull);
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {   // the whole warp, converged; one elected lane issues
      const uint64_t dK = sw128_desc(sb + KV_K, 16, 1024), dV = sw128_desc(sb + KV_V, 16, 1024),
                     dAQ = sw128_desc(sb + KV_AQ, 16, 1024), dAO = sw128_desc(sb + KV_AO, 16, 1024),
                     dBQ = sw128_desc(sb + KV_BQ, 16384, 1024), dBO = sw128_desc(sb + KV_BO, 16384, 1024);
      const bool wide = S::wide(p);
      uint32_t g = 0, lu = 0;
      bool ok = true;
      // S^T (dP^T) of block gg into its one buffer: free, since the product that read the P^T
      // (dS^T) of the block before in it was issued before
      auto scores = [&](uint32_t gg) {   // by the elected lane
        const uint32_t s = gg & 1u;
        const uint64_t q0 = dplus(dAQ, s * 16384u);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (k == 4 && !wide) break;
          mma2_bf16(tmem, dplus(dK, (k >> 2) * 16384 + (k & 3) * 32), dplus(q0, (k >> 2) * 8192 + (k & 3) * 32),
                    IDESC_KK, k ? 1u : 0u);
        }
        commit2_mc(&c->qempty[s], 3);
        commit2_mc(&c->sfull, 3);
      };
      auto grads = [&](uint32_t gg, bool last) {
        const uint32_t s = gg & 1u;
        const uint64_t o0 = dplus(dAO, s * 16384u);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (k == 4 && !wide) break;
          mma2_bf16(tmem + KT_DP, dplus(dV, (k >> 2) * 16384 + (k & 3) * 32),
                    dplus(o0, (k >> 2) * 8192 + (k & 3) * 32), IDESC_KK, k ? 1u : 0u);
        }
        commit2_mc(&c->oempty[s], 3);
        commit2_mc(&c->dpfull, 3);
        if (last) commit2_mc(&c->rempty, 3);
      };
      auto q_of = [&](uint32_t gg, bool need) { return phase_f(&c->qfull[gg & 1u], gg >> 1, need); };
      auto o_of = [&](uint32_t gg, bool need) { return phase_f(&c->ofull[gg & 1u], gg >> 1, need); };
      typename S::Raw raw = S::kv_raw(p, pid);
      for (int rnd = 0, u = pid; u < p.n_units && ok; u = S::next_unit(++rnd, pid, npairs)) {
        KvUnit w;
        S::kv_unit(p, u, raw, w);
        raw = S::kv_raw(p, S::next_unit(rnd + 1, pid, npairs));
        const int nblk = w.nh * w.nbl;
        if (nblk == 0) continue;
        if (!warp_wait_all(c, p.limit_ns, phase_f(&c->rfull, lu), q_of(g, true))) { ok = false; break; }
        tc_fence_after();
        if (elect_one()) scores(g);
        __syncwarp();
        if (!warp_wait_all(c, p.limit_ns, o_of(g, true))) { ok = false; break; }
        tc_fence_after();
        if (elect_one()) grads(g, nblk == 1);
        __syncwarp();
        for (int n = 0; n < nblk; ++n, ++g) {
          const bool more = n + 1 < nblk;
          // dV += P^T dO (the unit's first overwrites), then the next block's S^T
          if (!warp_wait_all(c, p.limit_ns, phase_f(&c->pready_l, g), phase_c(&c->pready_r, g), phase_f(&c->bofull, g),
                             q_of(g + 1, more), phase_c(&c->accempty, lu ^ 1u, n == 0))) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            // P^T: 16 columns at the start of each epilogue warp's 32
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma2_bf16_ts(tmem + KT_DV, tmem + 32 * (k >> 1) + 8 * (k & 1), dplus(dBO, k * 2048), IDESC_KM,
                           (n || k) ? 1u : 0u);
            commit2_mc(&c->boempty, 3);
            if (more) scores(g + 1);
          }
          __syncwarp();
          // dK += dS^T Q, then the next block's dP^T
          if (!warp_wait_all(c, p.limit_ns, phase_f(&c->dsready_l, g), phase_c(&c->dsready_r, g), phase_f(&c->bqfull, g),
                             o_of(g + 1, more))) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma2_bf16_ts(tmem + KT_DK, tmem + KT_DP + 32 * (k >> 1) + 8 * (k & 1), dplus(dBQ, k * 2048), IDESC_KM,
                           (n || k) ? 1u : 0u);
            commit2_mc(&c->bqempty, 3);
            if (more) grads(g + 1, n + 2 == nblk);
            else commit2_mc(&c->accfull, 3);
          }
          __syncwarp();
        }
        if (!ok) break;
        ++lu;
      }
      if (elect_one()) {
        if (!ok) fail_f(c, p.status);
        commit2_mc(&c->mdone, 1);
      }
      wait_inl<false>(&c->mdone, 0, nullptr, 200000000ull);
    }
    __syncwarp();
  } else if (warp == KV_LD_WARP) {
    // -lse * log2(e) (two stages) and -D of each block's 128 queries into shared memory;
    // loads issued a block ahead
    float* ld = reinterpret_cast<float*>(base + KV_LD);
    uint32_t g = 0;
    bool ok = true;
    typename S::Raw raw = S::kv_raw(p, pid);
    for (int rnd = 0, u = pid; u < p.n_units && ok; u = S::next_unit(++rnd, pid, npairs)) {
      KvUnit w;
      S::kv_unit(p, u, raw, w);
      raw = S::kv_raw(p, S::next_unit(rnd + 1, pid, npairs));
      const int nblk = w.nh * w.nbl;
      for (int n = 0, z = w.z0, b = w.b0; n < nblk; ++n, ++g, kv_next(w, z, b)) {
        float lv[4], dv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int q = p.c0 + 128 * b + lane + 32 * i;
          const bool v = q < p.c1;
          const int64_t o = (int64_t)z * p.T + q;
          lv[i] = v ? p.lse[o] * L2E : 0.f;
          dv[i] = v ? __ldcg(p.D + o) : 0.f;   // past the L1, where k_attn_q may have left an older value
        }
        const uint32_t s = g & 1u;
        if (!warp_wait_c(&c->lempty[s], (g >> 1) ^ 1u, c, p.limit_ns)) { ok = false; break; }
#pragma unroll
        for (int i = 0; i < 4; ++i) ld[128 * s + lane + 32 * i] = -lv[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->lfull[s]);
        if (!warp_wait_c(&c->dempty, g ^ 1u, c, p.limit_ns)) { ok = false; break; }
#pragma unroll
        for (int i = 0; i < 4; ++i) ld[256 + lane + 32 * i] = -dv[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->dfull);
      }
    }
    if (!ok) fail_f(c, p.status);
  } else {
    const int q = warp & 3, cg = (warp - 2) >> 2;   // lane quadrant, 32-column group
    const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(32 * cg);
    const float* ld = reinterpret_cast<const float*>(base + KV_LD);
    uint32_t g = 0, lu = 0;
    bool ok = true;
    // the next unit's entry and key ranges are loaded while this one's outputs leave
    auto first_key = [&](const KvUnit& x) { return 256 * x.kp + 128 * (int)rank + 32 * q; };   // this warp's
    KvUnit w;
    int lo, hi;   // queries that see this thread's key
    S::kv_unit(p, pid, S::kv_raw(p, pid), w);
    S::key_range(p, first_key(w) + lane, lo, hi);
    for (int rnd = 0, u = pid; u < p.n_units && ok; u = S::next_unit(++rnd, pid, npairs)) {
      const int nblk = w.nh * w.nbl;
      const int kw = first_key(w), key = kw + lane;
      const int un = S::next_unit(rnd + 1, pid, npairs);
      const KvRows rows{lo, hi, kw + lane / 4};
      if constexpr (!S::kAddOut) {
        if (nblk == 0) {   // no query sees these keys
          S::store_zero(p, w.plane, key, 32 * cg);
          S::kv_unit(p, un, S::kv_raw(p, un), w);
          S::key_range(p, first_key(w) + lane, lo, hi);
          continue;
        }
      }
      typename S::Scale sc = S::scale_of(p, w.z0);
      for (int n = 0, z = w.z0, b = w.b0; n < nblk; ++n, ++g) {
        const int qg = p.c0 + 128 * b + 32 * cg;   // first of this thread's 32 queries
        int lo0, lo1, hi0, hi1;   // over the warp's keys
        S::key_warp(p, kw, lo, hi, lo0, lo1, hi0, hi1);
        const bool none = qg + 31 < lo0 || qg >= hi1, all = qg >= lo1 && qg + 31 < hi0;
        const uint32_t s = g & 1u;
        uint32_t rs[2][16];                        // scores, then probabilities
        const int q0 = qg + 2 * (lane & 3);        // the first of the thread's queries
        const float2* ldq = reinterpret_cast<const float2*>(ld) + 16 * cg + (lane & 3);
        // what is there long before comes before the wait that is not
        if (!warp_wait_f(&c->lfull[s], g >> 1, c, p.limit_ns)) { ok = false; break; }
        float2 nl[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) nl[i] = ldq[64 * s + 4 * i];
        if (!warp_wait_c(&c->sfull, g, c, p.limit_ns)) { ok = false; break; }
        tc_fence_after();
        __syncwarp();
        {
          tmem_ld_frag(trow, rs[0]);
          tmem_ld_frag(trow + (16u << 16), rs[1]);
          tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < 2; ++h) {            // 16 keys at a time, over this warp's own scores
            uint32_t pk[8] = {};
            if (all) kv_probs<S, false>(rs[h], h, nl, sc, q0, rows, pk);
            else if (!none) kv_probs<S, true>(rs[h], h, nl, sc, q0, rows, pk);
            __syncwarp();
            tmem_st_frag(trow + ((uint32_t)(16 * h) << 16), pk);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          arrive_leader(rank, &c->pready_l, &c->pready_r);
          mbar_arrive(&c->lempty[s]);
        }
        if (!warp_wait_f(&c->dfull, g, c, p.limit_ns)) { ok = false; break; }
        float2 nD[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) nD[i] = ldq[128 + 4 * i];
        if (!warp_wait_c(&c->dpfull, g, c, p.limit_ns)) { ok = false; break; }
        tc_fence_after();
        __syncwarp();
        {
          uint32_t rd[2][16];
          tmem_ld_frag(trow + KT_DP, rd[0]);
          tmem_ld_frag(trow + KT_DP + (16u << 16), rd[1]);
          tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[8] = {};
            if (all) kv_grads<S, false>(rs[h], rd[h], h, nD, q0, rows, pk);
            else if (!none) kv_grads<S, true>(rs[h], rd[h], h, nD, q0, rows, pk);
            __syncwarp();
            tmem_st_frag(trow + KT_DP + ((uint32_t)(16 * h) << 16), pk);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          arrive_leader(rank, &c->dsready_l, &c->dsready_r);
          mbar_arrive(&c->dempty);
        }
        if (kv_next(w, z, b) && n + 1 < nblk) sc = S::scale_of(p, z);
      }
      if (!ok) break;
      // the unit's dV and dK, 32 of hd, out of tensor memory and through this warp's staging
      // block: asynchronous copies of whole rows (row-per-thread stores of them took 9100 cycles
      // a unit, as long as three blocks)
      const typename S::Raw raw = S::kv_raw(p, un);
      if (!warp_wait_c(&c->accfull, lu, c, p.limit_ns)) { ok = false; break; }
      ++lu;
      tc_fence_after();
      const KvUnit done = w;
      S::kv_unit(p, un, raw, w);
      S::key_range(p, first_key(w) + lane, lo, hi);
      const uint32_t stg = sb + KV_STG + (uint32_t)(warp - 2) * 4096u;
      const bool leaves = S::kv_leaves(p, kw, 32 * cg);
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {   // t = 0: dV, t = 1: s dK
        __syncwarp();
        uint32_t ra[32];
        tmem_ld32(trow + (t ? KT_DK : KT_DV), ra);
        tmem_ld_wait();
        if (t == 1) {   // both accumulators are in registers: the next unit may overwrite them
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_remote(mapa(saddr(&c->accempty), 0));
        }
        if (!leaves) continue;
        if (lane == 0) bulk_wait_read();   // the block's previous contents have left
        __syncwarp();
        S::kv_stage(p, t, ra, stg, lane);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          S::kv_copy(maps, p, t, stg, 32 * cg, kw, done);
          bulk_commit();
        }
      }
      __syncwarp();
    }
    if (!ok) fail_f(c, p.status);
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  teardown_f(c, warp);
}

// ===================================================================== k_attn_q (dQ)

// k_attn_q's epilogue: 32 keys of this thread's query row.  P = 2^(s S - lse log2 e), dS =
// P (dP - D), packed to bf16 pairs.  MASK: some row of the warp does not see all 32 keys;
// the other blocks skip the per-element test.  SUM: adds P (dP - D) into `sum` instead.
template <class S, bool MASK, bool SUM>
__device__ __forceinline__ void q_block(const uint32_t (&rs)[32], const uint32_t (&rd)[32],
                                        const typename S::Scale& sc, float lz, float Dq, int kg, int qr, int lo, int hi,
                                        uint32_t (&dw)[16], float2& sum) {
  const float2 nD = make_float2(-Dq, -Dq), nlz = make_float2(-lz, -lz);
  const float fd = (float)(qr - kg);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float2 dc;
    const float2 x = S::template log2p2<MASK>(sc, make_float2(__uint_as_float(rs[2 * i]), __uint_as_float(rs[2 * i + 1])), nlz, fd,
                               (float)(-2 * i), (float)(-2 * i - 1), dc);
    float2 pp = exp2_pair(x.x, x.y);
    const bool o0 = MASK && (kg + 2 * i < lo || kg + 2 * i >= hi);
    const bool o1 = MASK && (kg + 2 * i + 1 < lo || kg + 2 * i + 1 >= hi);
    if (o0) pp.x = 0.f;
    if (o1) pp.y = 0.f;
    float2 sv = mul2(SUM ? pp : S::fold(pp, dc),
                     add2(make_float2(__uint_as_float(rd[2 * i]), __uint_as_float(rd[2 * i + 1])), nD));
    if (S::kClearMasked && o0) sv.x = 0.f;
    if (S::kClearMasked && o1) sv.y = 0.f;
    if (SUM) sum = add2(sum, sv);
    else dw[i] = pack_bf16(sv.x, sv.y);
  }
}

template <class S>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Q_THREADS, 1)
    k_attn_q(const __grid_constant__ typename S::QMaps maps, const typename S::Q p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  CtrlQ* c = reinterpret_cast<CtrlQ*>(base + Q_CTRL);
  const uint32_t sb = saddr(base);
  const int warp = uniform_warp(), lane = threadIdx.x % 32;
  const uint32_t rank = ctarank();
  prologue_q(c, warp);
  wait_for_primary();
  dependents_may_start();
  const uint32_t tmem = c->tmem_base;
  const int pid = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (warp == 0) {
    if (lane == 0) {
      // the unit's Q and dO, then K and V of each key block (this CTA's 64 keys)
      prefetch_map(maps[Q_MQ]);
      prefetch_map(maps[Q_MO]);
      prefetch_map(maps[Q_MKA]);
      prefetch_map(maps[Q_MVA]);
      uint32_t g = 0, gv = 0, lu = 0;   // key blocks (K; V) and units loaded so far
      bool ok = true;
      typename S::Raw raw = S::q_raw(p, pid);
      typename S::Large large = S::q_large(p, pid, raw);   // the next unit's, loaded once its entry is there
      for (int rnd = 0, u = pid; u < p.n_units && ok; u = S::next_unit(++rnd, pid, npairs)) {
        int z, qp, j0, nj;
        S::q_unit(p, u, raw, z, qp, j0, nj);
        const SumBlocks pre = S::q_sums(raw, large);
        const int un = S::next_unit(rnd + 1, pid, npairs);
        raw = S::q_raw(p, un);
        if (nj == 0) {
          large = S::q_large(p, un, raw);
          continue;
        }
        const uint32_t rs = lu & 1u;
        if (!wait_c(&c->rempty[rs], (lu >> 1) ^ 1u, c, p.limit_ns)) { ok = false; break; }
        const uint32_t fr = mapa(saddr(&c->rfull[rs]), 0);
        if (rank == 0) mbar_expect_tx(&c->rfull[rs], 4u * 32768u);
        const int qrow = p.c0 + 256 * qp + 128 * (int)rank;
#pragma unroll
        for (int hb = 0; hb < 2; ++hb) {
          tma_load_3d_pair(sb + Q_R + rs * 65536u + hb * 16384, maps[Q_MQ], fr, 64 * hb, qrow, z);
          tma_load_3d_pair(sb + Q_R + rs * 65536u + 32768 + hb * 16384, maps[Q_MO], fr, 64 * hb, qrow, z);
        }
        ++lu;
        for (int n = -pre.n; n < nj; ++n) {
          const int krow = 128 * (n < 0 ? pre.j + pre.n + n : j0 + n) + 64 * (int)rank;
          const uint32_t s = g & 1u, ph = (g >> 1) ^ 1u;
          if (!wait_c(&c->kempty[s], ph, c, p.limit_ns)) { ok = false; break; }
          const uint32_t fk = mapa(saddr(&c->kfull[s]), 0), fv = mapa(saddr(&c->vfull[s]), 0);
          if (rank == 0) mbar_expect_tx(&c->kfull[s], 2u * 16384u);
#pragma unroll
          for (int hb = 0; hb < 2; ++hb)
            tma_load_3d_pair(sb + Q_K + s * 16384u + hb * 8192, maps[Q_MKA], fk, 64 * hb, krow, z / p.group);
          ++g;
          if (!wait_c(&c->vempty[s], ph, c, p.limit_ns)) { ok = false; break; }
          if (rank == 0) mbar_expect_tx(&c->vfull[s], 2u * 16384u);
#pragma unroll
          for (int hb = 0; hb < 2; ++hb)
            tma_load_3d_pair(sb + Q_V + s * 16384u + hb * 8192, maps[Q_MVA], fv, 64 * hb, krow, z / p.group);
          ++gv;
          if (n == -pre.n) large = S::q_large(p, un, raw);
        }
      }
      if (!ok) {   // wait for the copies in flight
        fail_f(c, p.status);
        if (rank == 0) {
          for (uint32_t i = lu > 2 ? lu - 2 : 0; i < lu; ++i)
            wait_inl<false>(&c->rfull[i & 1u], (i >> 1) & 1u, nullptr, 200000000ull);
          for (uint32_t i = g > 2 ? g - 2 : 0; i < g; ++i)
            wait_inl<false>(&c->kfull[i & 1u], (i >> 1) & 1u, nullptr, 200000000ull);
          for (uint32_t i = gv > 2 ? gv - 2 : 0; i < gv; ++i)
            wait_inl<false>(&c->vfull[i & 1u], (i >> 1) & 1u, nullptr, 200000000ull);
        }
      }
    } else if (lane == 16) {
      // K of each key block, 128 keys x this CTA's half of hd (B of dQ += dS K)
      prefetch_map(maps[Q_MKB]);
      int tail = -1;
      if constexpr (S::kTail) tail = S::tail_block(p);
      uint32_t g = 0;
      bool ok = true;
      typename S::Raw raw = S::q_raw(p, pid);
      for (int rnd = 0, u = pid; u < p.n_units && ok; u = S::next_unit(++rnd, pid, npairs)) {
        int z, qp, j0, nj;
        S::q_unit(p, u, raw, z, qp, j0, nj);
        raw = S::q_raw(p, S::next_unit(rnd + 1, pid, npairs));
        for (int j = 0; j < nj; ++j) {
          const uint32_t s = g & 1u;
          if (!wait_c(&c->yempty[s], (g >> 1) ^ 1u, c, p.limit_ns)) { ok = false; break; }
          const uint32_t fy = mapa(saddr(&c->yfull[s]), 0);
          if (rank == 0) mbar_expect_tx(&c->yfull[s], 2u * 16384u);
          const CUtensorMap* mk = maps[Q_MKB];
          int row = 128 * (j0 + j);
          if constexpr (S::kTail)
            if (j0 + j == tail) {
              mk = maps.template at<Q_MKT>();
              row = 0;
            }
          tma_load_3d_pair(sb + Q_Y + s * 16384u, mk, fy, 64 * (int)rank, row, z / p.group);
          ++g;
        }
      }
      if (!ok) {
        fail_f(c, p.status);
        if (rank == 0)
          for (uint32_t i = g > 2 ? g - 2 : 0; i < g; ++i)
            wait_inl<false>(&c->yfull[i & 1u], (i >> 1) & 1u, nullptr, 200000000ull);
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {   // the whole warp, converged; one elected lane issues
      const uint64_t dR = sw128_desc(sb + Q_R, 16, 1024), dK = sw128_desc(sb + Q_K, 16, 1024),
                     dV = sw128_desc(sb + Q_V, 16, 1024), dY = sw128_desc(sb + Q_Y, 16384, 1024);
      const bool wide = S::wide(p);
      uint32_t g = 0, gy = 0, lu = 0;   // blocks, blocks with a dQ product, units
      bool ok = true;
      // S of block gg into its buffer: free, since the dQ product that read the dS in it was
      // issued before
      auto scores = [&](uint32_t gg, uint64_t q0) {   // by the elected lane
        const uint32_t s = gg & 1u;
        const uint64_t k0 = dplus(dK, s * 16384u);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (k == 4 && !wide) break;
          mma2_bf16(tmem + 128 * s, dplus(q0, (k >> 2) * 16384 + (k & 3) * 32),
                    dplus(k0, (k >> 2) * 8192 + (k & 3) * 32), IDESC_KK, k ? 1u : 0u);
        }
        commit2_mc(&c->kempty[s], 3);
      };
      // dP of block gg, once the previous block's has been read; completes the block's S too
      auto grads = [&](uint32_t gg, uint64_t o0) {
        const uint32_t s = gg & 1u;
        const uint64_t v0 = dplus(dV, s * 16384u);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (k == 4 && !wide) break;
          mma2_bf16(tmem + QT_DP, dplus(o0, (k >> 2) * 16384 + (k & 3) * 32),
                    dplus(v0, (k >> 2) * 8192 + (k & 3) * 32), IDESC_KK, k ? 1u : 0u);
        }
        commit2_mc(&c->vempty[s], 3);
        commit2_mc(&c->tfull, 3);
      };
      auto k_of = [&](uint32_t gg, bool need) { return phase_f(&c->kfull[gg & 1u], gg >> 1, need); };
      auto v_of = [&](uint32_t gg) { return phase_f(&c->vfull[gg & 1u], gg >> 1); };
      typename S::Raw raw = S::q_raw(p, pid);
      typename S::Large large = S::q_large(p, pid, raw);
      for (int rnd = 0, u = pid; u < p.n_units && ok; u = S::next_unit(++rnd, pid, npairs)) {
        int z, qp, j0, nj;
        S::q_unit(p, u, raw, z, qp, j0, nj);
        const int first = -S::q_sums(raw, large).n, un = S::next_unit(rnd + 1, pid, npairs);
        raw = S::q_raw(p, un);
        if (nj == 0) {
          large = S::q_large(p, un, raw);
          continue;
        }
        const uint32_t rs = lu & 1u;
        const uint64_t q0 = dplus(dR, rs * 65536u), o0 = dplus(q0, 32768);
        // the tensor pipe always has the next block's S and dP to form while the epilogue
        // works on a block: S two blocks ahead, dP one
        if (!warp_wait_all(c, p.limit_ns, phase_f(&c->rfull[rs], lu >> 1), k_of(g, true), v_of(g),
                           phase_f(&c->tempty_l, g ^ 1u), phase_c(&c->tempty_r, g ^ 1u), k_of(g + 1, nj - first > 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          scores(g, q0);
          grads(g, o0);
          if (nj - first > 1) scores(g + 1, q0);
        }
        __syncwarp();
        for (int n = first; n < nj; ++n, ++g) {
          const uint32_t s = g & 1u;
          if (n + 1 < nj) {
            if (!warp_wait_all(c, p.limit_ns, phase_f(&c->tempty_l, g), phase_c(&c->tempty_r, g), v_of(g + 1))) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          if (elect_one()) {
            if (n + 1 < nj) grads(g + 1, o0);
            if (n == max(nj - 2, first)) commit2_mc(&c->rempty[rs], 3);   // the unit's last S, dP are issued
          }
          __syncwarp();
          const bool more = n + 2 < nj;
          if (!warp_wait_all(c, p.limit_ns, phase_f(&c->oready_l[s], g >> 1), phase_c(&c->oready_r[s], g >> 1),
                             phase_f(&c->yfull[gy & 1u], gy >> 1, n >= 0), k_of(g + 2, more),
                             phase_c(&c->accempty, lu ^ 1u, n == 0))) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            if (n >= 0) {
              // dS: 16 columns at the start of each epilogue warp's 32
              const uint64_t y0 = dplus(dY, (gy & 1u) * 16384u);
#pragma unroll
              for (int k = 0; k < 8; ++k)
                mma2_bf16_ts(tmem + QT_DQ, tmem + 128 * s + 32 * (k >> 1) + 8 * (k & 1), dplus(y0, k * 2048), IDESC_KM,
                             (n || k) ? 1u : 0u);
              commit2_mc(&c->yempty[gy & 1u], 3);
              if (n == nj - 1) commit2_mc(&c->dqfull, 3);
            }
            if (more) scores(g + 2, q0);
          }
          __syncwarp();
          if (n == first) large = S::q_large(p, un, raw);
          gy += n >= 0;
        }
        if (!ok) break;
        ++lu;
      }
      if (elect_one()) {
        if (!ok) fail_f(c, p.status);
        commit2_mc(&c->mdone, 1);
      }
      wait_inl<false>(&c->mdone, 0, nullptr, 200000000ull);
    }
    __syncwarp();
  } else {
    const int q = warp & 3, cg = (warp - 2) >> 2;   // lane quadrant, 32-column group
    const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(32 * cg);
    uint32_t g = 0, lu = 0, summed = 0;   // blocks, units, units that summed first
    bool ok = true;
    // the next unit's entry is loaded during this one, its rows' values while this one's dQ leaves
    int z, qp, j0, nj, qw, lo, hi;   // qw: this warp's first query; keys this thread's query sees
    typename S::Raw entry;
    typename S::Large large;
    float lz, Dq;
    auto rows_of = [&](int u, typename S::Raw r) {
      S::q_unit(p, u, r, z, qp, j0, nj);
      entry = r;
      large = S::q_large(p, u, r);
      qw = p.c0 + 256 * qp + 128 * (int)rank + 32 * q;
      const int qr = qw + lane;
      const bool v = u < p.n_units && qr < p.c1;
      const int64_t ro = (int64_t)z * p.T + qr;
      lz = v ? p.lse[ro] : 0.f;
      Dq = v ? p.D[ro] : 0.f;
      S::query_range(p, qr, lo, hi);
    };
    uint32_t left = 0;   // units whose dQ has left its staging block (the unit's own Q)
    auto release = [&]() {
      if (left == lu) return;
      if (lane == 0) {
        bulk_wait_read();
        mbar_arrive(&c->rempty[left & 1u]);
      }
      left = lu;
    };
    rows_of(pid, S::q_raw(p, pid));
    for (int rnd = 0, u = pid; u < p.n_units && ok; u = S::next_unit(++rnd, pid, npairs)) {
      const int un = S::next_unit(rnd + 1, pid, npairs);
      const typename S::Raw raw = S::q_raw(p, un);
      const typename S::Scale sc = S::scale_of(p, z);
      const int qr = qw + lane;   // this thread's query
      const float lz2 = lz * L2E;
      int lo0, lo1, hi0, hi1;     // over the warp's queries
      S::query_warp(p, qw, lo, hi, lo0, lo1, hi0, hi1);
      if constexpr (!S::kAddOut) {
        if (nj == 0) {   // queries that see no key
          if (qr < p.c1) S::store_dq_zero(p, (int64_t)z * p.T + qr, 32 * cg);
          rows_of(un, raw);
          continue;
        }
      }
      const SumBlocks pre = S::q_sums(entry, large);
      float Dv = Dq;
      float2 sum = make_float2(0.f, 0.f);
      for (int n = -pre.n; n < nj; ++n, ++g) {
        if (!warp_wait_c(&c->tfull, g, c, p.limit_ns)) { ok = false; break; }
        tc_fence_after();
        uint32_t rs[32], rd[32], dw[16];   // dw: bf16 pairs of dS over this thread's 32 keys
        tmem_ld32(trow + QT_DP, rd);
        tmem_ld32(trow + 128 * (g & 1u), rs);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader(rank, &c->tempty_l, &c->tempty_r);   // dP is in registers: the next block's may be formed
        const bool sums = S::kSumFirst && n < 0;
        const int kg = 128 * (sums ? pre.j + pre.n + n : j0 + n) + 32 * cg;    // first key
        const bool none = kg + 31 < lo0 || kg >= hi1, all = kg >= lo1 && kg + 31 < hi0;
        if constexpr (S::kSumFirst) {
          if (sums && all) q_block<S, false, true>(rs, rd, sc, lz2, Dv, kg, qr, lo, hi, dw, sum);
          else if (sums && !none) q_block<S, true, true>(rs, rd, sc, lz2, Dv, kg, qr, lo, hi, dw, sum);
        }
        if (!sums) {
          if (none) {
#pragma unroll
            for (int i = 0; i < 16; ++i) dw[i] = 0u;
          } else if (all) {
            q_block<S, false, false>(rs, rd, sc, lz2, Dv, kg, qr, lo, hi, dw, sum);
          } else {
            q_block<S, true, false>(rs, rd, sc, lz2, Dv, kg, qr, lo, hi, dw, sum);
          }
          __syncwarp();
          tmem_st16(trow + 128 * (g & 1u), dw);       // over this warp's own scores
          tmem_st_wait();
        }
        if constexpr (S::kSumFirst) {
          if (n == -1) {   // the rows' sums over the four column groups, by way of the scores' place
            __syncwarp();
            tmem_st1(trow + 128 * (g & 1u), __float_as_uint(sum.x + sum.y));
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->sums[q]);
            if (!warp_wait_f(&c->sums[q], summed++, c, p.limit_ns)) { ok = false; break; }
            tc_fence_after();
            __syncwarp();
            uint32_t part[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) tmem_ld1(trow + 128 * (g & 1u) + 32 * (k - cg), part[k]);
            tmem_ld_wait();
            if (lo >= 128 * pre.j && hi <= 128 * (pre.j + pre.n)) {   // all of the row's keys were in the sum
#pragma unroll
              for (int k = 0; k < 4; ++k) Dv += __uint_as_float(part[k]);
            }
            if (cg == 0 && qr < p.c1) p.D[(int64_t)z * p.T + qr] = Dv;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader(rank, &c->oready_l[g & 1u], &c->oready_r[g & 1u]);
        release();
      }
      if (!ok) break;
      // dQ of the unit's queries, s * accumulator in bf16: this warp's 32 rows and 32 of hd leave
      // through the space of the unit's Q, which no product reads any more
      const int zu = z, qu = qw;
      const uint32_t stg = sb + Q_R + (lu & 1u) * 65536u + (uint32_t)(warp - 2) * 2048u;
      rows_of(un, raw);
      if (!warp_wait_c(&c->dqfull, lu, c, p.limit_ns)) { ok = false; break; }
      ++lu;
      tc_fence_after();
      __syncwarp();
      uint32_t ra[32];
      tmem_ld32(trow + QT_DQ, ra);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_remote(mapa(saddr(&c->accempty), 0));
      if (qu < p.c1 && 32 * cg < S::width(p)) {
        stage_bf16(ra, p.scale, stg, lane);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(maps[Q_MOUT], stg, 32 * cg, qu, zu);
          bulk_commit();
        }
      }
      __syncwarp();
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
    if (!ok) fail_f(c, p.status);
  }
  teardown_f(c, warp);
}

}  // namespace fa
}  // namespace tc
}  // namespace sbp
