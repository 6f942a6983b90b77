// Attention over packed documents: the preparing kernel, the score policy of the backward
// kernels (sbp_attn_fused.cuh), and the entry points.  The forward kernel is in
// sbp_attn_fwd.cu, the definition of what a query sees in sbp_attn_packed.cuh.
#include <algorithm>
#include <cmath>

#include "sbp_attn_fused.cuh"
#include "sbp_attn_packed.cuh"

namespace sbp {
namespace tc {
namespace pk {

struct KvParams {
  int H, Hkv, T, c0, c1, hd, group, n_units;
  float scale;
  Scale sc;
  const float *slopes, *lse, *D;
  const int32_t *qlo, *qhi;
  const PackedKvUnit* units;
  const int32_t* tail;
  __nv_bfloat16 *dK, *dV;
  // parts > 1: the query heads of a group are shared out to `parts` units of `per_part` heads,
  // which leave fp32 sums in part_k, part_v [parts, Hkv, T, hd]
  int parts, per_part;
  float *part_k, *part_v;
  int32_t* status;
  uint64_t limit_ns;
};
struct QParams {
  int H, T, c0, c1, hd, group, n_units;
  float scale;
  Scale sc;
  const float *slopes, *lse;
  float* D;
  const int32_t *lo, *hi;
  const PackedQUnit* units;
  const uint32_t* large;   // [H, n_units / H]
  const int32_t* tail;
  __nv_bfloat16* dQ;
  int32_t* status;
  uint64_t limit_ns;
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

constexpr int D_ROWS = 64;   // rows of D a block of the preparing kernel: one byte of `large`

// Score policy (see CausalScores): documents, prefixes, cap and distance bias; the units
// and intervals come from the preparing kernel, and every output element is written once,
// in bf16 (dK and dV of a key sum over the group's heads in tensor memory).
template <bool CAP, bool BIAS>
struct PackedScores {
  using Kv = KvParams;
  using Q = QParams;
  using KvMaps = fa::MapArray<fa::KV_MAPS + 2>;
  using QMaps = fa::MapArray<fa::Q_MAPS + 1>;   // + the last block's K
  // a masked pair's score may be infinite or NaN (another document's values)
  static constexpr bool kClearMasked = true;
  static constexpr bool kAddOut = false;
  using Scale = ScaleZ;

  static __device__ __forceinline__ int next_unit(int t, int pid, int npairs) { return pk::next_unit(t, pid, npairs); }
  using Raw = int4;   // a unit's list entry: {qp, ja0, jb0 or jb1, sums} or {kp, b0, nb}
  static __device__ __forceinline__ Raw kv_raw(const Kv& p, int u) {
    return u < p.n_units ? *reinterpret_cast<const int4*>(p.units + u / (p.parts * p.Hkv)) : make_int4(0, 0, 0, 0);
  }
  static __device__ __forceinline__ Raw q_raw(const Q& p, int u) {
    if (u >= p.n_units) return make_int4(0, 0, 0, 0);
    const int4* s = reinterpret_cast<const int4*>(p.units + u / p.H);
    const int4 b = s[1];
    int4 a = s[0];
    a.z = max(a.z, b.x);
    a.w = b.y;
    return a;
  }
  static __device__ __forceinline__ void kv_unit(const Kv& p, int u, Raw v, fa::KvUnit& w) {
    const int planes = p.parts * p.Hkv, i = u / planes;
    w.plane = u - i * planes;
    const int part = w.plane / p.Hkv, h0 = part * p.per_part;
    w.zk = w.plane - part * p.Hkv;
    w.kp = v.x;
    w.b0 = v.y;
    w.nbl = v.z;
    w.z0 = w.zk * p.group + h0;
    w.nh = min(p.per_part, p.group - h0);
  }
  static __device__ __forceinline__ void key_range(const Kv& p, int key, int& lo, int& hi) {
    lo = key < p.T ? p.qlo[key] : p.T;
    hi = key < p.T ? p.qhi[key] : p.T;
  }
  static __device__ __forceinline__ void ends(int lo, int hi, int& lo0, int& lo1, int& hi0, int& hi1) {
    lo0 = __shfl_sync(0xffffffffu, lo, 0);
    lo1 = __shfl_sync(0xffffffffu, lo, 31);
    hi0 = __shfl_sync(0xffffffffu, hi, 0);
    hi1 = __shfl_sync(0xffffffffu, hi, 31);
  }
  static __device__ __forceinline__ void key_warp(const Kv&, int, int lo, int hi, int& lo0, int& lo1, int& hi0,
                                                  int& hi1) {
    ends(lo, hi, lo0, lo1, hi0, hi1);
  }
  static __device__ __forceinline__ void q_unit(const Q& p, int u, Raw v, int& z, int& qp, int& j0, int& nj) {
    z = u % p.H;
    qp = v.x;
    j0 = v.y;
    nj = v.z - v.y;
  }
  static __device__ __forceinline__ void query_range(const Q& p, int q, int& lo, int& hi) {
    lo = q < p.T ? p.lo[q] : p.T;
    hi = q < p.T ? p.hi[q] : p.T;
  }
  static __device__ __forceinline__ void query_warp(const Q&, int, int lo, int hi, int& lo0, int& lo1, int& hi0,
                                                    int& hi1) {
    ends(lo, hi, lo0, lo1, hi0, hi1);
  }
  static constexpr bool kTail = true;
  template <class P>
  static __device__ __forceinline__ int tail_block(const P& p) { return *p.tail; }
  template <class P>
  static __device__ __forceinline__ Scale scale_of(const P& p, int z) {
    return scale_z(p.sc, BIAS ? p.slopes[z] : 0.f);
  }
  template <bool MASK>
  static __device__ __forceinline__ float2 log2p2(const Scale& sc, float2 s, float2 nlz, float d, float o0, float o1,
                                                  float2& dc) {
    float2 x;
    if (CAP) {
      const float2 r = cap_parts<MASK>(sc, s);
      dc = mul2(r, fma2(r, make_float2(-4.f, -4.f), make_float2(4.f, 4.f)));   // 1 - tanh^2 = 4 r (1 - r)
      x = fma2(r, make_float2(-2.f * sc.c2, -2.f * sc.c2), add2(nlz, make_float2(sc.c2, sc.c2)));
    } else {
      dc = make_float2(1.f, 1.f);
      x = fma2(s, make_float2(sc.sl2, sc.sl2), nlz);
    }
    if (BIAS) {
      x.x = fmaf(-sc.slope2, fabsf(d + o0), x.x);
      x.y = fmaf(-sc.slope2, fabsf(d + o1), x.y);
    }
    return x;
  }
  static __device__ __forceinline__ float2 fold(float2 p, float2 dc) { return CAP ? mul2(p, dc) : p; }

  // How 32 x 32 blocks of dV (t = 0) and dK (t = 1) leave (see CausalScores): bf16, or the parts'
  // fp32 sums.
  static __device__ __forceinline__ bool kv_leaves(const Kv& p, int kw, int c) { return kw < p.T && c < p.hd; }
  static __device__ __forceinline__ void kv_stage(const Kv& p, int t, const uint32_t (&ra)[32], uint32_t stg, int lane) {
    if (p.parts == 1) fa::stage_bf16(ra, t ? p.scale : 1.f, stg, lane);
    else fa::stage_f32(ra, t ? p.scale : 1.f, stg, lane);
  }
  static __device__ __forceinline__ void kv_copy(const KvMaps& maps, const Kv&, int t, uint32_t stg, int c, int kw,
                                                 const fa::KvUnit& w) {
    tma_store_3d(maps[t ? fa::KV_MOUTK : fa::KV_MOUTV], stg, c, kw, w.plane);
  }
  // Keys that no query sees: 32 columns of 0.
  static __device__ __forceinline__ void store_zero(const Kv& p, int plane, int key, int c) {
    if (key >= p.T) return;
    const int64_t row = ((int64_t)plane * p.T + key) * p.hd + c;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c + 8 * k < p.hd) {
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
        if (p.parts == 1) {
          *reinterpret_cast<uint4*>(p.dV + row + 8 * k) = z;
          *reinterpret_cast<uint4*>(p.dK + row + 8 * k) = z;
        } else {
          for (float* o : {p.part_v + row + 8 * k, p.part_k + row + 8 * k}) {
            *reinterpret_cast<uint4*>(o) = z;
            *reinterpret_cast<uint4*>(o + 4) = z;
          }
        }
      }
  }
  // 32 columns of dQ of a query that sees no key (row ro of [H, T])
  static __device__ __forceinline__ void store_dq_zero(const Q& p, int64_t ro, int c) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c + 8 * k < p.hd) *reinterpret_cast<uint4*>(p.dQ + ro * p.hd + c + 8 * k) = make_uint4(0u, 0u, 0u, 0u);
  }
  // D as dO . O is off by O's rounding to bf16, up to 2^-9 |dO| |O|, which dS = P (dP - D)
  // does not outgrow where a few keys hold nearly all of a row: at documents of 16 tokens and scores
  // of +-30, dQ and dK were off by 0.9%, 0.25% with D = sum P dP.  So units walk some of their
  // blocks once more for the sum of P (dP - D), and rows whose keys all lie in those correct D by
  // it, for themselves and for k_attn_kv.  Units of up to kSumBlocks blocks walk all of them;
  // longer ones those around their own rows, from the first document that lies in the unit or in the
  // block before it to one block behind the unit: what a document of up to 128 tokens sees is
  // within them wherever it stands.  Of the rows with more keys those need it whose O is large
  // against V (over half of it in norm): few keys hold the row, or V has a part in common that
  // dP - D does not see.  A unit with such a row walks all of its blocks first; the rest of the rows
  // add less than a tenth to the error that the two roundings to bf16 leave (0.24% in norm).
  // All units twice would be two products in seven: 16384 tokens forward and backward 7640 us, 6220
  // with this rule (normal inputs: no unit but the first).  4099 tokens with scores of +-10, a cap
  // and a bias: 429 us, 359 where long units look at their short documents alone, whose error is
  // then 0.38%; values with a mean of four times their deviation: 0.9% without.
  static constexpr bool kSumFirst = true;
  using Large = uint32_t;   // loaded once the unit's entry is there, looked at when the unit begins
  static __device__ __forceinline__ Large q_large(const Q& p, int u, Raw v) {
    static_assert(D_ROWS == 64, "four bytes a unit");
    return u < p.n_units ? p.large[(int64_t)(u % p.H) * (p.n_units / p.H) + v.x] : 0u;
  }
  static __device__ __forceinline__ fa::SumBlocks q_sums(Raw v, Large large) {
    return fa::SumBlocks{large ? v.y : v.w >> 3, large ? v.z - v.y : v.w & 7};
  }
  template <class P>
  static __device__ __forceinline__ bool wide(const P& p) { return p.hd > 64; }
  static __device__ __forceinline__ int width(const Q& p) { return p.hd; }
};

// ------------------------------------------------------------------- preparing kernel

constexpr int PREP_THREADS = 256;
// Units are put in order of their length up to this many (ranking them is quadratic);
// above, they keep the order of their rows.
constexpr int RANK_MAX = 8192;

struct PrepP {
  const int32_t *cu, *prefix;   // nullable
  int32_t n_seq;
  int T, n_units;
  int32_t *lo, *hi, *qlo, *qhi;
  PackedQUnit *qraw, *qunits;
  PackedKvUnit *kvraw, *kvunits;   // nullptr in the forward
  int32_t* tail;
  int token_blocks, tail_blocks, hd;
  // copies of the last block's rows (a block a head): operand i has heads[i] heads
  const __nv_bfloat16* tsrc[3];
  __nv_bfloat16* tdst[3];
  int heads[3];
  // D = dO . O of the backward, and which rows have an O that is large against V
  const __nv_bfloat16 *O, *dO, *V;
  int group;
  float* D;
  uint8_t* large;
  int32_t* status;
};

// End of the documents, within [0, T].
__device__ __forceinline__ int doc_end(const PrepP& p) { return p.cu ? min(max(p.cu[p.n_seq], 0), p.T) : p.T; }

// Document of token t < doc_end: its rows [s, e) and its prefix length.
__device__ __forceinline__ void doc_of(const PrepP& p, int t, int& s, int& e, int& pre) {
  int d = 0;
  if (p.cu) {
    int a = 0, b = p.n_seq - 1;   // last d with cu[d] <= t (empty documents are passed over)
    while (a < b) {
      const int mid = a + (b - a + 1) / 2;
      if (p.cu[mid] <= t) a = mid; else b = mid - 1;
    }
    d = a;
    s = min(max(p.cu[d], 0), p.T);
    e = min(max(p.cu[d + 1], s), p.T);
  } else {
    s = 0;
    e = p.T;
  }
  pre = p.prefix ? min(max(p.prefix[d], 0), e - s) : 0;
}
__device__ __forceinline__ int upper_of(int t, int s, int pre) { return max(t + 1, s + pre); }
__device__ __forceinline__ int qlower_of(int t, int s, int pre) { return t < s + pre ? s : t; }

// Block 0: checks the documents and lists the units.  Then token_blocks blocks: the four
// interval ends of each token; tail_blocks blocks: the last block's copies; the others: D.
__global__ void __launch_bounds__(PREP_THREADS) k_packed_prep(const PrepP p) {
  const int tid = threadIdx.x;
  dependents_may_start();
  if (blockIdx.x == 0) {
    __shared__ int bad;
    if (tid == 0) bad = 0;
    __syncthreads();
    if (p.cu) {
      bool b = tid == 0 && (p.cu[0] != 0 || p.cu[p.n_seq] > p.T);
      for (int i = tid; i < p.n_seq; i += PREP_THREADS)
        b = b || p.cu[i + 1] < p.cu[i] || (p.prefix && p.prefix[i] < 0);
      if (b) bad = 1;
    } else if (p.prefix && tid == 0 && p.prefix[0] < 0) {
      bad = 1;
    }
    __syncthreads();
    const int n_tok = doc_end(p);
    if (tid == 0) *p.tail = n_tok < p.T && n_tok % 128 ? n_tok / 128 : -1;
    if (tid == 0) *p.status = bad ? SBP_ERR_SEQLENS : SBP_OK;
    const int nb = (p.T + 127) / 128;
    for (int i = tid; i < p.n_units; i += PREP_THREADS) {
      PackedQUnit w;
      w.qp = i;
      int ja[2], jb[2];
      for (int h = 0; h < 2; ++h) {
        const int q0 = 256 * i + 128 * h, q1 = min(q0 + 127, n_tok - 1);
        if (q0 >= n_tok) {
          ja[h] = jb[h] = h ? jb[0] : 0;
          continue;
        }
        int s, e, pre;
        doc_of(p, q0, s, e, pre);
        ja[h] = s / 128;
        doc_of(p, q1, s, e, pre);
        jb[h] = min((upper_of(q1, s, pre) + 127) / 128, nb);
        jb[h] = max(jb[h], ja[h]);
      }
      w.ja0 = ja[0];
      w.jb0 = jb[0];
      // unbroken for any table: the second range starts within or right behind the first
      w.ja1 = min(max(ja[1], ja[0]), jb[0]);
      w.jb1 = max(jb[1], w.ja1);
      const int j0 = w.ja0, j1 = max(w.jb0, w.jb1);
      int s0 = j0, s1 = j1;
      if (j1 - j0 > kSumBlocks) {
        s0 = max(j0, 2 * i - 1);
        s1 = min(j1, 2 * i + 3);
        // the ends of the rows' intervals do not decrease: the first row that begins at s0 or
        // behind, of the unit's first document or of the one after it, is the one to ask
        int q = 256 * i, s, e, pre;
        doc_of(p, q, s, e, pre);
        if (s < 128 * s0) {
          q = e;
          if (q < min(256 * i + 256, n_tok)) doc_of(p, q, s, e, pre);
        }
        if (q >= min(256 * i + 256, n_tok) || upper_of(q, s, pre) > 128 * s1) s1 = s0;
        else s0 = max(s0, s / 128);   // no row that is asked for begins before its document
      }
      w.sums = 8 * s0 + max(s1 - s0, 0);
      p.qraw[i] = w;
      if (p.kvraw) {
        const int k0 = 256 * i, k1 = min(k0 + 255, n_tok - 1);
        PackedKvUnit v{i, 0, 0, 0};
        if (k0 < n_tok) {
          int s, e, pre;
          doc_of(p, k0, s, e, pre);
          v.b0 = qlower_of(k0, s, pre) / 128;
          doc_of(p, k1, s, e, pre);
          v.nb = max(min((e + 127) / 128, nb) - v.b0, 0);
        }
        p.kvraw[i] = v;
      }
    }
    __syncthreads();
    // longest units first: the last wave then holds the short ones
    for (int i = tid; i < p.n_units; i += PREP_THREADS) {
      const PackedQUnit w = p.qraw[i];
      const int len = (w.jb0 - w.ja0) + (w.jb1 - w.ja1);
      int r = i;
      if (p.n_units <= RANK_MAX) {
        r = 0;
        for (int k = 0; k < p.n_units; ++k) {
          const PackedQUnit o = p.qraw[k];
          const int lo = (o.jb0 - o.ja0) + (o.jb1 - o.ja1);
          r += lo > len || (lo == len && k < i);
        }
      }
      p.qunits[r] = w;
      if (p.kvraw) {
        const PackedKvUnit v = p.kvraw[i];
        r = i;
        if (p.n_units <= RANK_MAX) {
          r = 0;
          for (int k = 0; k < p.n_units; ++k) {
            const int lo = p.kvraw[k].nb;
            r += lo > v.nb || (lo == v.nb && k < i);
          }
        }
        p.kvunits[r] = v;
      }
    }
    return;
  }
  if ((int)blockIdx.x <= p.token_blocks) {
    const int t = ((int)blockIdx.x - 1) * PREP_THREADS + tid;
    if (t >= p.T) return;
    int lo = p.T, hi = p.T, qlo = p.T, qhi = p.T;
    if (t < doc_end(p)) {
      int s, e, pre;
      doc_of(p, t, s, e, pre);
      lo = s;
      hi = upper_of(t, s, pre);
      qlo = qlower_of(t, s, pre);
      qhi = e;
    }
    p.lo[t] = lo;
    p.hi[t] = hi;
    p.qlo[t] = qlo;
    p.qhi[t] = qhi;
    return;
  }
  if ((int)blockIdx.x <= p.token_blocks + p.tail_blocks) {
    const int n_tok = doc_end(p);
    if (n_tok >= p.T || n_tok % 128 == 0) return;
    int h = (int)blockIdx.x - 1 - p.token_blocks, i = 0;
    while (h >= p.heads[i]) h -= p.heads[i++];
    const int r0 = n_tok / 128 * 128, per = p.hd / 8;
    for (int k = tid; k < 128 * per; k += PREP_THREADS) {
      const int r = k / per, c = 8 * (k - r * per);
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (r0 + r < n_tok) v = *reinterpret_cast<const uint4*>(p.tsrc[i] + ((int64_t)h * p.T + r0 + r) * p.hd + c);
      *reinterpret_cast<uint4*>(p.tdst[i] + ((int64_t)h * 128 + r) * p.hd + c) = v;
    }
    return;
  }
  // D: 64 rows of a head, sixteen lanes a row, 16 bytes a lane and operand (hd <= 128)
  constexpr int K = D_ROWS / 16;
  static_assert(PREP_THREADS == 256 && 256 % D_ROWS == 0, "sixteen rows at a time, whole blocks a unit");
  const int blk = (int)blockIdx.x - 1 - p.token_blocks - p.tail_blocks, per_head = 256 / D_ROWS * p.n_units;
  const int h = blk / per_head, t0 = D_ROWS * (blk - h * per_head), c = 8 * (tid % 16);
  if (t0 >= p.T) {
    if (tid == 0) p.large[blk] = 0;
    return;
  }
  uint4 a[K] = {}, b[K] = {}, v = {};
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int t = t0 + tid / 16 + 16 * k;
    if (t < p.T && c < p.hd) {
      const int64_t r = ((int64_t)h * p.T + t) * p.hd + c;
      a[k] = *reinterpret_cast<const uint4*>(p.O + r);
      b[k] = *reinterpret_cast<const uint4*>(p.dO + r);
      if (k == 0) v = *reinterpret_cast<const uint4*>(p.V + ((int64_t)(h / p.group) * p.T + t) * p.hd + c);
    }
  }
  const int n_tok = doc_end(p);
  float acc[K] = {}, o2[K] = {}, v2 = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const uint32_t av[4] = {a[k].x, a[k].y, a[k].z, a[k].w}, bv[4] = {b[k].x, b[k].y, b[k].z, b[k].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack_bf16(av[i]), y = unpack_bf16(bv[i]);
      acc[k] = fmaf(x.x, y.x, acc[k]);
      acc[k] = fmaf(x.y, y.y, acc[k]);
      o2[k] = fmaf(x.x, x.x, fmaf(x.y, x.y, o2[k]));
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) {
      acc[k] += __shfl_xor_sync(0xffffffffu, acc[k], o);
      o2[k] += __shfl_xor_sync(0xffffffffu, o2[k], o);
    }
  }
  // |O|^2 > |V|^2 / 4, with the mean of the first sixteen rows for |V|^2; rows that their unit's
  // first walk covers anyway do not count
  __shared__ float norms[8];
  const uint32_t vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 z = unpack_bf16(vv[i]);
    if (t0 + tid / 16 < n_tok) v2 = fmaf(z.x, z.x, fmaf(z.y, z.y, v2));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) v2 += __shfl_xor_sync(0xffffffffu, v2, o);
  if (tid % 32 == 0) norms[tid / 32] = v2;
  __syncthreads();
  bool need = false;
  if (c == 0) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += norms[i];
    const float count = (float)(4 * min(16, n_tok - t0));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int t = t0 + tid / 16 + 16 * k;
      if (t < p.T) p.D[(int64_t)h * p.T + t] = acc[k];
      if (t < n_tok && o2[k] * count > sum) {
        int s, e, pre;
        doc_of(p, t, s, e, pre);
        const int unit = t / 256;
        need = need || s < 128 * (2 * unit - 1) || upper_of(t, s, pre) > 128 * (2 * unit + 3);
      }
    }
  }
  const int any = __syncthreads_or(need);
  if (tid == 0) p.large[blk] = any ? 1 : 0;
}

// dK and dV from the parts' fp32 sums, in the parts' order: eight elements a thread.
__global__ void __launch_bounds__(256) k_packed_join(const float* __restrict__ pk, const float* __restrict__ pv, int parts,
                                                     int64_t n, __nv_bfloat16* __restrict__ dK,
                                                     __nv_bfloat16* __restrict__ dV) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  const float* src = blockIdx.y ? pv : pk;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
  for (int k = 0; k < parts; ++k) {
    const float4* q = reinterpret_cast<const float4*>(src + (int64_t)k * n + i);
    const float4 x = q[0], y = q[1];
    a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
    b.x += y.x; b.y += y.y; b.z += y.z; b.w += y.w;
  }
  *reinterpret_cast<uint4*>((blockIdx.y ? dV : dK) + i) =
      make_uint4(pack2(a.x, a.y), pack2(a.z, a.w), pack2(b.x, b.y), pack2(b.z, b.w));
}

}  // namespace pk
}  // namespace tc

// ========================================================================== host side

namespace {

struct PackedLayout {
  size_t off_lo = 0, off_hi = 0, off_qlo = 0, off_qhi = 0, off_qraw = 0, off_qunits = 0, off_kvraw = 0,
         off_kvunits = 0, off_tail = 0, off_tq = 0, off_to = 0, off_tkv = 0, off_d = 0, off_large = 0, off_pk = 0, off_pv = 0, total = 0;
  int parts = 1, per_part = 1;   // of the backward's query-head groups (k_attn_kv); backward only, as what follows off_tkv
  Guards guards;   // checked build only
};

bool packed_shape(int64_t H, int64_t Hkv, int64_t T, int64_t hd) {
  return H >= 1 && Hkv >= 1 && Hkv <= H && H % Hkv == 0 && T >= 0 && hd >= 1;
}
// 16-byte rows; the kernels' tile is 128 wide; int32 row numbers
bool packed_supported(int64_t H, int64_t T, int64_t hd) {
  return hd % 8 == 0 && hd <= 128 && T <= (int64_t)1 << 30 && H <= (int64_t)1 << 20 &&
         H * (256 / tc::pk::D_ROWS * ((T + 255) / 256) + 3) + T / 256 < INT32_MAX / 2;   // blocks of the preparing kernel
}

// Query heads of a group that one k_attn_kv unit walks: all of them where that leaves two units
// or more for each SM pair (a key's dK and dV are then summed on chip), else as few as give four,
// the sums joined by k_packed_join.  The backward with and without (H / Hkv x tokens, hd 128):
// 16/1 x 128 36 and 55 us, 32/8 x 256 36 and 42, 32/8 x 1024 68 and 92; 20/4 x 4099 in
// two parts 281, in five 271; the other way from two units a pair on, 32/8 x 8192 in documents,
// 492 and 480 (the join reads and writes the sums again).
int kv_heads_per_part(int64_t H, int64_t Hkv, int64_t T) {
  const int64_t group = H / Hkv, units = std::max<int64_t>(1, (T + 255) / 256 * Hkv), pairs = std::max(1, num_sms() / 2);
  if (units >= 2 * pairs) return (int)group;
  const int64_t parts = std::min(group, (4 * pairs + units - 1) / units);
  return (int)((group + parts - 1) / parts);
}

// Regions of a call's workspace.  The forward has its own, without what only the backward writes.
// The backward with `per_part` query heads a unit of k_attn_kv: 0 for the choice above, the whole
// group for the smallest workspace, whose size does not fall as T grows.
enum class Pass { FORWARD, BACKWARD };
bool packed_layout(int64_t H, int64_t Hkv, int64_t T, int64_t hd, Pass pass, int per_part, PackedLayout* L) {
  if (!packed_shape(H, Hkv, T, hd) || !packed_supported(H, T, hd)) return false;
  PackedLayout l;
  const size_t t = (size_t)std::max<int64_t>(T, 1), n = (t + 255) / 256;
  const bool bwd = pass == Pass::BACKWARD;
  size_t o = 0;
  l.off_lo = take_region(o, t * sizeof(int32_t), l.guards);
  l.off_hi = take_region(o, t * sizeof(int32_t), l.guards);
  l.off_qlo = take_region(o, t * sizeof(int32_t), l.guards);
  l.off_qhi = take_region(o, t * sizeof(int32_t), l.guards);
  l.off_qraw = take_region(o, n * sizeof(PackedQUnit), l.guards);
  l.off_qunits = take_region(o, n * sizeof(PackedQUnit), l.guards);
  l.off_tail = take_region(o, sizeof(int32_t), l.guards);
  l.off_tkv = take_region(o, (size_t)Hkv * 128 * hd * 2, l.guards);
  if (bwd) {
    l.off_kvraw = take_region(o, n * sizeof(PackedKvUnit), l.guards);
    l.off_kvunits = take_region(o, n * sizeof(PackedKvUnit), l.guards);
    l.off_tq = take_region(o, (size_t)H * 128 * hd * 2, l.guards);
    l.off_to = take_region(o, (size_t)H * 128 * hd * 2, l.guards);
    l.off_d = take_region(o, (size_t)H * t * sizeof(float), l.guards);
    l.off_large = take_region(o, (size_t)H * n * (256 / tc::pk::D_ROWS), l.guards);
    l.per_part = per_part ? per_part : kv_heads_per_part(H, Hkv, T);
    l.parts = (int)((H / Hkv + l.per_part - 1) / l.per_part);
    if (l.parts > 1) {
      l.off_pk = take_region(o, (size_t)l.parts * Hkv * t * hd * sizeof(float), l.guards);
      l.off_pv = take_region(o, (size_t)l.parts * Hkv * t * hd * sizeof(float), l.guards);
    }
  }
  l.total = o;
  *L = l;
  return true;
}
// The backward's layout in `bytes`: the fastest one that fits, the sums of a group shared out to
// fewer parts where the workspace is smaller; else the smallest.
bool packed_layout_within(int64_t H, int64_t Hkv, int64_t T, int64_t hd, size_t bytes, PackedLayout* L) {
  if (!packed_layout(H, Hkv, T, hd, Pass::BACKWARD, 0, L)) return false;
  for (int parts = L->parts; L->total > bytes && parts > 1;) {
    const int64_t group = H / Hkv;
    --parts;
    packed_layout(H, Hkv, T, hd, Pass::BACKWARD, (int)((group + parts - 1) / parts), L);
  }
  return true;
}

// Shared checks of both directions; everything here runs before anything is enqueued.
int packed_check(const PackedArgs& a, std::initializer_list<const void*> tensors, Pass pass, void* ws, size_t ws_bytes,
                 PackedLayout* L) {
  if (!packed_shape(a.H, a.Hkv, a.T, a.hd) || !a.status) return SBP_ERR_INVALID_ARG;
  if (!(a.scale > 0.f) || std::isinf(a.scale) || !(a.softcap >= 0.f) || std::isinf(a.softcap))
    return SBP_ERR_INVALID_ARG;
  if ((a.cu && a.n_seq < 1) || (!a.cu && a.n_seq != 0)) return SBP_ERR_INVALID_ARG;
  if (a.softcap > 0.f && (a.softcap < 1e-6f || a.softcap > 256.f)) return SBP_ERR_UNSUPPORTED;
  const tc::pk::Scale sc = tc::pk::make_scale(a.scale, a.softcap);
  if (std::isinf(sc.sl2) || std::isinf(sc.k)) return SBP_ERR_UNSUPPORTED;
  if (pass == Pass::FORWARD ? !packed_layout(a.H, a.Hkv, a.T, a.hd, pass, 0, L)
                            : !packed_layout_within(a.H, a.Hkv, a.T, a.hd, ws_bytes, L))
    return SBP_ERR_UNSUPPORTED;
  for (const void* q : tensors) {
    if (!q && a.T > 0) return SBP_ERR_INVALID_ARG;
    if (!aligned16(q)) return SBP_ERR_ALIGNMENT;
  }
  for (const void* q : {(const void*)a.cu, (const void*)a.prefix, (const void*)a.slopes, (const void*)a.status})
    if (reinterpret_cast<uintptr_t>(q) & 3u) return SBP_ERR_ALIGNMENT;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < L->total) return SBP_ERR_WORKSPACE;
  return SBP_OK;
}

PackedWork packed_work(const PackedLayout& L, char* w) {
  PackedWork k;
  k.lo = reinterpret_cast<int32_t*>(w + L.off_lo);
  k.hi = reinterpret_cast<int32_t*>(w + L.off_hi);
  k.qlo = reinterpret_cast<int32_t*>(w + L.off_qlo);
  k.qhi = reinterpret_cast<int32_t*>(w + L.off_qhi);
  k.qunits = reinterpret_cast<PackedQUnit*>(w + L.off_qunits);
  k.kvunits = reinterpret_cast<PackedKvUnit*>(w + L.off_kvunits);
  k.tail = reinterpret_cast<int32_t*>(w + L.off_tail);
  k.tail_q = w + L.off_tq;
  k.tail_do = w + L.off_to;
  k.tail_kv = w + L.off_tkv;
  k.D = reinterpret_cast<float*>(w + L.off_d);
  k.large = reinterpret_cast<uint8_t*>(w + L.off_large);
  return k;
}

cudaError_t packed_prep(const PackedArgs& a, const PackedLayout& L, char* w, bool backward, cudaStream_t s) {
  tc::pk::PrepP p{};
  p.cu = a.cu; p.prefix = a.prefix; p.n_seq = a.n_seq;
  p.T = (int)a.T; p.n_units = (int)((a.T + 255) / 256);
  p.lo = reinterpret_cast<int32_t*>(w + L.off_lo);
  p.hi = reinterpret_cast<int32_t*>(w + L.off_hi);
  p.qlo = reinterpret_cast<int32_t*>(w + L.off_qlo);
  p.qhi = reinterpret_cast<int32_t*>(w + L.off_qhi);
  p.qraw = reinterpret_cast<PackedQUnit*>(w + L.off_qraw);
  p.qunits = reinterpret_cast<PackedQUnit*>(w + L.off_qunits);
  p.tail = reinterpret_cast<int32_t*>(w + L.off_tail);
  p.hd = (int)a.hd;
  p.tsrc[0] = static_cast<const __nv_bfloat16*>(backward ? a.K : a.V);
  p.tdst[0] = reinterpret_cast<__nv_bfloat16*>(w + L.off_tkv);
  p.heads[0] = (int)a.Hkv;
  p.token_blocks = (int)((a.T + tc::pk::PREP_THREADS - 1) / tc::pk::PREP_THREADS);
  p.status = a.status;
  if (backward) {
    p.tsrc[1] = static_cast<const __nv_bfloat16*>(a.Q);
    p.tdst[1] = reinterpret_cast<__nv_bfloat16*>(w + L.off_tq);
    p.tsrc[2] = static_cast<const __nv_bfloat16*>(a.dO);
    p.tdst[2] = reinterpret_cast<__nv_bfloat16*>(w + L.off_to);
    p.heads[1] = p.heads[2] = (int)a.H;
  }
  p.tail_blocks = p.heads[0] + p.heads[1] + p.heads[2];
  int64_t blocks = 1 + p.token_blocks + p.tail_blocks;
  if (backward) {
    p.kvraw = reinterpret_cast<PackedKvUnit*>(w + L.off_kvraw);
    p.kvunits = reinterpret_cast<PackedKvUnit*>(w + L.off_kvunits);
    p.O = static_cast<const __nv_bfloat16*>(a.O);
    p.dO = static_cast<const __nv_bfloat16*>(a.dO);
    p.V = static_cast<const __nv_bfloat16*>(a.V);
    p.group = (int)(a.H / a.Hkv);
    p.D = reinterpret_cast<float*>(w + L.off_d);
    p.large = reinterpret_cast<uint8_t*>(w + L.off_large);
    blocks += a.H * p.n_units * (256 / tc::pk::D_ROWS);
  }
  tc::pk::k_packed_prep<<<(unsigned)blocks, tc::pk::PREP_THREADS, 0, s>>>(p);
  return cudaGetLastError();
}

template <bool CAP, bool BIAS>
cudaError_t packed_backward_kernels(const PackedArgs& a, const PackedLayout& L, char* base, void* dQ, void* dK,
                                    void* dV, cudaStream_t s) {
  const PackedWork w = packed_work(L, base);
  using namespace tc::fa;
  using S = tc::pk::PackedScores<CAP, BIAS>;
  static int attr_state[64] = {};
  static std::mutex mu;
  if (!tc::once_per_device(attr_state, mu, [] {
        return cudaFuncSetAttribute(k_attn_kv<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_KV) ==
                   cudaSuccess &&
               cudaFuncSetAttribute(k_attn_q<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_Q) ==
                   cudaSuccess;
      }))
    return cudaErrorInvalidConfiguration;
  const int n = (int)((a.T + 255) / 256);
  MapArray<KV_MAPS + 2> mk;
  MapArray<Q_MAPS + 1> mq;
  const struct { CUtensorMap* m; const void* ptr; int64_t T, heads; uint32_t rows; } list[] = {
      {&mk.m[KV_MK], a.K, a.T, a.Hkv, 128},  {&mk.m[KV_MV], a.V, a.T, a.Hkv, 128},
      {&mk.m[KV_MQA], a.Q, a.T, a.H, 64},    {&mk.m[KV_MOA], a.dO, a.T, a.H, 64},
      {&mk.m[KV_MQB], a.Q, a.T, a.H, 128},   {&mk.m[KV_MOB], a.dO, a.T, a.H, 128},
      {&mk.m[KV_MQT], w.tail_q, 128, a.H, 128}, {&mk.m[KV_MOT], w.tail_do, 128, a.H, 128},
      {&mq.m[Q_MKA], a.K, a.T, a.Hkv, 64},   {&mq.m[Q_MVA], a.V, a.T, a.Hkv, 64},
      {&mq.m[Q_MKT], w.tail_kv, 128, a.Hkv, 128}};
  for (const auto& e : list)
    if (!tc::make_map_heads(e.m, e.ptr, e.T, e.heads, a.hd, e.rows)) return cudaErrorInvalidValue;
  // outputs: dK and dV in bf16, or the parts' sums
  for (int t = 0; t < 2; ++t) {
    CUtensorMap* m = &mk.m[t ? KV_MOUTV : KV_MOUTK];
    const bool ok = L.parts == 1 ? tc::make_map_out(m, t ? dV : dK, a.T, a.T, a.Hkv, a.hd, 2)
                                 : tc::make_map_out(m, base + (t ? L.off_pv : L.off_pk), a.T, a.T, L.parts * a.Hkv, a.hd, 4);
    if (!ok) return cudaErrorInvalidValue;
  }
  mq.m[Q_MQ] = mk.m[KV_MQB];
  mq.m[Q_MO] = mk.m[KV_MOB];
  mq.m[Q_MKB] = mk.m[KV_MK];
  if (!tc::make_map_out(&mq.m[Q_MOUT], dQ, a.T, a.T, a.H, a.hd, 2)) return cudaErrorInvalidValue;
  tc::pk::KvParams k;
  k.H = (int)a.H; k.Hkv = (int)a.Hkv; k.T = (int)a.T; k.c0 = 0; k.c1 = (int)a.T; k.hd = (int)a.hd;
  k.group = (int)(a.H / a.Hkv); k.n_units = n * k.Hkv * L.parts;
  k.parts = L.parts; k.per_part = L.per_part;
  k.part_k = reinterpret_cast<float*>(base + L.off_pk); k.part_v = reinterpret_cast<float*>(base + L.off_pv);
  k.scale = a.scale; k.sc = tc::pk::make_scale(a.scale, a.softcap);
  k.slopes = a.slopes; k.lse = a.lse; k.D = w.D; k.qlo = w.qlo; k.qhi = w.qhi; k.units = w.kvunits; k.tail = w.tail;
  k.dK = static_cast<__nv_bfloat16*>(dK); k.dV = static_cast<__nv_bfloat16*>(dV);
  k.status = a.status; k.limit_ns = tc::wait_limit_ns();
  const int kv_pairs = std::min(tc::max_pairs((const void*)k_attn_kv<S>, SMEM_KV, KV_THREADS), k.n_units);
  tc::pk::QParams q;
  q.H = k.H; q.T = k.T; q.c0 = 0; q.c1 = k.c1; q.hd = k.hd; q.group = k.group; q.n_units = n * k.H;
  q.scale = k.scale; q.sc = k.sc; q.slopes = k.slopes; q.lse = k.lse; q.D = w.D; q.lo = w.lo; q.hi = w.hi;
  q.units = w.qunits; q.large = reinterpret_cast<const uint32_t*>(w.large); q.tail = w.tail; q.dQ = static_cast<__nv_bfloat16*>(dQ); q.status = k.status; q.limit_ns = k.limit_ns;
  const int q_pairs = std::min(tc::max_pairs((const void*)k_attn_q<S>, SMEM_Q, Q_THREADS), q.n_units);
  // k_attn_q first: it corrects D; k_attn_kv starts as its pairs of SMs end, and waits for it
  cudaError_t e = tc::launch_early(k_attn_q<S>, 2 * q_pairs, Q_THREADS, SMEM_Q, s, mq, q);
  if (e != cudaSuccess) return e;
  e = tc::launch_early(k_attn_kv<S>, 2 * kv_pairs, KV_THREADS, SMEM_KV, s, mk, k);
  if (e != cudaSuccess) return e;
  if (L.parts > 1) {
    const int64_t m = a.Hkv * a.T * a.hd;
    tc::pk::k_packed_join<<<dim3((unsigned)((m / 8 + 255) / 256), 2), 256, 0, s>>>(k.part_k, k.part_v, L.parts, m, k.dK,
                                                                                  k.dV);
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace sbp

using namespace sbp;

extern "C" {

size_t sbp_attn_packed_workspace_bytes(int64_t H, int64_t Hkv, int64_t T, int64_t hd) {
  PackedLayout L;
  return packed_layout(H, Hkv, T, hd, Pass::BACKWARD, 0, &L) ? L.total : 0;
}

size_t sbp_attn_packed_workspace_bytes_lean(int64_t H, int64_t Hkv, int64_t T, int64_t hd) {
  PackedLayout L;
  return packed_layout_within(H, Hkv, T, hd, 0, &L) ? L.total : 0;
}

size_t sbp_attn_packed_forward_workspace_bytes(int64_t H, int64_t Hkv, int64_t T, int64_t hd) {
  PackedLayout L;
  return packed_layout(H, Hkv, T, hd, Pass::FORWARD, 0, &L) ? L.total : 0;
}

int sbp_attn_packed_forward(const void* Q, const void* K, const void* V, const int32_t* cu_seqlens,
                            const int32_t* prefix_lens, int32_t n_seq, const float* slopes, int64_t H, int64_t Hkv,
                            int64_t T, int64_t hd, float scale, float softcap, void* O, float* lse, void* workspace,
                            size_t ws_bytes, int32_t* dev_status, void* stream) {
  PackedArgs a{Q, K, V, nullptr, nullptr, nullptr, cu_seqlens, prefix_lens, slopes, H, Hkv, T, hd, n_seq, scale,
               softcap, dev_status};
  PackedLayout L;
  const int rc = packed_check(a, {Q, K, V, O, lse}, Pass::FORWARD, workspace, ws_bytes, &L);
  if (rc != SBP_OK) return rc;
  NvtxRange nv("sbp_attn_packed_forward");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(workspace);
  if (T == 0) {
    set_launch_count(0);
    return cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) == cudaSuccess ? SBP_OK : SBP_ERR_CUDA;
  }
  int launches = 2;
  int st = workspace_guards(w, L.guards, 0, dev_status, s, &launches);
  if (st != SBP_OK) return st;
  if (packed_prep(a, L, w, false, s) != cudaSuccess) return SBP_ERR_CUDA;
  if (packed_forward(a, packed_work(L, w), O, lse, s) != cudaSuccess) return SBP_ERR_CUDA;
  st = workspace_guards(w, L.guards, 1, dev_status, s, &launches);
  if (st == SBP_OK) set_launch_count(launches);
  return st;
}

int sbp_attn_packed_backward(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                             const float* lse, const int32_t* cu_seqlens, const int32_t* prefix_lens, int32_t n_seq,
                             const float* slopes, int64_t H, int64_t Hkv, int64_t T, int64_t hd, float scale,
                             float softcap, void* dQ, void* dK, void* dV, void* workspace, size_t ws_bytes,
                             int32_t* dev_status, void* stream) {
  PackedArgs a{Q, K, V, O, dO, lse, cu_seqlens, prefix_lens, slopes, H, Hkv, T, hd, n_seq, scale, softcap, dev_status};
  PackedLayout L;
  const int rc = packed_check(a, {Q, K, V, O, dO, lse, dQ, dK, dV}, Pass::BACKWARD, workspace, ws_bytes, &L);
  if (rc != SBP_OK) return rc;
  NvtxRange nv("sbp_attn_packed_backward");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(workspace);
  if (T == 0) {
    set_launch_count(0);
    return cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) == cudaSuccess ? SBP_OK : SBP_ERR_CUDA;
  }
  int launches = L.parts > 1 ? 4 : 3;
  int st = workspace_guards(w, L.guards, 0, dev_status, s, &launches);
  if (st != SBP_OK) return st;
  if (packed_prep(a, L, w, true, s) != cudaSuccess) return SBP_ERR_CUDA;
  cudaError_t e;
  if (softcap > 0.f)
    e = slopes ? packed_backward_kernels<true, true>(a, L, w, dQ, dK, dV, s)
               : packed_backward_kernels<true, false>(a, L, w, dQ, dK, dV, s);
  else
    e = slopes ? packed_backward_kernels<false, true>(a, L, w, dQ, dK, dV, s)
               : packed_backward_kernels<false, false>(a, L, w, dQ, dK, dV, s);
  if (e != cudaSuccess) return SBP_ERR_CUDA;
  st = workspace_guards(w, L.guards, 1, dev_status, s, &launches);
  if (st == SBP_OK) set_launch_count(launches);
  return st;
}

}  // extern "C"
