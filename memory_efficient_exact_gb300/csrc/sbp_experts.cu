// Tokens sorted by expert and back (sm_103a).
//
//   sort     the slots (t, j) of ids [T, k] in the order of their experts, slots of one expert in
//            the order of t * k + j: a counting sort, so that the order never depends on timing.
//   gather   Xs[rows[t, j]] = X[t]                     (gradient: combine without weights)
//   combine  Y[t] = residual[t] + sum_j w[t, j] Ys[rows[t, j]]
//            dYs[rows[t, j]] = w[t, j] dY[t],  dw[t, j] = dY[t] . Ys[rows[t, j]]
//
// All but the sort are bound by device memory.  They walk the tokens and not the sorted rows: a
// token's row is read once for all its k slots, and what one token receives is summed by one
// thread in the order of j, without atomics.
#include <algorithm>

#include "sbp_rows.cuh"
#include "sbp_tc_common.cuh"

namespace sbp {
namespace {

constexpr int64_t MAX_EXPERTS = 1024, MAX_D = 16384;
constexpr int SORT_WARPS = 16, SORT_PER_LANE = 4;
constexpr int SORT_THREADS = 32 * SORT_WARPS;
constexpr int SORT_SLOTS = SORT_THREADS * SORT_PER_LANE;   // slots of a block
// From so many blocks on their counts are summed once (k_expert_scan) and not by every block, whose
// work grows with their square and with the experts that a thread has.  With the launch / without, us:
//   blocks           32         48         64         96         128        256        512
//   2 experts     11.3  9.4  11.3 10.3  11.3 10.3  11.3 11.4  11.3 12.3  12.3 16.5  15.7  31
//   64 experts    13.4 11.9  14.4 12.3  14.4 12.4  14.4 14.4  14.8 15.0  16.5 20.5  23.7  42
//   256 experts   15.2 13.1  15.4 14.4  15.4 14.4  16.2 15.6  16.4 16.4  18.5 22.6  27.7  55
//   512 experts   16.4 14.4  16.4 15.2  16.4 16.4  17.3 16.5  17.4 18.5  20.5 27.3  30.8  68
//   1024 experts  18.5 18.5  18.5 20.1  19.0 20.6  19.5 22.6  19.5 25.4  22.6 41.2  36.9 117
bool sum_once(int64_t blocks, int64_t E) { return blocks >= std::min<int64_t>(128, 49152 / E); }

struct SortP {
  const int32_t* ids;
  int64_t n;          // slots
  int E, blocks;
  int32_t *rows, *slots, *offsets;
  int32_t* counts;    // [blocks, E]; scanned: what the blocks before have, and [E] of all behind
  int scanned;
  int32_t* status;
};

// How many of each block's slots go to each expert.
__global__ void __launch_bounds__(SORT_THREADS) k_expert_count(const SortP p) {
  __shared__ int hist[MAX_EXPERTS];
  for (int e = threadIdx.x; e < p.E; e += SORT_THREADS) hist[e] = 0;
  __syncthreads();
  const int64_t r0 = (int64_t)blockIdx.x * SORT_SLOTS;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < SORT_PER_LANE; ++i) {
    const int64_t s = r0 + i * SORT_THREADS + threadIdx.x;
    const int id = s < p.n ? p.ids[s] : -1;
    bad |= id >= p.E;
    if (id >= 0 && id < p.E) atomicAdd(&hist[id], 1);
  }
  if (bad) atomicCAS(p.status, 0, SBP_ERR_EXPERT_RANGE);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += SORT_THREADS) p.counts[(int64_t)blockIdx.x * p.E + e] = hist[e];
}

// Each expert's counts summed over the blocks before, once for all: a warp takes a thirty-second of
// the blocks, a lane an expert.
constexpr int SCAN_WARPS = 32, SCAN_AHEAD = 8;
__global__ void __launch_bounds__(32 * SCAN_WARPS) k_expert_scan(const SortP p) {
  __shared__ int part[SCAN_WARPS][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, e = blockIdx.x * 32 + lane;
  const int per = (p.blocks + SCAN_WARPS - 1) / SCAN_WARPS;
  const int b0 = min(warp * per, p.blocks), b1 = e < p.E ? min(b0 + per, p.blocks) : b0;
  int sum = 0;
#pragma unroll 8
  for (int b = b0; b < b1; ++b) sum += p.counts[(int64_t)b * p.E + e];
  part[warp][lane] = sum;
  __syncthreads();
  int at = 0;
  for (int w = 0; w < warp; ++w) at += part[w][lane];
  if (warp == SCAN_WARPS - 1 && e < p.E) p.counts[(int64_t)p.blocks * p.E + e] = at + sum;
  for (int b = b0; b < b1; b += SCAN_AHEAD) {
    int c[SCAN_AHEAD];
#pragma unroll
    for (int i = 0; i < SCAN_AHEAD; ++i) c[i] = b + i < b1 ? p.counts[(int64_t)(b + i) * p.E + e] : 0;
#pragma unroll
    for (int i = 0; i < SCAN_AHEAD; ++i) {
      if (b + i < b1) p.counts[(int64_t)(b + i) * p.E + e] = at;
      at += c[i];
    }
  }
}

// Each warp counts its 128 slots by expert, 32 at a time (lanes of one expert find one another
// with match_any, once); the counts' prefix over experts, blocks and warps is where each warp's
// slots of an expert begin, and a second walk over ids and lanes, kept in registers, places them.
__global__ void __launch_bounds__(SORT_THREADS) k_expert_place(const SortP p) {
  extern __shared__ int sh[];
  int* total = sh;                 // [E] of all blocks, then the experts' first rows
  int* wcnt = sh + p.E;            // [SORT_WARPS][E]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t w0 = (int64_t)blockIdx.x * SORT_SLOTS + warp * 32 * SORT_PER_LANE;
  int id[SORT_PER_LANE];
#pragma unroll
  for (int i = 0; i < SORT_PER_LANE; ++i) {
    const int64_t s = w0 + 32 * i + lane;
    id[i] = s < p.n ? p.ids[s] : -1;
  }
  for (int i = threadIdx.x; i < SORT_WARPS * p.E; i += SORT_THREADS) wcnt[i] = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < SORT_PER_LANE; ++i) {
    bad |= id[i] >= p.E;
    if (id[i] < 0 || id[i] >= p.E) id[i] = -1;
  }
  bad = __syncthreads_or(bad);
  if (p.blocks == 1 && threadIdx.x == 0) *p.status = bad ? SBP_ERR_EXPERT_RANGE : SBP_OK;
  int* mine = wcnt + warp * p.E;
  uint32_t same[SORT_PER_LANE];   // lanes of the same expert
#pragma unroll
  for (int i = 0; i < SORT_PER_LANE; ++i) {
    same[i] = 0;
    if (w0 + 32 * i >= p.n) continue;
    same[i] = __match_any_sync(0xffffffffu, id[i]);
    if (id[i] >= 0 && (same[i] & ((1u << lane) - 1u)) == 0) mine[id[i]] += __popc(same[i]);
    __syncwarp();
  }
  __syncthreads();
  // each expert's slots of the blocks before this one, and of all
  for (int e = threadIdx.x; e < p.E; e += SORT_THREADS) {
    int all = 0, before = 0;
    if (p.blocks == 1) {
      for (int w = 0; w < SORT_WARPS; ++w) all += wcnt[w * p.E + e];
    } else if (p.scanned) {
      before = p.counts[(int64_t)blockIdx.x * p.E + e];
      all = p.counts[(int64_t)p.blocks * p.E + e];
    } else {
#pragma unroll 8
      for (int b = 0; b < p.blocks; ++b) {
        const int c = p.counts[(int64_t)b * p.E + e];
        all += c;
        before += b < (int)blockIdx.x ? c : 0;
      }
    }
    total[e] = all;
    int at = before;
    for (int w = 0; w < SORT_WARPS; ++w) {
      const int c = wcnt[w * p.E + e];
      wcnt[w * p.E + e] = at;
      at += c;
    }
  }
  __syncthreads();
  if (warp == 0) {   // exclusive prefix over the experts
    int base = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const int c = e < p.E ? total[e] : 0;
      int x = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (e < p.E) {
        total[e] = base + x - c;
        if (blockIdx.x == 0) p.offsets[e] = base + x - c;
      }
      base += __shfl_sync(0xffffffffu, x, 31);
    }
    if (blockIdx.x == 0 && lane == 0) p.offsets[p.E] = base;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < SORT_PER_LANE; ++i) {
    if (w0 + 32 * i >= p.n) break;
    const int64_t s = w0 + 32 * i + lane;
    const int rank = __popc(same[i] & ((1u << lane) - 1u));
    int at = -1;
    if (id[i] >= 0) {
      at = total[id[i]] + mine[id[i]] + rank;
      p.slots[at] = (int32_t)s;
    }
    if (s < p.n) p.rows[s] = at;
    __syncwarp();
    if (id[i] >= 0 && rank == 0) mine[id[i]] += __popc(same[i]);
    __syncwarp();
  }
}

struct GatherP {
  const uint4* X;
  const float* scales;    // 8-bit rows: [T, nblk], else null
  const int32_t* rows;    // [T, k]
  int64_t T, n_rows;
  int k, nvec, nblk;      // 16-byte vectors of a row
  uint4* Xs;
  float* scales_s;
};

constexpr int GATHER_VECS = 2;   // 16-byte vectors of a thread, both in flight

// blockDim.x threads a token, blockDim.y tokens a block.
__global__ void __launch_bounds__(256) k_expert_gather(const GatherP p) {
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= p.T) return;
  const int v0 = blockIdx.y * blockDim.x * GATHER_VECS + threadIdx.x;
  uint4 x[GATHER_VECS];
#pragma unroll
  for (int i = 0; i < GATHER_VECS; ++i) {
    const int v = v0 + i * blockDim.x;
    if (v < p.nvec) x[i] = p.X[t * p.nvec + v];
  }
  const int32_t* rows = p.rows + t * p.k;
  for (int j = 0; j < p.k; ++j) {
    const int64_t r = rows[j];
    if (r < 0 || r >= p.n_rows) continue;
#pragma unroll
    for (int i = 0; i < GATHER_VECS; ++i) {
      const int v = v0 + i * blockDim.x;
      if (v < p.nvec) p.Xs[r * p.nvec + v] = x[i];
    }
    if (p.scales && blockIdx.y == 0)
      for (int c = threadIdx.x; c < p.nblk; c += blockDim.x) p.scales_s[r * p.nblk + c] = p.scales[t * p.nblk + c];
  }
}

struct CombineP {
  const void *Ys, *residual;
  const int32_t* rows;
  const float* w;         // null: ones
  int64_t T, n_rows;
  int k, d;
  void* Y;
};

// KU slots' rows in flight at a time: first where they lie and their weights, then the rows, then
// the sum.  Six blocks an SM and four rows in flight a thread do better than fewer blocks with eight
// (8192 tokens, 8 slots, d = 4096: 88 us, 6850 GB/s; 103 to 117).  In fp32 the 40 registers that six
// blocks leave do not hold four rows and the sums, and one or two slots spill 12 and 8 bytes; blocks
// still count for more: 8192 tokens, d = 4096, one and two slots 47 and 60 us, 55 and 67 with four or
// three blocks, 4096 tokens of 8 slots 88 either way; 4099 tokens, two slots, d = 2560 20.1, 22.5.
template <typename E, int KU>
__global__ void __launch_bounds__(256, 6) k_expert_combine(const CombineP p) {
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int c = 8 * (blockIdx.y * blockDim.x + threadIdx.x);
  if (t >= p.T || c >= p.d) return;
  Raw<E> res;
  res.zero();
  if (p.residual) res.load(static_cast<const E*>(p.residual) + t * p.d + c);
  F8 acc = res.f();
  const int32_t* rows = p.rows + t * p.k;
  const float* weights = p.w ? p.w + t * p.k : nullptr;
  for (int j0 = 0; j0 < p.k; j0 += KU) {
    int r[KU];
    float w[KU];
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      r[u] = j0 + u < p.k ? rows[j0 + u] : -1;
      w[u] = weights && j0 + u < p.k ? weights[j0 + u] : 1.f;
    }
    Raw<E> y[KU];
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      y[u].zero();
      if (r[u] >= 0 && r[u] < p.n_rows) y[u].load(static_cast<const E*>(p.Ys) + (int64_t)r[u] * p.d + c);
      else w[u] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      const F8 f = y[u].f();
#pragma unroll
      for (int i = 0; i < 8; ++i) acc.v[i] = fmaf(w[u], f.v[i], acc.v[i]);
    }
  }
  store8(static_cast<E*>(p.Y) + t * p.d + c, acc);
}

struct CombineBwdP {
  const void *dY, *Ys;
  const int32_t* rows;
  const float* w;
  int64_t T, n_rows;
  int k, d;
  void* dYs;
  float* dw;
};

// blockDim.x threads a token (a power of two, 8 to 256), blockDim.y tokens a block, KU slots at a
// time.  The products of a slot are summed by the thread, then over the lanes, then over the
// token's warps.  (8192 tokens, 8 slots, d = 4096, bf16: 174 us, 6560 GB/s, with three blocks an SM,
// 202 with two.)
template <typename E, int KU>
__global__ void __launch_bounds__(256, KU <= 2 ? 4 : 3) k_expert_combine_bwd(const CombineBwdP p) {
  __shared__ float red[8][KU];
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = t < p.T;
  const int tx = blockDim.x, lanes = min(tx, 32);
  const int warp = (threadIdx.y * tx + threadIdx.x) / 32;
  for (int j0 = 0; j0 < p.k; j0 += KU) {
    int r[KU];
    float w[KU], dot[KU];
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      const int j = j0 + u;
      r[u] = live && j < p.k ? p.rows[t * p.k + j] : -1;
      if (r[u] >= p.n_rows) r[u] = -1;
      w[u] = r[u] >= 0 ? p.w[t * p.k + j] : 0.f;
      dot[u] = 0.f;
    }
    for (int c = 8 * threadIdx.x; live && c < p.d; c += 8 * tx) {
      Raw<E> g, y[KU];
      g.load(static_cast<const E*>(p.dY) + t * p.d + c);
#pragma unroll
      for (int u = 0; u < KU; ++u)
        if (r[u] >= 0) y[u].load(static_cast<const E*>(p.Ys) + (int64_t)r[u] * p.d + c);
        else y[u].zero();
      const F8 gf = g.f();
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        if (r[u] < 0) continue;
        const F8 yf = y[u].f();
        F8 o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dot[u] = fmaf(gf.v[i], yf.v[i], dot[u]);
          o.v[i] = w[u] * gf.v[i];
        }
        store8(static_cast<E*>(p.dYs) + (int64_t)r[u] * p.d + c, o);
      }
    }
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      float s = dot[u];
      for (int o = lanes / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (tx > 32) {
        if (threadIdx.x % 32 == 0) red[warp][u] = s;
      } else if (live && threadIdx.x == 0 && j0 + u < p.k) {
        p.dw[t * p.k + j0 + u] = s;
      }
    }
    if (tx > 32) {
      __syncthreads();
      if (live && threadIdx.x < KU && j0 + threadIdx.x < p.k) {
        float s = 0.f;
        for (int i = 0; i < tx / 32; ++i) s += red[warp + i][threadIdx.x];
        p.dw[t * p.k + j0 + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------------------------ host side

struct SortLayout {
  int64_t n = 0, blocks = 0;
  size_t off_counts = 0, total = 0;
  Guards guards;   // checked build only
};
int sort_layout(int64_t T, int64_t k, int64_t E, SortLayout* L) {
  if (T < 0 || k < 1 || E < 1) return SBP_ERR_INVALID_ARG;
  if (E > MAX_EXPERTS || T > (int64_t(1) << 30) || k > (int64_t(1) << 30) || T * k > (int64_t(1) << 30))
    return SBP_ERR_UNSUPPORTED;
  L->n = T * k;
  L->blocks = (L->n + SORT_SLOTS - 1) / SORT_SLOTS;
  size_t o = 0;
  if (L->blocks > 1) L->off_counts = take_region(o, (size_t)(L->blocks + 1) * E * sizeof(int32_t), L->guards);
  L->total = o;   // 0: one block keeps its counts to itself
  return SBP_OK;
}

// Threads of a token (a power of two, at least 8, at most 256) and tokens of a block.
dim3 token_block(int64_t vecs) {
  unsigned x = 8;
  while (x < vecs && x < 256) x *= 2;
  return dim3(x, 256 / x);
}

int rows_check(int64_t T, int64_t k, int64_t n_rows, int64_t d, int dtype) {
  if (T < 0 || k < 1 || n_rows < 0 || d < 1 || (dtype != SBP_BF16 && dtype != SBP_FP32)) return SBP_ERR_INVALID_ARG;
  if (d % 8 != 0 || d > MAX_D || T > (int64_t(1) << 30) || k > (int64_t(1) << 30) || T * k > (int64_t(1) << 30) ||
      n_rows > (int64_t(1) << 31))
    return SBP_ERR_UNSUPPORTED;
  return SBP_OK;
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int launched() {
  if (cudaGetLastError() != cudaSuccess) return SBP_ERR_CUDA;
  set_launch_count(1);
  return SBP_OK;
}

template <typename E>
void launch_combine(const CombineP& p, cudaStream_t s) {
  const int64_t vecs = p.d / 8;
  const dim3 b = token_block(vecs), g((unsigned)((p.T + b.y - 1) / b.y), (unsigned)((vecs + b.x - 1) / b.x));
  if (p.k == 1) k_expert_combine<E, 1><<<g, b, 0, s>>>(p);
  else if (p.k == 2) k_expert_combine<E, 2><<<g, b, 0, s>>>(p);
  else k_expert_combine<E, 4><<<g, b, 0, s>>>(p);
}
template <typename E>
void launch_combine_bwd(const CombineBwdP& p, cudaStream_t s) {
  const dim3 b = token_block(p.d / 8), g((unsigned)((p.T + b.y - 1) / b.y));
  if (p.k == 1) k_expert_combine_bwd<E, 1><<<g, b, 0, s>>>(p);
  else if (p.k == 2) k_expert_combine_bwd<E, 2><<<g, b, 0, s>>>(p);
  else if constexpr (sizeof(E) == 4) k_expert_combine_bwd<E, 4><<<g, b, 0, s>>>(p);
  else if (p.k <= 4) k_expert_combine_bwd<E, 4><<<g, b, 0, s>>>(p);
  else k_expert_combine_bwd<E, 8><<<g, b, 0, s>>>(p);
}

}  // namespace
}  // namespace sbp

using namespace sbp;

extern "C" {

size_t sbp_expert_sort_workspace_bytes(int64_t T, int64_t k, int64_t E) {
  SortLayout L;
  return sort_layout(T, k, E, &L) == SBP_OK ? std::max<size_t>(L.total, 256) : 0;
}

int sbp_expert_sort(const int32_t* ids, int64_t T, int64_t k, int64_t E, int32_t* rows, int32_t* slots,
                    int32_t* offsets, void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
  SortLayout L;
  const int rc = sort_layout(T, k, E, &L);
  if (rc != SBP_OK) return rc;
  if (!offsets || !dev_status || (L.n > 0 && (!ids || !rows || !slots))) return SBP_ERR_INVALID_ARG;
  for (const void* q : {(const void*)ids, (const void*)rows, (const void*)slots, (const void*)offsets,
                        (const void*)dev_status})
    if (!aligned4(q)) return SBP_ERR_ALIGNMENT;
  if (L.total > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || ws_bytes < L.total))
    return SBP_ERR_WORKSPACE;
  NvtxRange nv("sbp_expert_sort");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(workspace);
  int launches = 1;
  const size_t smem = (size_t)(1 + SORT_WARPS) * E * sizeof(int);
  static int attr_state[64] = {};
  static std::mutex mu;
  if (!tc::once_per_device(attr_state, mu, [] {
        return cudaFuncSetAttribute(k_expert_place, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)((1 + SORT_WARPS) * MAX_EXPERTS * sizeof(int))) == cudaSuccess;
      }))
    return SBP_ERR_CUDA;
  SortP p{ids, L.n, (int)E, (int)std::max<int64_t>(L.blocks, 1), rows, slots, offsets,
          reinterpret_cast<int32_t*>(w + L.off_counts), sum_once(L.blocks, E), dev_status};
  // (a block alone writes the status itself)
  if (p.blocks > 1 && cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) != cudaSuccess) return SBP_ERR_CUDA;
  int st = workspace_guards(w, L.guards, 0, dev_status, s, &launches);
  if (st != SBP_OK) return st;
  if (p.blocks > 1) {
    k_expert_count<<<p.blocks, SORT_THREADS, 0, s>>>(p);
    ++launches;
  }
  if (p.scanned) {
    k_expert_scan<<<(unsigned)((E + 31) / 32), 32 * SCAN_WARPS, 0, s>>>(p);
    ++launches;
  }
  k_expert_place<<<p.blocks, SORT_THREADS, smem, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SBP_ERR_CUDA;
  st = workspace_guards(w, L.guards, 1, dev_status, s, &launches);
  if (st == SBP_OK) set_launch_count(launches);
  return st;
}

int sbp_expert_gather(const void* X, const float* scales, const int32_t* rows, int64_t T, int64_t k, int64_t n_rows,
                      int64_t d, int dtype, void* Xs, float* scales_s, void* stream) {
  const bool q8 = dtype == SBP_E4M3;
  const int rc = rows_check(T, k, n_rows, d, q8 ? SBP_BF16 : dtype);
  if (rc != SBP_OK) return rc;
  if (q8 && d % 16 != 0) return SBP_ERR_UNSUPPORTED;
  if (!q8 && (scales || scales_s)) return SBP_ERR_INVALID_ARG;
  if (T > 0 && (!X || !rows || (n_rows > 0 && !Xs) || (q8 && (!scales || (n_rows > 0 && !scales_s)))))
    return SBP_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(Xs) || !aligned4(rows) || !aligned4(scales) || !aligned4(scales_s))
    return SBP_ERR_ALIGNMENT;
  NvtxRange nv("sbp_expert_gather");
  set_launch_count(0);
  if (T == 0 || n_rows == 0) return SBP_OK;
  const int64_t nvec = d * (q8 ? 1 : dtype == SBP_BF16 ? 2 : 4) / 16;
  GatherP p{static_cast<const uint4*>(X), scales, rows, T, n_rows, (int)k, (int)nvec, (int)((d + 127) / 128),
            static_cast<uint4*>(Xs), scales_s};
  const dim3 b = token_block((nvec + GATHER_VECS - 1) / GATHER_VECS);
  const dim3 g((unsigned)((T + b.y - 1) / b.y), (unsigned)((nvec + b.x * GATHER_VECS - 1) / (b.x * GATHER_VECS)));
  k_expert_gather<<<g, b, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return launched();
}

int sbp_expert_combine(const void* Ys, const int32_t* rows, const float* weights, const void* residual, int64_t T,
                       int64_t k, int64_t n_rows, int64_t d, int dtype, void* Y, void* stream) {
  const int rc = rows_check(T, k, n_rows, d, dtype);
  if (rc != SBP_OK) return rc;
  if (T > 0 && (!rows || !Y || (n_rows > 0 && !Ys))) return SBP_ERR_INVALID_ARG;
  if (!aligned16(Ys) || !aligned16(residual) || !aligned16(Y) || !aligned4(rows) || !aligned4(weights))
    return SBP_ERR_ALIGNMENT;
  NvtxRange nv("sbp_expert_combine");
  set_launch_count(0);
  if (T == 0) return SBP_OK;
  CombineP p{Ys, residual, rows, weights, T, n_rows, (int)k, (int)d, Y};
  if (dtype == SBP_BF16) launch_combine<__nv_bfloat16>(p, static_cast<cudaStream_t>(stream));
  else launch_combine<float>(p, static_cast<cudaStream_t>(stream));
  return launched();
}

int sbp_expert_combine_backward(const void* dY, const void* Ys, const int32_t* rows, const float* weights, int64_t T,
                                int64_t k, int64_t n_rows, int64_t d, int dtype, void* dYs, float* dweights,
                                void* stream) {
  const int rc = rows_check(T, k, n_rows, d, dtype);
  if (rc != SBP_OK) return rc;
  if (T > 0 && (!dY || !rows || !weights || !dweights || (n_rows > 0 && (!Ys || !dYs)))) return SBP_ERR_INVALID_ARG;
  if (!aligned16(dY) || !aligned16(Ys) || !aligned16(dYs) || !aligned4(rows) || !aligned4(weights) ||
      !aligned4(dweights))
    return SBP_ERR_ALIGNMENT;
  NvtxRange nv("sbp_expert_combine_backward");
  set_launch_count(0);
  if (T == 0) return SBP_OK;
  CombineBwdP p{dY, Ys, rows, weights, T, n_rows, (int)k, (int)d, dYs, dweights};
  if (dtype == SBP_BF16) launch_combine_bwd<__nv_bfloat16>(p, static_cast<cudaStream_t>(stream));
  else launch_combine_bwd<float>(p, static_cast<cudaStream_t>(stream));
  return launched();
}

}  // extern "C"
