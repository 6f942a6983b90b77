// Chunked causal-attention backward at head dimension 128: launches of the fused kernels
// (sbp_attn_fused.cuh) over causal chunks.
#include "sbp_attn_fused.cuh"

namespace sbp {

// ========================================================================== host side

namespace {

bool fused_attrs() {
  static int attr_state[64] = {};
  static std::mutex mu;
  return tc::once_per_device(attr_state, mu, [] {
    return cudaFuncSetAttribute(tc::fa::k_attn_kv<tc::fa::CausalScores>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)tc::fa::SMEM_KV) == cudaSuccess &&
           cudaFuncSetAttribute(tc::fa::k_attn_q<tc::fa::CausalScores>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)tc::fa::SMEM_Q) == cudaSuccess;
  });
}

}  // namespace

bool AttnFusedPlan::init(const void* Q, const void* K, const void* V, const void* dO, float* dK_, float* dV_,
                         int64_t T_, int64_t H_, int64_t Hkv_) {
  T = T_;
  H = H_;
  Hkv = Hkv_;
  // query-side operands over H heads, key / value side (and dK, dV) over Hkv heads
  using tc::make_map_heads;
  return make_map_heads(&K128, K, T, Hkv, 128, 128) && make_map_heads(&V128, V, T, Hkv, 128, 128) &&
         make_map_heads(&Q64, Q, T, H, 128, 64) && make_map_heads(&O64, dO, T, H, 128, 64) &&
         make_map_heads(&Q128, Q, T, H, 128, 128) && make_map_heads(&O128, dO, T, H, 128, 128) &&
         make_map_heads(&K64, K, T, Hkv, 128, 64) && make_map_heads(&V64, V, T, Hkv, 128, 64) &&
         tc::make_map_out(&dK, dK_, T, T, Hkv, 128, 4) && tc::make_map_out(&dV, dV_, T, T, Hkv, 128, 4);
}

cudaError_t attn_fused_kv(const AttnFusedPlan& plan, int64_t c0, int64_t c1, float scale, const float* lse,
                          const float* D, int32_t* status, cudaStream_t s) {
  using namespace tc;
  using namespace tc::fa;
  if (!fused_attrs()) return cudaErrorInvalidConfiguration;
  KvP p;
  p.H = (int)plan.H; p.T = (int)plan.T; p.c0 = (int)c0; p.c1 = (int)c1;
  p.nb = (int)((c1 - c0 + 127) / 128);
  p.Hkv = (int)plan.Hkv;
  p.group = (int)(plan.H / plan.Hkv);
  p.n_units = (int)((c1 + 255) / 256) * p.Hkv;
  p.scale = scale; p.lse = lse; p.D = D; p.status = status; p.limit_ns = wait_limit_ns();
  int pairs = max_pairs((const void*)k_attn_kv<CausalScores>, SMEM_KV, KV_THREADS);
  if (pairs > p.n_units) pairs = p.n_units;
  k_attn_kv<CausalScores><<<2 * pairs, KV_THREADS, SMEM_KV, s>>>(
      MapArray<KV_MAPS>{{plan.K128, plan.V128, plan.Q64, plan.O64, plan.Q128, plan.O128, plan.dK, plan.dV}}, p);
  return cudaGetLastError();
}

cudaError_t attn_fused_q(const AttnFusedPlan& plan, int64_t c0, int64_t c1, float scale, const float* lse,
                         const float* D, void* dQ, int32_t* status, cudaStream_t s) {
  using namespace tc;
  using namespace tc::fa;
  if (!fused_attrs()) return cudaErrorInvalidConfiguration;
  QP p;
  p.H = (int)plan.H; p.T = (int)plan.T; p.c0 = (int)c0; p.c1 = (int)c1;
  p.n_qp = (int)((c1 - c0 + 255) / 256);
  p.n_units = p.n_qp * p.H;
  p.group = (int)(plan.H / plan.Hkv);
  p.scale = scale; p.lse = lse; p.D = D; p.status = status; p.limit_ns = wait_limit_ns();
  int pairs = max_pairs((const void*)k_attn_q<CausalScores>, SMEM_Q, Q_THREADS);
  if (pairs > p.n_units) pairs = p.n_units;
  MapArray<Q_MAPS> maps{{plan.Q128, plan.O128, plan.K64, plan.V64, plan.K128}};
  // the chunk's rows of dQ and no later ones
  if (!make_map_out(&maps.m[Q_MOUT], dQ, c1, plan.T, plan.H, 128, 2)) return cudaErrorInvalidValue;
  k_attn_q<CausalScores><<<2 * pairs, Q_THREADS, SMEM_Q, s>>>(maps, p);
  return cudaGetLastError();
}

}  // namespace sbp
