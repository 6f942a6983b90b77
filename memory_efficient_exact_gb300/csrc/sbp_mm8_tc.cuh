// Shared by the tcgen05 kernels of the block-scaled 8-bit product.
#pragma once

#include "sbp_mm8.cuh"
#include "sbp_tc_common.cuh"

namespace sbp {
namespace tc {

__device__ __forceinline__ void mma2_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(
          d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// Instruction descriptor of tcgen05.mma kind::f8f6f4: D fp32 (bits 4-5 = 1), A and B e4m3 (bits
// 7-9 and 10-12 = 0), both K-major, N >> 3 at bit 17, M >> 4 at bit 24.
constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

template <class C>
__device__ __forceinline__ void fail_mm8(C* c, int32_t* status) {
  *(volatile int*)&c->abort = 1;
  if (status) atomicCAS(status, 0, SBP_ERR_TIMEOUT);
}
// An arrival on a barrier of this CTA, or on one of the pair's (no branch).  The remote one has the
// instruction's default semantics, as arrive_remote: nothing in memory is handed over with it, only an
// accumulator whose values tcgen05.wait::ld has shown to be in registers.  A release at cluster scope
// costs 548 us instead of 288 for 32768 x 2560 x 4096 of 32 experts, 99 instead of 33 for 501 x 4096 x
// 12288, 233 instead of 108 for 64 rows of 64 experts.
__device__ __forceinline__ void arrive_if(bool here, uint32_t local, bool there, uint32_t remote) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %0, 0;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%1];\n\t@q mbarrier.arrive.shared::cluster.b64 _, [%3];\n\t}" ::"r"(
          (int)here),
      "r"(local), "r"((int)there), "r"(remote)
      : "memory");
}
template <bool CLUSTER, class C>
__device__ __forceinline__ bool warp_wait(uint64_t* b, uint32_t parity, C* c, uint64_t limit) {
  return __all_sync(0xffffffffu, wait_inl<CLUSTER>(b, parity & 1u, &c->abort, limit));
}
// Tiles are walked in bands of this many units of rows, all columns of a band before the next:
// the 76 pairs' tiles then share 8 blocks of A's rows and 9 or 10 of B's.  (16: 2% slower.)
constexpr int BAND = 8;

struct Tile {
  mm8::Unit w;
  int n0;
};
__device__ __forceinline__ Tile tile_of(const mm8::P& p, int unit, int units, int ntn, int bn, int t) {
  const int band = t / (BAND * ntn), r = t - band * BAND * ntn;
  const int high = min(BAND, units - band * BAND);
  Tile o;
  o.w = mm8::unit_of(p, unit, band * BAND + r % high);
  o.n0 = r / high * bn;
  return o;
}

// Map over a row-major array of bytes, boxes of 128 bytes x `rows`, 128-byte swizzle, zeros outside.
inline bool make_map_u8(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer, uint64_t pitch,
                        uint32_t rows) {
  auto enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {pitch};
  cuuint32_t box[2] = {128, rows};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc
}  // namespace sbp
