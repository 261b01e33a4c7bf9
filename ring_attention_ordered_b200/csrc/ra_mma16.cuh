// The 16-bit tcgen05.mma sequences of one attention tile (kind::f16, bf16 or
// fp16 by the instruction descriptor), shared by the bf16 forward kernel and
// the cache attention kernel.  A tile row of D values is D / 64 boxes of 64
// columns (one 128-byte swizzle row each), BOX_BYTES apart.
#pragma once

#include <cstdint>

#include "ptx_sm100.cuh"

namespace ra {

constexpr int BOX_BYTES = 128 * 128;

template <int KK>
struct QkStep {
  static constexpr uint32_t OFF = ((KK / 4) * BOX_BYTES + (KK % 4) * 32) >> 4;
};

// S = Q K^T over the head dimension: D/16 MMAs of K = 16, each issued by
// the elected lane.
template <int D>
__device__ __forceinline__ void mma_qk_steps(uint32_t d, uint32_t a, uint32_t b, uint32_t hi,
                                             uint32_t idesc) {
  if (elect_one()) mma_ss<QkStep<0>::OFF, QkStep<0>::OFF>(d, a, hi, b, hi, idesc, 0u);
  if (elect_one()) mma_ss<QkStep<1>::OFF, QkStep<1>::OFF>(d, a, hi, b, hi, idesc, 1u);
  if (elect_one()) mma_ss<QkStep<2>::OFF, QkStep<2>::OFF>(d, a, hi, b, hi, idesc, 1u);
  if (elect_one()) mma_ss<QkStep<3>::OFF, QkStep<3>::OFF>(d, a, hi, b, hi, idesc, 1u);
  if constexpr (D == 128) {
    if (elect_one()) mma_ss<QkStep<4>::OFF, QkStep<4>::OFF>(d, a, hi, b, hi, idesc, 1u);
    if (elect_one()) mma_ss<QkStep<5>::OFF, QkStep<5>::OFF>(d, a, hi, b, hi, idesc, 1u);
    if (elect_one()) mma_ss<QkStep<6>::OFF, QkStep<6>::OFF>(d, a, hi, b, hi, idesc, 1u);
    if (elect_one()) mma_ss<QkStep<7>::OFF, QkStep<7>::OFF>(d, a, hi, b, hi, idesc, 1u);
  }
}

// O (+)= P V over one half of the 128 keys (HALF 0: keys 0-63, 1: keys
// 64-127): 4 MMAs of K = 16; P's 16 keys are 8 TMEM columns of bf16 pairs,
// V's 16 keys are 16 rows of 128 bytes (2048 bytes).  `acc` applies to the
// first MMA of the first half only.
template <int HALF>
__device__ __forceinline__ void mma_pv_half(uint32_t d, uint32_t p_tmem, uint32_t b, uint32_t hi,
                                            uint32_t idesc, uint32_t acc) {
  constexpr uint32_t C0 = 32 * HALF, B0 = 512 * HALF;
  if (elect_one()) mma_ts<C0 + 0, B0 + 0>(d, p_tmem, b, hi, idesc, HALF ? 1u : acc);
  if (elect_one()) mma_ts<C0 + 8, B0 + 128>(d, p_tmem, b, hi, idesc, 1u);
  if (elect_one()) mma_ts<C0 + 16, B0 + 256>(d, p_tmem, b, hi, idesc, 1u);
  if (elect_one()) mma_ts<C0 + 24, B0 + 384>(d, p_tmem, b, hi, idesc, 1u);
}

}  // namespace ra
