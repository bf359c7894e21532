// Device helpers shared by the differential-attention read kernels.
#pragma once

#include "pa_tc_common.cuh"

namespace pa {
namespace diff {

// Probabilities enter the products as two T parts (value and remainder) of
// 2^(s - m + shift), m the row's running maximum, which may lag behind by `lazy`;
// their sum carries the same factor, so it cancels. bf16 has f32's exponents.
// fp16 ends below 2^16 and its least step is 2^-24, which no remainder passes:
// with shift + lazy = 15 a probability is off by 2^-25 / 2^shift = 2^-34 of the
// row's largest at most. (With shift 0 and 2^-25, a key that takes nearly all of the
// weight at a value near zero left relative errors of up to 4e-2, as the norm
// scales up the small rest. A smaller lag leaves more room below, but a tile
// whose maximum passes the running one by more is computed twice: prefill of
// 26 drawn cases takes 1.3 % longer with 4 than with 8, 0.5 % with 6.)
template <typename T> struct Prob;
template <> struct Prob<__nv_bfloat16> {
  static constexpr float lazy = 8.f, shift = 0.f;
};
template <> struct Prob<__half> {
  static constexpr float lazy = 6.f, shift = 9.f;
};

// True in one lane of the warp (converged). Code behind `if (elect_one())` is
// known to run in a single lane, so its TMA and MMA operands stay in uniform
// registers; behind `if (lane == 0)` every such instruction moved them there
// again (some 90 cycles per MMA, 190 per TMA copy).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

}  // namespace diff
}  // namespace pa
