// Device helpers shared by the differential-attention read kernels.
#pragma once

#include "pa_tc_common.cuh"

namespace pa {
namespace diff {

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
