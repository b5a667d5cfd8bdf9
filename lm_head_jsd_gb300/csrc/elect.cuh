// One lane of a warp that stays together: the issuing warps of the products run
// their loops with all lanes and elect one for each group of copies or products,
// rather than entering the loop with one lane. The compiler then knows that what these
// instructions take from uniform registers (descriptors, barriers, addresses) is the
// same in all lanes; in a loop of one lane it cannot, and issuing a block's products
// takes longer. With one lane and with the warp: 4096 rows of 4096 x 128256 logits
// 2242 and 2100 us, 333 rows of 2048 x 40960 94 and 83, one row of 4096 x 128256 183
// and 177, the 8-bit product 1823 and 1765.
#pragma once

#include <cstdint>

namespace fljsd {

// True in one lane. All lanes of the warp must be here.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      :
      : "memory");
  return r != 0;
}

}  // namespace fljsd
