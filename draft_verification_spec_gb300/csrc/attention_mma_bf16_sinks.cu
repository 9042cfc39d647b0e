// bf16 instances of the mma.sync attention kernel with first tokens that stay visible.
#include "attention_mma.cuh"

namespace sv {

template <>
const void* attn_mma_fn<true, true>(int dp, int bm) {
  if (bm == 16)
    return dp == 64    ? reinterpret_cast<const void*>(&attn_mma_kernel<true, 64, 1, true>)
           : dp == 128 ? reinterpret_cast<const void*>(&attn_mma_kernel<true, 128, 1, true>)
                       : reinterpret_cast<const void*>(&attn_mma_kernel<true, 256, 1, true>);
  return dp == 64    ? reinterpret_cast<const void*>(&attn_mma_kernel<true, 64, 4, true>)
         : dp == 128 ? reinterpret_cast<const void*>(&attn_mma_kernel<true, 128, 4, true>)
                     : reinterpret_cast<const void*>(&attn_mma_kernel<true, 256, 4, true>);
}

}  // namespace sv
