// bf16 instances of the mma.sync attention kernel.
#include "attention_mma.cuh"

namespace sv {

template <>
const void* attn_mma_fn<true>(int dp, int bm) {
  if (bm == 16)
    return dp == 64    ? reinterpret_cast<const void*>(&attn_mma_kernel<true, 64, 1>)
           : dp == 128 ? reinterpret_cast<const void*>(&attn_mma_kernel<true, 128, 1>)
                       : reinterpret_cast<const void*>(&attn_mma_kernel<true, 256, 1>);
  return dp == 64    ? reinterpret_cast<const void*>(&attn_mma_kernel<true, 64, 4>)
         : dp == 128 ? reinterpret_cast<const void*>(&attn_mma_kernel<true, 128, 4>)
                     : reinterpret_cast<const void*>(&attn_mma_kernel<true, 256, 4>);
}

}  // namespace sv
