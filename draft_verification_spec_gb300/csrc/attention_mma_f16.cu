// f16 instances of the mma.sync attention kernel.
#include "attention_mma.cuh"

namespace sv {

template <>
const void* attn_mma_fn<false, false>(int dp, int bm) {
  if (bm == 16)
    return dp == 64    ? reinterpret_cast<const void*>(&attn_mma_kernel<false, 64, 1, false>)
           : dp == 128 ? reinterpret_cast<const void*>(&attn_mma_kernel<false, 128, 1, false>)
                       : reinterpret_cast<const void*>(&attn_mma_kernel<false, 256, 1, false>);
  return dp == 64    ? reinterpret_cast<const void*>(&attn_mma_kernel<false, 64, 4, false>)
         : dp == 128 ? reinterpret_cast<const void*>(&attn_mma_kernel<false, 128, 4, false>)
                     : reinterpret_cast<const void*>(&attn_mma_kernel<false, 256, 4, false>);
}

}  // namespace sv
