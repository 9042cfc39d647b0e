// bf16 instances of the attention over 4-bit caches.
#include "attention_fp4.cuh"

namespace sv {

template <>
const void* attn_fp4_fn<true>(int dp) {
  return dp == 64    ? reinterpret_cast<const void*>(&attn_fp4_kernel<true, 64>)
         : dp == 128 ? reinterpret_cast<const void*>(&attn_fp4_kernel<true, 128>)
                     : reinterpret_cast<const void*>(&attn_fp4_kernel<true, 256>);
}

}  // namespace sv
