// bf16 instances of the attention over 4-bit caches.
#include "attention_fp4.cuh"

namespace sv {

template <>
const void* attn_fp4_fn<true>(int dp, int bm) {
  if (bm == 8)
    return dp == 64    ? reinterpret_cast<const void*>(&attn_fp4_kernel<true, 64, 1>)
           : dp == 128 ? reinterpret_cast<const void*>(&attn_fp4_kernel<true, 128, 1>)
                       : reinterpret_cast<const void*>(&attn_fp4_kernel<true, 256, 1>);
  if (bm == 32)
    return dp == 64 ? reinterpret_cast<const void*>(&attn_fp4_kernel<true, 64, 4>)
                    : reinterpret_cast<const void*>(&attn_fp4_kernel<true, 128, 4>);
  return dp == 64    ? reinterpret_cast<const void*>(&attn_fp4_kernel<true, 64, 2>)
         : dp == 128 ? reinterpret_cast<const void*>(&attn_fp4_kernel<true, 128, 2>)
                     : reinterpret_cast<const void*>(&attn_fp4_kernel<true, 256, 2>);
}

}  // namespace sv
