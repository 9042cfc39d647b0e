// bf16 instances of the tcgen05 attention kernel over 4-bit caches.
#include "attention_tc.cuh"

namespace sv {

template <>
const void* attn_tc_fp4_fn<true>(int dp, bool wide) {
  if (wide)
    return dp == 64 ? reinterpret_cast<const void*>(&attn_tc_kernel<true, 64, true, true, true>)
                    : reinterpret_cast<const void*>(&attn_tc_kernel<true, 128, true, true, true>);
  return dp == 64 ? reinterpret_cast<const void*>(&attn_tc_kernel<true, 64, false, true, true>)
                  : reinterpret_cast<const void*>(&attn_tc_kernel<true, 128, false, true, true>);
}

}  // namespace sv
