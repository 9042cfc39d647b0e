// f16 instances of the tcgen05 attention kernel.
#include "attention_tc.cuh"

namespace sv {

template <>
const void* attn_tc_fn<false>(int dp, bool wide) {
  if (wide)
    return dp == 64 ? reinterpret_cast<const void*>(&attn_tc_kernel<false, 64, true>)
                    : reinterpret_cast<const void*>(&attn_tc_kernel<false, 128, true>);
  return dp == 64 ? reinterpret_cast<const void*>(&attn_tc_kernel<false, 64, false>)
                  : reinterpret_cast<const void*>(&attn_tc_kernel<false, 128, false>);
}

}  // namespace sv
