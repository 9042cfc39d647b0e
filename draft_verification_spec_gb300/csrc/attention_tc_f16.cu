// f16 instances of the tcgen05 attention kernel.
#include "attention_tc.cuh"

namespace sv {

template <>
const void* attn_tc_fn<false, false>(int dp, bool wide) {
  if (wide)
    return dp == 64 ? reinterpret_cast<const void*>(&attn_tc_kernel<false, 64, true, false, false, false>)
                    : reinterpret_cast<const void*>(&attn_tc_kernel<false, 128, true, false, false, false>);
  return dp == 64 ? reinterpret_cast<const void*>(&attn_tc_kernel<false, 64, false, false, false, false>)
                  : reinterpret_cast<const void*>(&attn_tc_kernel<false, 128, false, false, false, false>);
}

}  // namespace sv
