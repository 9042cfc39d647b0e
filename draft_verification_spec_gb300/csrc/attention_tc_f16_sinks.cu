// f16 instances of the tcgen05 attention kernel with first tokens that stay visible.
#include "attention_tc.cuh"

namespace sv {

template <>
const void* attn_tc_fn<false, true>(int dp, bool wide) {
  if (wide)
    return dp == 64 ? reinterpret_cast<const void*>(&attn_tc_kernel<false, 64, true, true, false, false>)
                    : reinterpret_cast<const void*>(&attn_tc_kernel<false, 128, true, true, false, false>);
  return dp == 64 ? reinterpret_cast<const void*>(&attn_tc_kernel<false, 64, false, true, false, false>)
                  : reinterpret_cast<const void*>(&attn_tc_kernel<false, 128, false, true, false, false>);
}

}  // namespace sv
