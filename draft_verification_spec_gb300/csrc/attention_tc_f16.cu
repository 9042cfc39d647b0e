// f16 instances of the tcgen05 attention kernel.
#include "attention_tc.cuh"

namespace sv {

template <>
const void* attn_tc_fn<false>(int dp) {
  return dp == 64 ? reinterpret_cast<const void*>(&attn_tc_kernel<false, 64>)
                  : reinterpret_cast<const void*>(&attn_tc_kernel<false, 128>);
}

}  // namespace sv
