// bf16 instances of the tcgen05 attention kernel over 4-bit caches.
#include "attention_tc.cuh"

namespace sv {

template <bool WHOLE>
static const void* instance(int dp, bool wide) {
  if (wide)
    return dp == 64 ? reinterpret_cast<const void*>(&attn_tc_kernel<true, 64, true, true, true, WHOLE>)
                    : reinterpret_cast<const void*>(&attn_tc_kernel<true, 128, true, true, true, WHOLE>);
  return dp == 64 ? reinterpret_cast<const void*>(&attn_tc_kernel<true, 64, false, true, true, WHOLE>)
                  : reinterpret_cast<const void*>(&attn_tc_kernel<true, 128, false, true, true, WHOLE>);
}

template <>
const void* attn_tc_fp4_fn<true>(int dp, bool wide, bool whole) {
  return whole ? instance<true>(dp, wide) : instance<false>(dp, wide);
}

}  // namespace sv
