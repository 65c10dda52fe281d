#include "attn_fwd_impl.h"

namespace ssm {

hipError_t attn_fwd_f32(const AttnLaunch& l, hipStream_t s) {
  return attn_fwd_narrow<float, 1>(l, s);
}

// bf16 inputs and an o in f32: P in three bf16 parts, all 24 bits.
hipError_t attn_fwd_bf16_f32(const AttnLaunch& l, hipStream_t s) {
  return attn_fwd_narrow<bf16s, 3>(l, s);
}

}  // namespace ssm
