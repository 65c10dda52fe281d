#include "attn_bwd_impl.h"

namespace ssm {

hipError_t attn_bwd_f32(const AttnArgs& a, hipStream_t s) { return attn_bwd_d<float, 1>(a, s); }

// bf16 inputs and gradients in f32: P and dS in three bf16 parts
hipError_t attn_bwd_bf16_f32(const AttnArgs& a, hipStream_t s) { return attn_bwd_d<bf16s, 3>(a, s); }

}  // namespace ssm
