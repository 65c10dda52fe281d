#include "attn_fwd_impl.h"

namespace ssm {

// P enters its product in two bf16 parts for an o in bf16.
hipError_t attn_fwd_bf16(const AttnLaunch& l, hipStream_t s) {
  // 128 queries a workgroup where that still gives every CU two workgroups
  if (l.a.vec == 2 && attn_tiles(l.a, 128, false) * l.a.h >= 512) return attn_fwd_d<bf16s, 2, 2, true>(l, s);
  return attn_fwd_narrow<bf16s, 2>(l, s);
}

hipError_t launch_attn_fwd(const AttnLaunch& l, hipStream_t s) {
  if (l.a.rows_q == 0 || l.a.nseq == 0) return hipSuccess;
  if (l.in_dtype != kBF16) return attn_fwd_f32(l, s);
  return l.o_dtype == kBF16 ? attn_fwd_bf16(l, s) : attn_fwd_bf16_f32(l, s);
}

}  // namespace ssm
