#include "attn_fwd_impl.h"

namespace ssm {

// P enters its product in two bf16 parts for an o in bf16: with one it would be 1.4 times as far from the exact
// value as its own rounding makes it.
hipError_t attn_fwd_bf16(const AttnLaunch& l, hipStream_t s) {
  const AttnArgs& a = l.a;
  const long blocks = attn_tiles(a, 128, false) * a.h;
  // 128 queries a workgroup where that fills the CUs twice; where it does not, and the workgroups have 1024
  // keys and more to go through, the kernel whose workgroup fills a CU by itself (500 queries behind 15000
  // tokens, 2 x 32 heads of 128: 320 us, with 64 queries a workgroup 486, with the wide kernel 697; 512 of 1024
  // keys, 8 heads: 23.6 and 23.9 with 64 queries); else 64
  // queries a workgroup.
  if (a.vec == 2 && blocks >= 512) return attn_fwd_wide<2>(l, false, s);
  if (a.vec == 2 && a.lk >= 1024 && a.window >= 1024) return attn_fwd_wide<2>(l, true, s);
  return attn_fwd_narrow<bf16s, 2>(l, s);
}

hipError_t launch_attn_fwd(const AttnLaunch& l, hipStream_t s) {
  if (l.a.rows_q == 0 || l.a.nseq == 0) return hipSuccess;
  if (l.in_dtype != kBF16) return attn_fwd_f32(l, s);
  return l.o_dtype == kBF16 ? attn_fwd_bf16(l, s) : attn_fwd_bf16_f32(l, s);
}

}  // namespace ssm
