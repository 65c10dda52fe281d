#include "attn_fwd_impl.h"

namespace ssm {
namespace {

// Joins the parts of a (query, head) by their maxima and sums: a wave for one, two channels a lane
__global__ __launch_bounds__(256) void attn_fwd_join_kernel(const AttnArgs a) {
  const size_t row = static_cast<size_t>(blockIdx.x) * 4 + threadIdx.x / 64, rows = static_cast<size_t>(a.rows_q) * a.h;
  if (row >= rows) return;
  const int lane = threadIdx.x % 64, dq = (a.D + 31) / 32 * 32, d = 2 * lane;
  const float2* const stats = reinterpret_cast<const float2*>(a.part + rows * a.nsplit * dq) + row * a.nsplit;
  float top = -INFINITY;
  for (int y = lane; y < a.nsplit; y += 64) top = fmaxf(top, stats[y].x);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
  const float sub = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f, x0 = 0.0f, x1 = 0.0f;
  const float* const p = a.part + row * a.nsplit * dq + d;
#pragma unroll 4
  for (int y = 0; y < a.nsplit; ++y) {
    const float2 st = stats[y];
    const float f = exp2_fast(st.x - sub);
    sum = fmaf(st.y, f, sum);
    if (d < a.D) {
      const float2 v = *reinterpret_cast<const float2*>(p + static_cast<size_t>(y) * dq);
      x0 = fmaf(v.x, f, x0);
      x1 = fmaf(v.y, f, x1);
    }
  }
  const bool some = sum > 0.0f || sum != sum;
  const float inv = some ? 1.0f / sum : 0.0f;
  if (a.lse && lane == 0) a.lse[row] = some ? (top + log2_fast(sum)) * kLn2 : -INFINITY;
  if (d >= a.D) return;
  x0 *= inv;
  x1 *= inv;
  *reinterpret_cast<uint32_t*>(static_cast<bf16s*>(a.o) + row * a.D + d) = pack_rne(x0, x1);
  if (a.o_rest) *reinterpret_cast<uint32_t*>(static_cast<bf16s*>(a.o_rest) + row * a.D + d) = pack_rne(rest_of(x0), rest_of(x1));
}

}  // namespace

// P enters its product in two bf16 parts for an o in bf16: with one it would be 1.4 times as far from the exact
// value as its own rounding makes it.
hipError_t attn_fwd_bf16(const AttnLaunch& l, hipStream_t s) {
  const AttnArgs& a = l.a;
  const long blocks = attn_tiles(a, 128, false) * a.h;
  // 128 queries a workgroup where that fills the CUs twice; where it does not, and the workgroups may have 1024
  // keys and more to go through, the kernel whose workgroup fills a CU by itself (500 queries behind 15000
  // tokens, 2 x 32 heads of 128: 320 us, with 64 queries a workgroup 486, with the wide kernel 697; 512 of 1024
  // keys, 8 heads: 23.6 and 23.9 with 64 queries); else 64 queries a workgroup.  The host knows the keys of a packed
  // call only in total: a pack of short prompts goes to the kernel for long ones too (32 of 40 tokens, 8 heads of
  // 128: 20 us, with 64 queries a workgroup 7).
  if (a.vec == 2 && blocks >= 512) return attn_fwd_wide<2>(l, false, s);
  if (a.vec == 2 && a.lk >= 1024 && a.window >= 1024) {
    const hipError_t e = attn_fwd_wide<2>(l, true, s);
    if (e != hipSuccess || a.nsplit == 1) return e;
    hipLaunchKernelGGL(attn_fwd_join_kernel, dim3(static_cast<unsigned>((a.rows_q * a.h + 3) / 4)), dim3(256), 0, s, a);
    return hipGetLastError();
  }
  return attn_fwd_narrow<bf16s, 2>(l, s);
}

hipError_t launch_attn_fwd(const AttnLaunch& l, hipStream_t s) {
  if (l.a.rows_q == 0 || l.a.nseq == 0) return hipSuccess;
  if (l.in_dtype != kBF16) return attn_fwd_f32(l, s);
  return l.o_dtype == kBF16 ? attn_fwd_bf16(l, s) : attn_fwd_bf16_f32(l, s);
}

}  // namespace ssm
