#include "attn_bwd_impl.h"

namespace ssm {
namespace {

// delta = sum_d do o: 16 lanes per (query, head), 8 channels each, four rows in turn (a launch's 2^32
// threads hold 2^30 rows that way)
template <typename T, typename OT>
__global__ __launch_bounds__(256) void attn_delta_kernel(const AttnArgs a, long rows) {
  const int d = threadIdx.x % 16 * 8;
  for (int i = 0; i < 4; ++i) {
    const long row = static_cast<long>(blockIdx.x) * 64 + 16 * i + threadIdx.x / 16;
    if (row >= rows) return;  // whole lane groups leave together
    float x = 0.0f;
    if (d < a.D) {
      const T* const p = static_cast<const T*>(a.dout) + row * a.D;
      const OT* const q = static_cast<const OT*>(a.o) + row * a.D;
      Row8<T> u;
      Row8<OT> v;
      const bool vec = a.vec == 2 && a.D % 8 == 0;
      u.load(p, d, a.D, vec);
      v.load(q, d, a.D, vec);
      float f[8], h[8];
      u.get(a.D - d, f);
      v.get(a.D - d, h);
#pragma unroll
      for (int e = 0; e < 8; ++e) x = fmaf(f[e], h[e], x);
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) x += __shfl_xor(x, o);
    if (threadIdx.x % 16 == 0) a.delta[row] = x;
  }
}

// Adds the pieces' partial sums of the keys of the sinks' tiles, in order: a workgroup per (sequence, key
// head, tile)
__global__ __launch_bounds__(256) void attn_sink_kernel(const AttnArgs a) {
  const int tile = blockIdx.x % a.sink_tiles, r = blockIdx.x / a.sink_tiles, kh = r % a.hk, s = r / a.hk;
  const AttnSeq q = attn_seq(a, s);
  const long slot = a.cu_q ? q.q0 / a.span + s : static_cast<long>(s) * ((a.lq + a.span - 1) / a.span);
  const int pieces = (q.nq + a.span - 1) / a.span;
  const int rows = min(64, q.nk - tile * 64);
  for (int e = threadIdx.x; e < rows * a.D; e += 256) {
    float k = 0.0f, v = 0.0f;
    for (int p = 0; p < pieces; ++p) {
      const size_t at = ((static_cast<size_t>(slot + p) * a.hk + kh) * a.sink_tiles + tile) * 64 * a.D + e;
      k += a.dk_part[at];
      v += a.dv_part[at];
    }
    const size_t to = (static_cast<size_t>(q.k0 + tile * 64 + e / a.D) * a.hk + kh) * a.D + e % a.D;
    if (a.grad_bf16) {
      if (a.dk) st<bf16s>(a.dk, to, k);
      if (a.dv) st<bf16s>(a.dv, to, v);
    } else {
      if (a.dk) st<float>(a.dk, to, k);
      if (a.dv) st<float>(a.dv, to, v);
    }
  }
}

template <typename T, typename OT>
hipError_t delta_go(const AttnArgs& a, hipStream_t s) {
  const long rows = a.rows_q * a.h;
  hipLaunchKernelGGL((attn_delta_kernel<T, OT>), dim3(static_cast<unsigned>((rows + 63) / 64)), dim3(256), 0, s, a, rows);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_sinks(const AttnArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(attn_sink_kernel, dim3(static_cast<unsigned>(a.nseq) * a.hk * a.sink_tiles), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t attn_bwd_bf16(const AttnLaunch& l, hipStream_t s) { return attn_bwd_d<bf16s, 1, 2>(l, s); }

hipError_t launch_attn_bwd(const AttnLaunch& l, hipStream_t s) {
  if (l.a.nseq == 0) return hipSuccess;
  if (l.a.rows_q > 0) {
    hipError_t e;
    if (l.in_dtype == kBF16) e = l.o_dtype == kBF16 ? delta_go<bf16s, bf16s>(l.a, s) : delta_go<bf16s, float>(l.a, s);
    else e = l.o_dtype == kBF16 ? delta_go<float, bf16s>(l.a, s) : delta_go<float, float>(l.a, s);
    if (e != hipSuccess) return e;
  }
  if (l.in_dtype != kBF16) return attn_bwd_f32(l, s);
  return l.grad_dtype == kBF16 ? attn_bwd_bf16(l, s) : attn_bwd_bf16_f32(l, s);
}

}  // namespace ssm
