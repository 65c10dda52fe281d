#include "attn_bwd_impl.h"

namespace ssm {
namespace {

// delta = sum_d do (o + o_rest): 16 lanes per (query, head), 8 channels each, four rows in turn (a launch's 2^32
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
      if (a.o_rest) {
        Row8<bf16s> w;
        w.load(static_cast<const bf16s*>(a.o_rest) + row * a.D, d, a.D, vec);
        w.get(a.D - d, h);
#pragma unroll
        for (int e = 0; e < 8; ++e) x = fmaf(f[e], h[e], x);
      }
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) x += __shfl_xor(x, o);
    if (threadIdx.x % 16 == 0) a.delta[row] = x;
  }
}

// Adds the pieces' partial sums of the keys of the sinks' tiles, in order: a workgroup for four keys of a
// (sequence, key head, tile)
__global__ __launch_bounds__(256) void attn_sink_kernel(const AttnArgs a) {
  const int part = blockIdx.y;
  unsigned r = blockIdx.x;
  const int tile = r % a.sink_tiles;
  r /= a.sink_tiles;
  const int kh = r % a.hk, s = r / a.hk;
  const AttnSeq q = attn_seq(a, s);
  const long slot = a.cu_q ? q.q0 / a.span + s : static_cast<long>(s) * ((a.lq + a.span - 1) / a.span);
  const int pieces = (q.nq + a.span - 1) / a.span, j0 = tile * kSinkRows;
  const int rows = min(4, q.nk - j0 - 4 * part);
  const size_t step = static_cast<size_t>(a.hk) * a.sink_tiles * kSinkRows * a.D;  // from a piece to the next
  for (int e = threadIdx.x; e < rows * a.D; e += 256) {
    const int row = 4 * part + e / a.D, d = e % a.D;
    const size_t at = (((static_cast<size_t>(slot) * a.hk + kh) * a.sink_tiles + tile) * kSinkRows + row) * a.D + d;
    float k = 0.0f, v = 0.0f;
#pragma unroll 4
    for (int p = 0; p < pieces; ++p) {
      k += a.dk_part[at + p * step];
      v += a.dv_part[at + p * step];
    }
    const size_t to = (static_cast<size_t>(q.k0 + j0 + row) * a.hk + kh) * a.D + d;
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
  hipLaunchKernelGGL(attn_sink_kernel, dim3(static_cast<unsigned>(a.nseq) * a.hk * a.sink_tiles, kSinkRows / 4), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t attn_bwd_bf16(const AttnArgs& a, hipStream_t s) {
  return a.vec == 2 ? attn_bwd_wide<2>(a, s) : attn_bwd_vec<bf16s, 2, false>(a, s);
}

hipError_t launch_attn_bwd(const AttnLaunch& l, hipStream_t s) {
  if (l.a.nseq == 0) return hipSuccess;
  if (l.a.rows_q > 0) {
    hipError_t e;
    if (l.in_dtype == kBF16) e = l.o_dtype == kBF16 ? delta_go<bf16s, bf16s>(l.a, s) : delta_go<bf16s, float>(l.a, s);
    else e = l.o_dtype == kBF16 ? delta_go<float, bf16s>(l.a, s) : delta_go<float, float>(l.a, s);
    if (e != hipSuccess) return e;
  }
  if (l.in_dtype != kBF16) return attn_bwd_f32(l.a, s);
  return l.grad_dtype == kBF16 ? attn_bwd_bf16(l.a, s) : attn_bwd_bf16_f32(l.a, s);
}

}  // namespace ssm
