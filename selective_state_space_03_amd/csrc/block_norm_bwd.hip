// Backward of the block norm (formulas in block_norm_fwd.hip) from its inputs: a and
// t are recomputed, so the forward saves nothing.  Three sums per row, each needing
// the one before: sum y^2; sum t^2 with sum dout out_w t; sum dn n (dn the gradient
// of the normalised y, n that value).
//
// Bound by memory: a row's tensors are read once, the next row's while this one is
// computed.  The weights' gradients are column sums: every workgroup keeps running
// sums in registers over the rows it walks and writes one partial row, and a second
// kernel adds the partials in a fixed order (no atomics, the same result every time).
// 8192 x 2560, every part, f32 residual (461 MB): 141 us, 3.3 TB/s, and 6 us for the
// sums; what is left is the three sums in turn at two waves per SIMD (260 us with the
// weights read among the rows' loads, which return in order; 410 us one load at a time).
// Scratch per lane, as the compiler reports it: none to 24 bytes with one access per
// lane and known types, with two (rows of 2049 to 8192 values) none for a bf16 residual
// beside a bf16 x, 56 and 64 for an f32 one, 128 and 132 for f32 throughout; 116 to 268
// with types as the call says; gate_first up to 112 bytes more.
#include "block_norm_bwd_impl.h"

namespace ssm {
namespace {

// Column sums of the partial rows: 32 columns x 8 runs of partials per workgroup,
// eight loads of a run in flight
__global__ __launch_bounds__(256) void norm_reduce_kernel(NormArgs a) {
  __shared__ float sh[8][33];
  const int which = blockIdx.z;
  float* out = which == 0 ? a.dnorm_w : which == 1 ? a.dscale : a.dout_w;
  if (!out) return;
  const int c = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  const float* src = a.part + static_cast<size_t>(which) * a.n + (col < a.n ? col : 0);
  const int step = 8 * a.w_period;
  for (int wr = blockIdx.y; wr < a.w_period; wr += gridDim.y) {
    float s = 0.0f;
    if (col < a.n) {
      for (int p = wr + run * a.w_period; p < a.parts; p += 8 * step) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int q = p + i * step;
          v[i] = src[static_cast<size_t>(q < a.parts ? q : p) * 3 * a.n];
          if (q >= a.parts) v[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s += v[i];
      }
    }
    sh[run][c] = s;
    __syncthreads();
    if (run == 0 && col < a.n) {
      float t = sh[0][c];
#pragma unroll
      for (int i = 1; i < 8; ++i) t += sh[i][c];
      out[static_cast<size_t>(wr) * a.n + col] = t;
    }
    __syncthreads();
  }
}

long gcd(long a, long b) { return b == 0 ? a : gcd(b, a % b); }

// Lanes per row: one access each up to 256, then two (2560 values: 141 us for 8192
// rows; with 320 lanes and one access 160 us, 314 us at four waves per SIMD, where it
// spills), and 512 lanes beyond 4096 values (5120 values, 4096 rows, gate and bf16:
// 189 us; four accesses of 256 lanes 577 us).  Workgroups: two per CU, as many as the
// registers allow, where there are rows for them, a whole number of turns round the
// weight rows.
NormBwdShape bwd_shape(long rows, int n, int period) {
  NormBwdShape b;
  const int chunks = (n + kChunk - 1) / kChunk;
  b.nch = chunks <= 256 ? 1 : chunks <= 1024 ? 2 : 4;
  b.tpr = chunks <= 16 ? 16 : chunks <= 32 ? 32 : chunks <= 64 ? 64 : chunks <= 128 ? 128 : chunks <= 512 ? 256 : 512;
  const long teams = norm_block(b.tpr) / b.tpr;
  long blocks = (rows + teams - 1) / teams;
  blocks = blocks < 1 ? 1 : blocks < 512 ? blocks : 512;
  const long unit = period / gcd(period, teams);
  b.blocks = (blocks + unit - 1) / unit * unit;
  return b;
}

}  // namespace

extern template hipError_t run_norm_bwd<true>(const NormArgs&, const NormBwdShape&, hipStream_t);
template hipError_t run_norm_bwd<false>(const NormArgs&, const NormBwdShape&, hipStream_t);

int norm_bwd_parts(long rows, int n, int period) {
  const NormBwdShape b = bwd_shape(rows, n, period);
  return static_cast<int>(period == 1 ? b.blocks : b.blocks * (norm_block(b.tpr) / b.tpr));
}

// (without rows the kernels still run: the weight gradients are then zeros)
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s) {
  const NormBwdShape b = bwd_shape(a.rows, a.n, a.w_period);
  const hipError_t e = a.gate_first ? run_norm_bwd<true>(a, b, s) : run_norm_bwd<false>(a, b, s);
  if (e != hipSuccess || (!a.dnorm_w && !a.dscale && !a.dout_w)) return e;
  const int wrows = a.w_period < 65535 ? a.w_period : 65535;  // (the most workgroups along y)
  hipLaunchKernelGGL(norm_reduce_kernel, dim3((a.n + 31) / 32, wrows, 3), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace ssm
