// The norms before and after a block with its gate and residual scale, in one pass
// over each row:
//   y = x (SiLU(z) first, with gate_first);  a = norm(y) norm_w;  (a SiLU(z), without)
//   t = residual + scale a;   out = norm(t) out_w;   norm(r) = r / sqrt(mean(r^2) + eps)
// every part optional; a grouped norm is the same with each group a row.
//
// Bound by memory: each row is read once into registers (8 values per lane and
// access, all of a row's loads in flight before the first is widened), its sums
// taken across the TPR lanes that share it, and the results written once; t is
// normalised from its 32-bit value, not from the residual as stored.
// 16383 x 2560 with an f32 residual (587 MB): 124 us, 4.7 TB/s, with 256 lanes to a
// row (135 us with a wave to a row and no barrier); 64 rows of it 6.1 us (10.2).  The
// mixer's 8192 x 32 groups of 128 (201 MB), 16 lanes to a group: 38 us, 5.3 TB/s.
#include "block_norm_device.h"

namespace ssm {
namespace {

// XD, RD: the dtypes of x, z and out, and of the residual, where every row takes
// 16-byte accesses; -1: types and accesses as a says (then a lane holds twice the
// registers for its raw values and every pointer's alternatives)
template <int TPR, int NCH, int XD, int RD>
__global__ __launch_bounds__(256) void norm_fwd_kernel(NormArgs a, long first) {
  __shared__ float sh[16];
  int turn = 0;
  constexpr bool kKnown = XD >= 0;
  const int vec = kKnown ? 8 : a.vec, xd = kKnown ? XD : a.x_dtype, rd = kKnown ? RD : a.res_dtype;
  const int od = kKnown ? XD : a.out_dtype;
  constexpr int RPB = 256 / TPR;  // rows per workgroup
  const int l = threadIdx.x % TPR;
  const long row_raw = first + static_cast<long>(blockIdx.x) * RPB + threadIdx.x / TPR;
  const bool act = row_raw < a.rows;  // (whole teams; with TPR 256 every row is there)
  const long row = act ? row_raw : a.rows - 1;
  const long call_row = row / a.groups;
  const int grp = static_cast<int>(row - call_row * a.groups);
  const size_t xo = call_row * a.x_stride + static_cast<size_t>(grp) * a.n;
  const size_t zo = call_row * a.z_stride + static_cast<size_t>(grp) * a.n;
  const size_t dense = static_cast<size_t>(row) * a.n;
  const size_t wo = static_cast<size_t>(row % a.w_period) * a.n;

  Raw rx[NCH], rz[NCH], rr[NCH];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int i0 = (l + c * TPR) * kChunk;
    rx[c] = raw8(a.x, xo, i0, a.n, xd, vec);
    if (a.z) rz[c] = raw8(a.z, zo, i0, a.n, xd, vec);
    if (a.res) rr[c] = raw8(a.res, dense, i0, a.n, rd, vec);
  }
  float y[NCH][8], g[NCH][8], t[NCH][8];
  float sum[1] = {0.0f};
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    widen(rx[c], xd, y[c]);
    if (a.z) widen(rz[c], xd, g[c]);
    if (a.res) widen(rr[c], rd, t[c]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (a.z) {
        g[c][i] *= sigmoid(g[c][i]);
        if (a.gate_first) y[c][i] *= g[c][i];
      }
      sum[0] = fmaf(y[c][i], y[c][i], sum[0]);
    }
  }
  float inv = 1.0f;
  if (a.norm_w) {
    row_sums<TPR, 1>(sum, sh, turn);
    inv = 1.0f / sqrtf(sum[0] / static_cast<float>(a.n) + a.eps);
  }
  sum[0] = 0.0f;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int i0 = (l + c * TPR) * kChunk;
    float w[8], sc[8];
    if (a.norm_w) get8(a.norm_w, wo, i0, a.n, kF32, vec, w);
    if (a.scale) get8(a.scale, 0, i0, a.n, kF32, vec, sc);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = y[c][i];
      if (a.norm_w) v *= inv * w[i];
      if (a.z && !a.gate_first) v *= g[c][i];
      if (a.scale) v *= sc[i];
      if (a.res) v += t[c][i];
      t[c][i] = v;
      sum[0] = fmaf(v, v, sum[0]);
    }
    if (act && a.res_out) put8(a.res_out, dense, i0, a.n, rd, vec, t[c]);
  }
  if (!a.out) return;
  if (a.out_w) {
    row_sums<TPR, 1>(sum, sh, turn);
    inv = 1.0f / sqrtf(sum[0] / static_cast<float>(a.n) + a.eps);
  }
  if (!act) return;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int i0 = (l + c * TPR) * kChunk;
    if (a.out_w) {
      float w[8];
      get8(a.out_w, 0, i0, a.n, kF32, vec, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[c][i] *= inv * w[i];
    }
    put8(a.out, dense, i0, a.n, od, vec, t[c]);
  }
}

// A launch holds fewer than 2^32 threads: calls of more rows take several.
constexpr long kMostBlocks = 1L << 23;

template <int TPR, int NCH>
hipError_t fwd(const NormArgs& a, hipStream_t s) {
  constexpr int RPB = 256 / TPR;
  return timed_launch(s, [&] {
    for (long first = 0; first < a.rows; first += kMostBlocks * RPB) {
      const long blocks = (a.rows - first + RPB - 1) / RPB;
      const dim3 grid(static_cast<unsigned>(blocks < kMostBlocks ? blocks : kMostBlocks));
      switch (known_types(a, !a.out || a.out_dtype == a.x_dtype)) {
        case 0: hipLaunchKernelGGL((norm_fwd_kernel<TPR, NCH, kF32, kF32>), grid, dim3(256), 0, s, a, first); break;
        case 1: hipLaunchKernelGGL((norm_fwd_kernel<TPR, NCH, kBF16, kF32>), grid, dim3(256), 0, s, a, first); break;
        case 2: hipLaunchKernelGGL((norm_fwd_kernel<TPR, NCH, kBF16, kBF16>), grid, dim3(256), 0, s, a, first); break;
        default: hipLaunchKernelGGL((norm_fwd_kernel<TPR, NCH, -1, -1>), grid, dim3(256), 0, s, a, first);
      }
    }
  });
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const int chunks = (a.n + kChunk - 1) / kChunk;
  if (chunks <= 16) return fwd<16, 1>(a, s);
  if (chunks <= 32) return fwd<32, 1>(a, s);
  if (chunks <= 64) return fwd<64, 1>(a, s);
  if (chunks <= 128) return fwd<128, 1>(a, s);
  if (chunks <= 256) return fwd<256, 1>(a, s);
  if (chunks <= 512) return fwd<256, 2>(a, s);
  if (chunks <= 1024) return fwd<256, 4>(a, s);
  return fwd<256, 8>(a, s);
}

}  // namespace ssm
