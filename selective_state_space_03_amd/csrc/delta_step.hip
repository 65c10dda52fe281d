// One token of the gated delta rule, state in place, for gfx950.
//
// Row v of a head's state (K values) takes the step by itself:
//   s <- e^g s;  u = beta (v - s.k);  s <- s + u k;  o = scale s.q
// so the step reads and writes the whole state once and nothing else of size:
// it is bound by HBM bandwidth.  K / 8 lanes (8 or 16) share a row, 8 values
// each in two 16-byte non-temporal accesses; the products s.k and s.q of the
// old state and k.q are summed across those lanes together, which gives the new
// state's product as e^g s.q + u k.q.
// 64 sequences, 80 heads of 96 x 64 (254 MB): 49 us, 5.15 TB/s, a copy's rate; four
// rows per lane group (one sum of the norms for them) 52.6 us.  One sequence, 32
// heads of 128 x 128: 4.2 us (5.4 with four rows).
#include "delta.h"
#include "ssm_device.h"

namespace ssm {
namespace {

template <typename IN>
__device__ __forceinline__ void load8(const IN* p, int d, int K, bool vec, float (&v)[8]) {
  if (vec) {
    if (sizeof(IN) == 2) {
      const uint4 r = load16_if(p + d, d < K);
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 r = load16_if(p + d + 4 * h, d < K);
        v[4 * h] = __uint_as_float(r.x); v[4 * h + 1] = __uint_as_float(r.y);
        v[4 * h + 2] = __uint_as_float(r.z); v[4 * h + 3] = __uint_as_float(r.w);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = d + i < K ? to_f32(p[d + i]) : 0.0f;
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) x += __shfl_xor(x, o);
  return x;
}

template <typename IN, int LPR>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaStepArgs a, unsigned rows) {
  const unsigned row = blockIdx.x * (256u / LPR) + threadIdx.x / LPR;  // (sequence, head, v)
  if (row >= rows) return;  // whole lane groups leave together
  const unsigned bh = row / a.V, v = row - bh * a.V;
  const unsigned b = bh / a.h, head = bh - b * a.h, kh = head / (a.h / a.hk);
  const int d = (threadIdx.x % LPR) * 8;

  float s[8], k[8], q[8];
  float* const p = a.state + static_cast<size_t>(row) * a.K + d;
  if (a.vec) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 f = d < a.K ? load_stream(reinterpret_cast<const float4*>(p) + h) : make_float4(0.f, 0.f, 0.f, 0.f);
      s[4 * h] = f.x; s[4 * h + 1] = f.y; s[4 * h + 2] = f.z; s[4 * h + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = d + i < a.K ? p[i] : 0.0f;
  }
  load8<IN>(static_cast<const IN*>(a.k) + b * a.k_stride + static_cast<long>(kh) * a.K, d, a.K, a.vec, k);
  load8<IN>(static_cast<const IN*>(a.q) + b * a.q_stride + static_cast<long>(kh) * a.K, d, a.K, a.vec, q);
  const float alpha = exp2_fast(a.g[bh] * kLog2e), beta = a.beta[bh];
  const float vv = to_f32(static_cast<const IN*>(a.v)[b * a.v_stride + static_cast<long>(head) * a.V + v]);
  float kk = 0.0f, qq = 0.0f, kq = 0.0f, sk = 0.0f, sq = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    kk = fmaf(k[i], k[i], kk);
    qq = fmaf(q[i], q[i], qq);
    kq = fmaf(k[i], q[i], kq);
    sk = fmaf(s[i], k[i], sk);
    sq = fmaf(s[i], q[i], sq);
  }
  float rk = 1.0f, rq = a.scale;
  if (a.qk_norm) {
    rk = 1.0f / sqrtf(row_sum<LPR>(kk) + a.eps);
    rq *= 1.0f / sqrtf(row_sum<LPR>(qq) + a.eps);
  }
  kq = row_sum<LPR>(kq);
  sk = row_sum<LPR>(sk);
  sq = row_sum<LPR>(sq);
  const float uk = beta * (vv - alpha * rk * sk) * rk;
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = fmaf(uk, k[i], alpha * s[i]);
  if (a.vec) {
    if (d < a.K) {
      store_stream(reinterpret_cast<float4*>(p), make_float4(s[0], s[1], s[2], s[3]));
      store_stream(reinterpret_cast<float4*>(p) + 1, make_float4(s[4], s[5], s[6], s[7]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (d + i < a.K) p[i] = s[i];
  }
  if (d == 0) {
    const float o = rq * fmaf(alpha, sq, uk * kq);
    if (a.o_bf16) st<bf16s>(a.o, row, o);
    else st<float>(a.o, row, o);
  }
}

template <typename IN, int LPR>
hipError_t go(const DeltaStepArgs& a, hipStream_t s) {
  const unsigned rows = static_cast<unsigned>(a.batch) * a.h * a.V;
  constexpr unsigned per_block = 256 / LPR;
  return timed_launch(s, [&] {
    hipLaunchKernelGGL((delta_step_kernel<IN, LPR>), dim3((rows + per_block - 1) / per_block), dim3(256), 0, s, a, rows);
  });
}

template <typename IN>
hipError_t pick(const DeltaStepArgs& a, hipStream_t s) {
  return a.K <= 64 ? go<IN, 8>(a, s) : go<IN, 16>(a, s);
}

}  // namespace

hipError_t launch_delta_step(const DeltaStepArgs& a, int in_dtype, hipStream_t s) {
  if (a.batch == 0) return hipSuccess;
  return in_dtype == kBF16 ? pick<bf16s>(a, s) : pick<float>(a, s);
}

}  // namespace ssm
