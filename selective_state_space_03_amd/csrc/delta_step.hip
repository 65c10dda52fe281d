// One token of the gated delta rule, state in place, for gfx950.
//
// Row v of a head's state (K values) takes the step by itself:
//   s <- e^g s;  u = beta (v - s.k);  s <- s + u k;  o = scale s.q
// so the step reads and writes the whole state once and nothing else of size:
// it is bound by HBM bandwidth.  K / 8 lanes (8 or 16) share a row, 8 values
// each in two 16-byte non-temporal accesses; the products s.k and s.q of the
// old state and k.q are summed across those lanes together, which gives the new
// state's product as e^g s.q + u k.q.  A lane holds its k and q values for
// several rows of the head (kRows), so their norms are summed once for them.
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

template <typename IN, int LPR, int ROWS>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaStepArgs a, unsigned groups_per_head, unsigned groups) {
  const unsigned gi = blockIdx.x * (256u / LPR) + threadIdx.x / LPR;
  if (gi >= groups) return;  // whole lane groups leave together
  const unsigned bh = gi / groups_per_head;
  const int v0 = static_cast<int>(gi - bh * groups_per_head) * ROWS;
  const unsigned b = bh / a.h, head = bh - b * a.h, kh = head / (a.h / a.hk);
  const int d = (threadIdx.x % LPR) * 8;

  float s[ROWS][8];
  float* const base = a.state + static_cast<size_t>(bh) * a.V * a.K;
#pragma unroll
  for (int x = 0; x < ROWS; ++x) {
    const float* p = base + static_cast<size_t>(min(v0 + x, a.V - 1)) * a.K + d;
    if (a.vec) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 f = d < a.K ? load_stream(reinterpret_cast<const float4*>(p) + h) : make_float4(0.f, 0.f, 0.f, 0.f);
        s[x][4 * h] = f.x; s[x][4 * h + 1] = f.y; s[x][4 * h + 2] = f.z; s[x][4 * h + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[x][i] = d + i < a.K ? p[i] : 0.0f;
    }
  }
  float k[8], q[8];
  load8<IN>(static_cast<const IN*>(a.k) + b * a.k_stride + static_cast<long>(kh) * a.K, d, a.K, a.vec, k);
  load8<IN>(static_cast<const IN*>(a.q) + b * a.q_stride + static_cast<long>(kh) * a.K, d, a.K, a.vec, q);
  const float alpha = exp2_fast(a.g[bh] * kLog2e), beta = a.beta[bh];
  float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    kk = fmaf(k[i], k[i], kk);
    qq = fmaf(q[i], q[i], qq);
    kq = fmaf(k[i], q[i], kq);
  }
  float rk = 1.0f, rq = a.scale;
  kq = row_sum<LPR>(kq);
  if (a.qk_norm) {
    rk = 1.0f / sqrtf(row_sum<LPR>(kk) + a.eps);
    rq *= 1.0f / sqrtf(row_sum<LPR>(qq) + a.eps);
  }
#pragma unroll
  for (int x = 0; x < ROWS; ++x) {
    float sk = 0.0f, sq = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sk = fmaf(s[x][i], k[i], sk);
      sq = fmaf(s[x][i], q[i], sq);
    }
    sk = row_sum<LPR>(sk);
    sq = row_sum<LPR>(sq);
    const int v = v0 + x;
    if (v >= a.V) continue;
    const float vv = to_f32(static_cast<const IN*>(a.v)[b * a.v_stride + static_cast<long>(head) * a.V + v]);
    const float u = beta * (vv - alpha * rk * sk);
    const float uk = u * rk;
    float* p = base + static_cast<size_t>(v) * a.K + d;
    float ns[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) ns[i] = fmaf(uk, k[i], alpha * s[x][i]);
    if (a.vec) {
      if (d < a.K) {
        store_stream(reinterpret_cast<float4*>(p), make_float4(ns[0], ns[1], ns[2], ns[3]));
        store_stream(reinterpret_cast<float4*>(p) + 1, make_float4(ns[4], ns[5], ns[6], ns[7]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (d + i < a.K) p[i] = ns[i];
    }
    if (d == 0) {
      const float o = rq * fmaf(alpha, sq, uk * kq);
      const size_t at = static_cast<size_t>(bh) * a.V + v;
      if (a.o_bf16) st<bf16s>(a.o, at, o);
      else st<float>(a.o, at, o);
    }
  }
}

template <typename IN, int LPR, int ROWS>
hipError_t go(const DeltaStepArgs& a, hipStream_t s) {
  const unsigned per_head = (a.V + ROWS - 1) / ROWS;
  const unsigned groups = static_cast<unsigned>(a.batch) * a.h * per_head;
  constexpr unsigned per_block = 256 / LPR;
  return timed_launch(s, [&] {
    hipLaunchKernelGGL((delta_step_kernel<IN, LPR, ROWS>), dim3((groups + per_block - 1) / per_block), dim3(256), 0, s, a,
                       per_head, groups);
  });
}

template <typename IN, int LPR>
hipError_t pick_rows(const DeltaStepArgs& a, hipStream_t s) {
  // four rows per lane group once that still leaves every CU two workgroups
  const long rows = static_cast<long>(a.batch) * a.h * a.V;
  return rows * LPR / 4 >= 2L * 256 * 256 ? go<IN, LPR, 4>(a, s) : go<IN, LPR, 1>(a, s);
}

template <typename IN>
hipError_t pick(const DeltaStepArgs& a, hipStream_t s) {
  return a.K <= 64 ? pick_rows<IN, 8>(a, s) : pick_rows<IN, 16>(a, s);
}

}  // namespace

hipError_t launch_delta_step(const DeltaStepArgs& a, int in_dtype, hipStream_t s) {
  if (a.batch == 0) return hipSuccess;
  return in_dtype == kBF16 ? pick<bf16s>(a, s) : pick<float>(a, s);
}

}  // namespace ssm
