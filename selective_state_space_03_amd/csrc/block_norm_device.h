// Device helpers of the block norm's kernels (block_norm_fwd.hip, block_norm_bwd.hip):
// rows in accesses of 8 values per lane, their sums across the lanes of a row, and
// the choice of a kernel by the tensors' types.
#pragma once
#include "delta.h"
#include "ssm_device.h"

namespace ssm {
namespace {

constexpr int kChunk = 8;

// 8 values from element i0 of a row of n, as loaded (vec: elements per aligned
// access).  Types and alignment are uniform branches; widening is kept apart from
// loading, so that a row's loads are all in flight before the first is waited for.
struct Raw {
  uint4 a, b;
};
__device__ __forceinline__ Raw raw8(const void* base, size_t row, int i0, int n, int dtype, int vec) {
  Raw r;
  r.a = r.b = make_uint4(0u, 0u, 0u, 0u);
  if (dtype == kBF16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + row + i0;
    if (vec == 8) {
      if (i0 < n) r.a = *reinterpret_cast<const uint4*>(p);
    } else if (vec == 4) {
      uint2 x = make_uint2(0u, 0u), y = x;
      if (i0 < n) x = *reinterpret_cast<const uint2*>(p);
      if (i0 + 4 < n) y = *reinterpret_cast<const uint2*>(p + 4);
      r.a = make_uint4(x.x, x.y, y.x, y.y);
    } else {
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = 0u;
        if (i0 + i < n) v[i] = p[i];
      }
      r.a = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
  } else {
    const float* p = static_cast<const float*>(base) + row + i0;
    if (vec >= 4) {
      if (i0 < n) r.a = *reinterpret_cast<const uint4*>(p);
      if (i0 + 4 < n) r.b = *reinterpret_cast<const uint4*>(p + 4);
    } else {
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = 0u;
        if (i0 + i < n) v[i] = __float_as_uint(p[i]);
      }
      r.a = make_uint4(v[0], v[1], v[2], v[3]);
      r.b = make_uint4(v[4], v[5], v[6], v[7]);
    }
  }
  return r;
}
__device__ __forceinline__ void widen(const Raw& r, int dtype, float (&v)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w}, x[4] = {r.b.x, r.b.y, r.b.z, r.b.w};
  const bool bf = dtype == kBF16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = __uint_as_float(bf ? (i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16) : w[i]);
    v[4 + i] = __uint_as_float(bf ? (i & 1 ? w[2 + (i >> 1)] & 0xffff0000u : w[2 + (i >> 1)] << 16) : x[i]);
  }
}
__device__ __forceinline__ void get8(const void* base, size_t row, int i0, int n, int dtype, int vec, float (&v)[8]) {
  widen(raw8(base, row, i0, n, dtype, vec), dtype, v);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ void put8(void* base, size_t row, int i0, int n, int dtype, int vec, const float (&v)[8]) {
  if (dtype == kBF16) {
    uint16_t* p = static_cast<uint16_t*>(base) + row + i0;
    const uint32_t w[4] = {pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])};
    if (vec == 8) {
      if (i0 < n) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if (vec == 4) {
      if (i0 < n) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
      if (i0 + 4 < n) *reinterpret_cast<uint2*>(p + 4) = make_uint2(w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i0 + i < n) p[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    }
  } else {
    float* p = static_cast<float*>(base) + row + i0;
    if (vec >= 4) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (i0 + 4 * h < n)
          *reinterpret_cast<float4*>(p + 4 * h) = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i0 + i < n) p[i] = v[i];
    }
  }
}

// Sums of NS values over the TPR lanes of a row.  sh: per row of the workgroup two
// copies of NS x waves floats used in turn, so a copy is rewritten only after a
// barrier has passed.
template <int TPR, int NS>
__device__ __forceinline__ void row_sums(float (&x)[NS], float* sh, int& turn) {
#pragma unroll
  for (int o = 1; o < (TPR < 64 ? TPR : 64); o <<= 1)
#pragma unroll
    for (int k = 0; k < NS; ++k) x[k] += __shfl_xor(x[k], o);
  if (TPR > 64) {
    constexpr int W = TPR / 64;
    float* s = sh + (threadIdx.x / TPR) * 4 * W + (turn & 1) * 2 * W;
    ++turn;
    const int w = (threadIdx.x % TPR) >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < NS; ++k) s[k * W + w] = x[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      float t = s[k * W];
#pragma unroll
      for (int i = 1; i < W; ++i) t += s[k * W + i];
      x[k] = t;
    }
  }
}

__device__ __forceinline__ float sigmoid(float z) { return rcp_fast(1.0f + exp2_fast(-z * kLog2e)); }

// The type combinations that have kernels of their own (same: the other tensors
// have the types of x and the residual), or -1
int known_types(const NormArgs& a, bool same) {
  if (a.vec != 8 || !same) return -1;
  const bool stream = a.res || a.res_out || a.dres || a.dresidual;  // a residual stream, in or out
  const int rd = stream ? a.res_dtype : a.x_dtype;
  if (a.x_dtype == kBF16) return rd == kBF16 ? 2 : 1;
  return rd == kF32 ? 0 : -1;
}

}  // namespace
}  // namespace ssm
