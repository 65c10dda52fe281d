// The norms before and after a block with its gate and residual scale, forward
// and backward, in one pass over each row.
//
//   y = x (SiLU(z) first, with gate_first);  a = norm(y) norm_w;  (a SiLU(z), without)
//   t = residual + scale a;   out = norm(t) out_w;   norm(r) = r / sqrt(mean(r^2) + eps)
// every part optional; a grouped norm is the same with each group a row.
//
// Bound by memory: each row is read once into registers (kChunk = 8 values per
// lane and access), its sums taken across the TPR lanes that share it, and the
// results written once; t is normalised from its 32-bit value, not from the
// residual as stored.  The backward pass recomputes a and t from the inputs (it
// needs no saved statistics) and takes the three sums of its formulas (sum y^2;
// sum t^2 with sum dout out_w t; sum dn n) in that order.  Its weight gradients
// are column sums: every workgroup keeps running sums in registers over the rows
// it walks and writes one partial row, and a second kernel adds the partials in
// a fixed order (no atomics, the same result every time).
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

// XD, RD: the dtypes of x, z and out, and of the residual, where every row takes
// 16-byte accesses; -1: types and accesses as a says (then a lane holds twice the
// registers for its raw values and every pointer's alternatives)
template <int TPR, int NCH, int XD, int RD>
__global__ __launch_bounds__(256) void norm_fwd_kernel(NormArgs a) {
  __shared__ float sh[16];
  int turn = 0;
  constexpr bool kKnown = XD >= 0;
  const int vec = kKnown ? 8 : a.vec, xd = kKnown ? XD : a.x_dtype, rd = kKnown ? RD : a.res_dtype;
  const int od = kKnown ? XD : a.out_dtype;
  constexpr int RPB = 256 / TPR;  // rows per workgroup
  const int l = threadIdx.x % TPR;
  const long row_raw = static_cast<long>(blockIdx.x) * RPB + threadIdx.x / TPR;
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

// GF: gate_first.  Parts that are missing cost no branch per element: an absent weight
// is held as ones, an absent gate as z sigmoid = 1.
template <int TPR, int NCH, int XD, int RD, bool GF>
__global__ __launch_bounds__(256, NCH == 1 ? 3 : NCH == 2 ? 2 : 1) void norm_bwd_kernel(NormArgs a) {
  constexpr int TEAMS = 256 / TPR;
  __shared__ float sh[16];
  int turn = 0;
  constexpr bool kKnown = XD >= 0;
  const int vec = kKnown ? 8 : a.vec, xd = kKnown ? XD : a.x_dtype, rd = kKnown ? RD : a.res_dtype;
  const int dod = kKnown ? XD : a.dout_dtype, drd = kKnown ? RD : a.dres_dtype, gd = kKnown ? XD : a.grad_dtype;
  const int l = threadIdx.x % TPR;
  const long team = static_cast<long>(blockIdx.x) * TEAMS + threadIdx.x / TPR;
  const long teams = static_cast<long>(gridDim.x) * TEAMS;  // a multiple of w_period
  const size_t wo = static_cast<size_t>(team % a.w_period) * a.n;
  const float rn = 1.0f / static_cast<float>(a.n);

  // The weights' columns are the same in every row: in registers with one access per
  // lane, in LDS with two.  Loads among the rows' own would come back after them (loads
  // return in order), which would undo the reading ahead below.
  constexpr bool kRegs = NCH == 1, kLds = !kRegs && NCH == 2;
  __shared__ __align__(16) float wsh[3][kLds ? TPR * NCH * kChunk : 4];
  float wreg[3][8];
  const float* const wsrc[3] = {a.norm_w ? a.norm_w + wo : nullptr, a.scale, a.out_w};
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (kRegs || kLds) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int i0 = (l + c * TPR) * kChunk;
        if (wsrc[k]) {
          get8(wsrc[k], 0, i0, a.n, kF32, vec, wreg[k]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) wreg[k][i] = 1.0f;
        }
        if (kLds) {
#pragma unroll
          for (int i = 0; i < 8; ++i) wsh[k][i0 + i] = wreg[k][i];  // (read again by this lane only)
        }
      }
    }
  auto weight = [&](int k, int c, float (&v)[8]) {
    const int i0 = (l + c * TPR) * kChunk;
    if (kRegs) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = wreg[k][i];
    } else if (kLds) {
      const float4 x = *reinterpret_cast<const float4*>(&wsh[k][i0]), y = *reinterpret_cast<const float4*>(&wsh[k][i0 + 4]);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
      v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    } else if (wsrc[k]) {
      get8(wsrc[k], 0, i0, a.n, kF32, vec, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 1.0f;
    }
  };

  float aw[NCH][8], as[NCH][8], ao[NCH][8];  // this team's column sums
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) aw[c][i] = as[c][i] = ao[c][i] = 0.0f;

  // A row's values as loaded; each is asked for again, for the team's next row, right
  // after its last use, so the loads have the rest of the row before to arrive.
  Raw rx[NCH], rz[NCH], rr[NCH], ro[NCH], re[NCH];
  struct At {
    size_t x, z, dense;
    bool act;
  };
  // every team of a workgroup walks the same number of rows (sums cross the
  // workgroup); a row past the end is computed from row 0 and counts for nothing
  auto at_row = [&](long base) {
    const long row_raw = base + threadIdx.x / TPR;
    At p;
    p.act = row_raw < a.rows;
    const long row = p.act ? row_raw : 0;
    const long call_row = row / a.groups;
    const size_t grp = static_cast<size_t>(row - call_row * a.groups) * a.n;
    p.x = call_row * a.x_stride + grp;
    p.z = call_row * a.z_stride + grp;
    p.dense = static_cast<size_t>(row) * a.n;
    return p;
  };
  auto load_in = [&](const At& p) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int i0 = (l + c * TPR) * kChunk;
      rx[c] = raw8(a.x, p.x, i0, a.n, xd, vec);
      if (a.z) rz[c] = raw8(a.z, p.z, i0, a.n, xd, vec);
    }
  };
  auto load_out = [&](const At& p) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int i0 = (l + c * TPR) * kChunk;
      if (a.res && a.out_w) rr[c] = raw8(a.res, p.dense, i0, a.n, rd, vec);
      if (a.dout) ro[c] = raw8(a.dout, p.dense, i0, a.n, dod, vec);
    }
  };
  auto load_res = [&](const At& p) {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
      if (a.dres) re[c] = raw8(a.dres, p.dense, (l + c * TPR) * kChunk, a.n, drd, vec);
  };
  const long first = static_cast<long>(blockIdx.x) * TEAMS;
  At cur = at_row(first);
  if (first < a.rows) {
    load_in(cur);
    load_out(cur);
    load_res(cur);
  }
  for (long base = first; base < a.rows; base += teams) {
    const bool act = TEAMS == 1 || cur.act;
    const size_t dense = cur.dense;
    cur = at_row(min(base + teams, a.rows));  // (the row after the last is none: row 0 again)

    // g: the gate z sigmoid(z), h: its derivative sigmoid(z) (1 + z (1 - sigmoid(z)))
    float x[NCH][8], g[NCH][8], h[NCH][8], d[NCH][8];
    float sum[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      widen(rx[c], xd, x[c]);
      if (a.z) {
        float z[8];
        widen(rz[c], xd, z);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float sg = sigmoid(z[i]);
          g[c][i] = z[i] * sg;
          h[c][i] = sg * fmaf(z[i], 1.0f - sg, 1.0f);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[c][i] = 1.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = GF ? x[c][i] * g[c][i] : x[c][i];
        sum[0] = fmaf(y, y, sum[0]);
      }
    }
    load_in(cur);
    float inv = 1.0f;
    if (a.norm_w) {
      row_sums<TPR, 1>(sum, sh, turn);
      inv = 1.0f / sqrtf(sum[0] * rn + a.eps);
    }
    // with an output norm: t and its two sums, then the gradient of t
    if (a.out_w && a.dout) {
      float sum2[2] = {0.0f, 0.0f};
      float t[NCH][8];
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        float w[8], sc[8], ow[8], dd[8];
        weight(0, c, w);
        weight(1, c, sc);
        weight(2, c, ow);
        if (a.res) {
          widen(rr[c], rd, t[c]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) t[c][i] = 0.0f;
        }
        widen(ro[c], dod, dd);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          t[c][i] = fmaf(x[c][i] * inv * w[i] * g[c][i], sc[i], t[c][i]);
          sum2[0] = fmaf(t[c][i], t[c][i], sum2[0]);
          sum2[1] = fmaf(dd[i] * ow[i], t[c][i], sum2[1]);
        }
      }
      row_sums<TPR, 2>(sum2, sh, turn);
      const float oi = 1.0f / sqrtf(sum2[0] * rn + a.eps);
      const float k = sum2[1] * rn * oi * oi * oi;
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        float ow[8], dd[8];
        weight(2, c, ow);
        widen(ro[c], dod, dd);
        if (act) {
#pragma unroll
          for (int i = 0; i < 8; ++i) ao[c][i] = fmaf(dd[i] * t[c][i], oi, ao[c][i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float e = dd[i] * ow[i] * oi;
          // (with one value the difference cancels: what is left is the epsilon's part)
          d[c][i] = TPR == 16 && a.n == 1 ? e * (a.eps * oi * oi) : fmaf(-k, t[c][i], e);
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        if (a.dout) {
          widen(ro[c], dod, d[c]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) d[c][i] = 0.0f;
        }
      }
    }
    load_out(cur);
    sum[0] = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int i0 = (l + c * TPR) * kChunk;
      if (a.dres) {
        float e[8];
        widen(re[c], drd, e);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[c][i] += e[i];
      }
      if (act && a.dresidual) put8(a.dresidual, dense, i0, a.n, rd, vec, d[c]);
      float w[8], sc[8];
      weight(0, c, w);
      weight(1, c, sc);
      if (act) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float n = GF ? x[c][i] * g[c][i] * inv : x[c][i] * inv;  // normalised, before its weight
          as[c][i] = fmaf(d[c][i], GF ? n * w[i] : n * w[i] * g[c][i], as[c][i]);
          aw[c][i] = fmaf(d[c][i] * sc[i], GF ? n : n * g[c][i], aw[c][i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[c][i] *= sc[i];
        sum[0] = fmaf(d[c][i] * w[i], x[c][i] * g[c][i] * inv, sum[0]);
      }
    }
    load_res(cur);
    float k = 0.0f;
    if (a.norm_w) {
      row_sums<TPR, 1>(sum, sh, turn);
      k = sum[0] * rn;
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int i0 = (l + c * TPR) * kChunk;
      float w[8], dz[8];
      weight(0, c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = GF ? x[c][i] * g[c][i] * inv : x[c][i] * inv;
        const float e = GF ? d[c][i] * w[i] : d[c][i] * w[i] * g[c][i];
        // (one value: as above)
        const float dy = TPR == 16 && a.norm_w && a.n == 1 ? inv * inv * inv * a.eps * e : inv * fmaf(-n, k, e);
        dz[i] = (GF ? dy * x[c][i] : d[c][i] * w[i] * n) * h[c][i];
        x[c][i] = GF ? dy * g[c][i] : dy;
      }
      if (act && a.dx) put8(a.dx, dense, i0, a.n, gd, vec, x[c]);
      if (act && a.dz) put8(a.dz, dense, i0, a.n, gd, vec, dz);
    }
  }

  // partial rows: one per workgroup where its teams share a weight row, else one per team
  const size_t cols = a.n;
  if (a.w_period == 1 && TEAMS > 1) {
    constexpr int kRow = TPR * NCH * 8, SLOTS = TPR <= 64 ? 4 : TEAMS;
    __shared__ float acc[SLOTS][kRow];
    const int slot = TPR <= 64 ? threadIdx.x >> 6 : threadIdx.x / TPR;
    for (int which = 0; which < 3; ++which) {
      float (*v)[8] = which == 0 ? aw : which == 1 ? as : ao;
      const bool need = which == 0 ? a.dnorm_w != nullptr : which == 1 ? a.dscale != nullptr : a.dout_w != nullptr;
      if (!need) continue;
#pragma unroll
      for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float s = v[c][i];
#pragma unroll
          for (int o = TPR; o < 64; o <<= 1) s += __shfl_xor(s, o);
          if ((threadIdx.x & 63) < TPR) acc[slot][(l + c * TPR) * 8 + i] = s;
        }
      __syncthreads();
      for (int i = threadIdx.x; i < a.n; i += 256) {
        float s = acc[0][i];
#pragma unroll
        for (int x = 1; x < SLOTS; ++x) s += acc[x][i];
        a.part[(static_cast<size_t>(blockIdx.x) * 3 + which) * cols + i] = s;
      }
      __syncthreads();
    }
  } else {
    float* p = a.part + static_cast<size_t>(team) * 3 * cols;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int i0 = (l + c * TPR) * kChunk;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i0 + i < a.n) {
          if (a.dnorm_w) p[i0 + i] = aw[c][i];
          if (a.dscale) p[cols + i0 + i] = as[c][i];
          if (a.dout_w) p[2 * cols + i0 + i] = ao[c][i];
        }
    }
  }
}

// Column sums of the partial rows: 32 columns x 8 runs of partials per workgroup,
// eight loads of a run in flight
__global__ __launch_bounds__(256) void norm_reduce_kernel(NormArgs a) {
  __shared__ float sh[8][33];
  const int which = blockIdx.z, wr = blockIdx.y;
  float* out = which == 0 ? a.dnorm_w : which == 1 ? a.dscale : a.dout_w;
  if (!out) return;
  const int c = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  float s = 0.0f;
  if (col < a.n) {
    const float* src = a.part + static_cast<size_t>(which) * a.n + col;
    const int step = 8 * a.w_period;
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
}

// The type combinations that have kernels of their own (same: the other tensors
// have the types of x and the residual), or -1
int known_types(const NormArgs& a, bool same) {
  if (a.vec != 8 || !same) return -1;
  const int rd = a.res || a.dres ? a.res_dtype : a.x_dtype;
  if (a.x_dtype == kBF16) return rd == kBF16 ? 2 : 1;
  return rd == kF32 ? 0 : -1;
}

template <int TPR, int NCH>
hipError_t fwd(const NormArgs& a, hipStream_t s) {
  constexpr int RPB = 256 / TPR;
  return timed_launch(s, [&] {
    const dim3 grid(static_cast<unsigned>((a.rows + RPB - 1) / RPB));
    switch (known_types(a, !a.out || a.out_dtype == a.x_dtype)) {
      case 0: hipLaunchKernelGGL((norm_fwd_kernel<TPR, NCH, kF32, kF32>), grid, dim3(256), 0, s, a); break;
      case 1: hipLaunchKernelGGL((norm_fwd_kernel<TPR, NCH, kBF16, kF32>), grid, dim3(256), 0, s, a); break;
      case 2: hipLaunchKernelGGL((norm_fwd_kernel<TPR, NCH, kBF16, kBF16>), grid, dim3(256), 0, s, a); break;
      default: hipLaunchKernelGGL((norm_fwd_kernel<TPR, NCH, -1, -1>), grid, dim3(256), 0, s, a);
    }
  });
}

long gcd(long a, long b) { return b == 0 ? a : gcd(b, a % b); }

struct BwdShape {
  int tpr, nch;
  long blocks;
};

// Lanes per row of the backward kernel, and its workgroups: two per CU (as many
// as its registers allow) where there are rows for them, a whole number of turns round the weight rows.
BwdShape bwd_shape(long rows, int n, int period) {
  BwdShape b;
  const int chunks = (n + kChunk - 1) / kChunk;
  // few registers per lane (three column sums and the row's values are held): two
  // accesses of a lane to a row where 256 lanes allow it
  b.tpr = chunks <= 16 ? 16 : chunks <= 32 ? 32 : chunks <= 64 ? 64 : chunks <= 128 ? 128 : 256;
  b.nch = b.tpr < 256 ? 1 : (chunks + 255) / 256;
  b.nch = b.nch <= 2 ? b.nch : b.nch <= 4 ? 4 : 8;
  const long teams = 256 / b.tpr;
  long blocks = (rows + teams - 1) / teams;
  blocks = blocks < 1 ? 1 : blocks < 512 ? blocks : 512;
  const long unit = period / gcd(period, teams);
  b.blocks = (blocks + unit - 1) / unit * unit;
  return b;
}

template <int TPR, int NCH>
hipError_t bwd(const NormArgs& a, long blocks, hipStream_t s) {
  return timed_launch(s, [&] {
    const dim3 grid(static_cast<unsigned>(blocks));
    auto run = [&](auto after, auto before) {
      if (a.gate_first) hipLaunchKernelGGL(before, grid, dim3(256), 0, s, a);
      else hipLaunchKernelGGL(after, grid, dim3(256), 0, s, a);
    };
    const bool same = (!a.dout || a.dout_dtype == a.x_dtype) && (!a.dres || a.dres_dtype == a.res_dtype) &&
                      a.grad_dtype == a.x_dtype;
    switch (known_types(a, same)) {
      case 0: run(norm_bwd_kernel<TPR, NCH, kF32, kF32, false>, norm_bwd_kernel<TPR, NCH, kF32, kF32, true>); break;
      case 1: run(norm_bwd_kernel<TPR, NCH, kBF16, kF32, false>, norm_bwd_kernel<TPR, NCH, kBF16, kF32, true>); break;
      case 2: run(norm_bwd_kernel<TPR, NCH, kBF16, kBF16, false>, norm_bwd_kernel<TPR, NCH, kBF16, kBF16, true>); break;
      default: run(norm_bwd_kernel<TPR, NCH, -1, -1, false>, norm_bwd_kernel<TPR, NCH, -1, -1, true>);
    }
  });
}

}  // namespace

int norm_bwd_parts(long rows, int n, int period) {
  const BwdShape b = bwd_shape(rows, n, period);
  return static_cast<int>(period == 1 ? b.blocks : b.blocks * (256 / b.tpr));
}

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const int chunks = (a.n + kChunk - 1) / kChunk;
  if (chunks <= 16) return fwd<16, 1>(a, s);
  if (chunks <= 32) return fwd<32, 1>(a, s);
  // a wave per row needs no barrier; with few rows four waves share one
  if (a.rows >= 1024 && chunks <= 512) {
    switch ((chunks + 63) / 64) {
      case 1: return fwd<64, 1>(a, s);
      case 2: return fwd<64, 2>(a, s);
      case 3: return fwd<64, 3>(a, s);
      case 4: return fwd<64, 4>(a, s);
      case 5: return fwd<64, 5>(a, s);
      case 6: return fwd<64, 6>(a, s);
      default: return fwd<64, 8>(a, s);
    }
  }
  if (chunks <= 256) return fwd<256, 1>(a, s);
  if (chunks <= 512) return fwd<256, 2>(a, s);
  if (chunks <= 1024) return fwd<256, 4>(a, s);
  return fwd<256, 8>(a, s);
}

// (without rows the kernels still run: the weight gradients are then zeros)
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s) {
  const BwdShape b = bwd_shape(a.rows, a.n, a.w_period);
  hipError_t e;
  if (b.tpr == 16) e = bwd<16, 1>(a, b.blocks, s);
  else if (b.tpr == 32) e = bwd<32, 1>(a, b.blocks, s);
  else if (b.tpr == 64) e = bwd<64, 1>(a, b.blocks, s);
  else if (b.tpr == 128) e = bwd<128, 1>(a, b.blocks, s);
  else if (b.nch == 1) e = bwd<256, 1>(a, b.blocks, s);
  else if (b.nch == 2) e = bwd<256, 2>(a, b.blocks, s);
  else if (b.nch == 4) e = bwd<256, 4>(a, b.blocks, s);
  else e = bwd<256, 8>(a, b.blocks, s);
  if (e != hipSuccess || (!a.dnorm_w && !a.dscale && !a.dout_w)) return e;
  hipLaunchKernelGGL(norm_reduce_kernel, dim3((a.n + 31) / 32, a.w_period, 3), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace ssm
