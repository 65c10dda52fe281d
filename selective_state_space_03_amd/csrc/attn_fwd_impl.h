// Forward of the window attention for gfx950.
//
// A workgroup of four waves takes 64 MT queries of one head, a wave 16 MT of them as columns; the keys and
// values of the tiles that some query sees (the tiles with sinks, then those from the window's begin to the
// last query) go through LDS, double buffered, the next tile's loads in flight during the products.  Per tile
//   S^T = K Q^T   (accumulator columns are queries, so a query's maximum and sum stay in four lanes)
//   P = 2^(scale log2(e) S - m),  m a running maximum, l the running sum
//   O^T += V^T P^T   (the tiles of P are operands as they stand; V is read transposed from LDS)
// m only follows a new maximum that is more than 2^8 above it: the products and sums are those of another
// common factor then, and most tiles leave O as it is.
#pragma once
#include "attn_device.h"

namespace ssm {

template <typename T, int DQ, int MT, int NP, bool VEC>
__global__ __launch_bounds__(256, 2) void attn_fwd_kernel(const AttnArgs a, int o_bf16) {
  using E = AttnEl<T>;
  constexpr int BN = E::kTile, KT = BN / 16, KS = DQ / E::kUnit, NT = DQ / 16, BM = 64 * MT;
  constexpr int PU = sizeof(T) == 2 ? 2 : 1, UN = KT / PU;  // accumulator tiles per unit of tokens, units per tile
  using Tile = AttnTile<T, BN, DQ, VEC>;
  __shared__ __align__(16) unsigned char lds[2][2 * Tile::kBytes];  // keys, values

  const AttnWork w = attn_work(a, blockIdx.x, BM, false, a.h / a.hk);
  if (w.tile < 0) return;
  const AttnSeq sq = w.seq;
  const int lane = threadIdx.x % 64, g = lane / 16, c = lane % 16;
  const int kh = w.head / (a.h / a.hk);
  const int off = sq.nk - sq.nq;                              // position of query 0
  const int i0 = w.tile * BM + threadIdx.x / 64 * (16 * MT);  // the wave's first query
  const T* const kb = static_cast<const T*>(a.k) + sq.k0 * a.k_stride + static_cast<long>(kh) * a.D;
  const T* const vb = static_cast<const T*>(a.v) + sq.k0 * a.v_stride + static_cast<long>(kh) * a.D;

  uint4 q[MT][KS];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int i = i0 + 16 * m + c;
    const T* row = static_cast<const T*>(a.q) + (sq.q0 + i) * a.q_stride + static_cast<long>(w.head) * a.D;
#pragma unroll
    for (int u = 0; u < KS; ++u) {
      q[m][u] = make_uint4(0u, 0u, 0u, 0u);
      if (i < sq.nq) q[m][u] = attn_chunk<T>(row, u * E::kUnit + g * E::kVec, a.D, a.vec);
    }
  }

  // tiles that some query of the workgroup sees
  const int last = off + min(w.tile * BM + BM, sq.nq) - 1;  // its last position
  const int lo = max(0, off + w.tile * BM - a.window + 1);
  const int first = lo / BN;
  const int ns = min((a.sinks + BN - 1) / BN, first);
  const int n = last < 0 ? 0 : ns + max(0, last / BN + 1 - first);

  f32x4 o[MT][NT];
  float mx[MT], l[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    mx[m] = -INFINITY;
    l[m] = 0.0f;
#pragma unroll
    for (int t = 0; t < NT; ++t) o[m][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  const float cs = a.scale * kLog2e;
  const int p0 = off + i0, p1 = p0 + 16 * MT - 1;  // the wave's positions

  uint4 kr[VEC ? 1 : Tile::kPer], vr[VEC ? 1 : Tile::kPer];
  const typename Tile::Source ks = Tile::source(a.k_stride, a.D), vs = Tile::source(a.v_stride, a.D);
  const auto key = [&](int t) { return (t < ns ? t : t - ns + first) * BN; };  // first key of tile t
  const auto load = [&](int t) {
    if constexpr (VEC) {
      Tile::load(lds[t & 1], ks, kb, a.k_stride, key(t), sq.nk, a.D);
      Tile::load(lds[t & 1] + Tile::kBytes, vs, vb, a.v_stride, key(t), sq.nk, a.D);
    } else {
      Tile::fetch(kb, a.k_stride, key(t), sq.nk, a.D, a.vec, kr);
      Tile::fetch(vb, a.v_stride, key(t), sq.nk, a.D, a.vec, vr);
    }
  };
  const auto put = [&](int t) {
    if constexpr (!VEC) {
      Tile::put(lds[t & 1], kr);
      Tile::put(lds[t & 1] + Tile::kBytes, vr);
    }
  };
  if (n > 0) {
    load(0);
    put(0);
  }
  for (int t = 0; t < n; ++t) {
    if constexpr (VEC) loads_done();
    lds_barrier();  // tile t is there, and nobody reads the tile before it any more
    if (t + 1 < n) load(t + 1);
    const int j0 = key(t);
    const unsigned char* const kl = lds[t & 1];
    const unsigned char* const vl = kl + Tile::kBytes;
    const bool some = j0 <= p1 && i0 < sq.nq && (j0 + BN - 1 > p0 - a.window || j0 < a.sinks);
    if (some) {
      f32x4 s[MT][KT];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int k = 0; k < KT; ++k) s[m][k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < KS; ++u)
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          const uint4 x = Tile::rows(kl, 16 * k, u, lane);
#pragma unroll
          for (int m = 0; m < MT; ++m) s[m][k] = attn_mma<T>(x, q[m][u], s[m][k]);
        }
      const bool whole = j0 + BN - 1 <= p0 && (j0 > p1 - a.window || j0 + BN <= a.sinks);
      if (!whole) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int p = p0 + 16 * m + c;
#pragma unroll
          for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = j0 + 16 * k + 4 * g + i;
              s[m][k][i] = j <= p && (j > p - a.window || j < a.sinks) ? s[m][k][i] : -INFINITY;
            }
        }
      }
      float top[MT];
      bool more = false;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float x = s[m][0][0];
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) x = fmaxf(x, s[m][k][i]);
        top[m] = group_max(x) * cs;  // (scale is not negative)
        more |= top[m] > mx[m] + 8.0f;
      }
      if (__any(more)) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float to = fmaxf(mx[m], top[m]);
          const float f = mx[m] == -INFINITY ? 0.0f : exp2_fast(mx[m] - to);
          mx[m] = to;
          l[m] *= f;
#pragma unroll
          for (int d = 0; d < NT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[m][d][i] *= f;
        }
      }
      Frag<NP> p[MT][UN];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float sub = mx[m] == -INFINITY ? 0.0f : mx[m];
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[m][k][i] = exp2_fast(fmaf(s[m][k][i], cs, -sub));
            l[m] += s[m][k][i];
          }
#pragma unroll
        for (int u = 0; u < UN; ++u) p[m][u] = attn_operand<T, NP>(&s[m][PU * u]);
      }
#pragma unroll
      for (int u = 0; u < UN; ++u)
#pragma unroll
        for (int d = 0; d < NT; ++d) {
          const uint4 x = Tile::cols(vl, 16 * PU * u, 16 * d, lane);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = NP - 1; e >= 0; --e) o[m][d] = attn_mma<T>(x, p[m][u].p[e], o[m][d]);
        }
    }
    if (t + 1 < n) put(t + 1);
  }

#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int i = i0 + 16 * m + c;
    const float sum = group_sum(l[m]);
    const float f = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;  // (nothing visible: zeros)
    if (i >= sq.nq) continue;
    const size_t row = static_cast<size_t>(sq.q0 + i) * a.h + w.head;
    if (a.lse && g == 0) a.lse[row] = sum > 0.0f || sum != sum ? (mx[m] + log2_fast(sum)) * kLn2 : -INFINITY;
#pragma unroll
    for (int d = 0; d < NT; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) o[m][d][r] *= f;
    attn_store_row<NT>(a.o, row * a.D, o[m], a.D, g, o_bf16, a.vec);
  }
}

template <typename T, int DQ, int MT, int NP, bool VEC>
hipError_t attn_fwd_go(const AttnLaunch& l, hipStream_t s) {
  const AttnArgs& a = l.a;
  const long blocks = attn_tiles(a, 64 * MT, false) * a.h;
  return timed_launch(s, [&] {
    hipLaunchKernelGGL((attn_fwd_kernel<T, DQ, MT, NP, VEC>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a,
                       l.o_dtype == kBF16);
  });
}

template <typename T, int MT, int NP, bool VEC>
hipError_t attn_fwd_d(const AttnLaunch& l, hipStream_t s) {
  switch (attn_dq(l.a.D)) {
    case 32: return attn_fwd_go<T, 32, MT, NP, VEC>(l, s);
    case 64: return attn_fwd_go<T, 64, MT, NP, VEC>(l, s);
    case 96: return attn_fwd_go<T, 96, MT, NP, VEC>(l, s);
    default: return attn_fwd_go<T, 128, MT, NP, VEC>(l, s);
  }
}
template <typename T, int NP>
hipError_t attn_fwd_narrow(const AttnLaunch& l, hipStream_t s) {  // 64 queries a workgroup
  return l.a.vec == 2 ? attn_fwd_d<T, 1, NP, true>(l, s) : attn_fwd_d<T, 1, NP, false>(l, s);
}

hipError_t attn_fwd_bf16(const AttnLaunch& l, hipStream_t s);
hipError_t attn_fwd_bf16_f32(const AttnLaunch& l, hipStream_t s);
hipError_t attn_fwd_f32(const AttnLaunch& l, hipStream_t s);

}  // namespace ssm
