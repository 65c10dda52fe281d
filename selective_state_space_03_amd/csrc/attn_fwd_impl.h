// Forward of the window attention for gfx950.
//
// A workgroup of four waves takes 64 MT queries of one head, a wave 16 MT of them as columns; the keys and
// values that some query sees (the sinks, then those from the window's begin to the last query, in tiles) go
// through LDS, double buffered, the next tile's loads in flight during the products.  Per tile
//   S^T = K Q^T   (accumulator columns are queries, so a query's maximum and sum stay in four lanes)
//   P = 2^(scale log2(e) S - m),  m a running maximum, l the running sum
//   O^T += V^T P^T   (the tiles of P are operands as they stand; V is read transposed from LDS)
// m only follows a new maximum that is more than 2^8 above it: the products and sums are those of another
// common factor then, and most tiles leave O as it is.
#pragma once
#include <type_traits>

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
  const int i0 = w.tile * BM + uniform(threadIdx.x / 64) * (16 * MT);  // the wave's first query
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
  const AttnKeys<BN> keys(a, off + w.tile * BM, last);
  const int n = keys.n;

  f32x4 o[MT][NT];
  float mx[MT], l[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    mx[m] = -INFINITY;
    l[m] = 0.0f;
#pragma unroll
    for (int t = 0; t < NT; ++t) o[m][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  const float cs = attn_log2_scale(a.scale);
  const int p0 = off + i0, p1 = p0 + 16 * MT - 1;  // the wave's positions

  uint4 kr[VEC ? 1 : Tile::kPer], vr[VEC ? 1 : Tile::kPer];
  const typename Tile::Source ks = Tile::source(a.k_stride, a.D), vs = Tile::source(a.v_stride, a.D);
  const auto load = [&](int t) {
    if constexpr (VEC) {
      Tile::load(lds_address(lds[t & 1]), ks, kb, a.k_stride, keys.key(t), keys.upto(t), a.D);
      Tile::load(lds_address(lds[t & 1]) + Tile::kBytes, vs, vb, a.v_stride, keys.key(t), keys.upto(t), a.D);
    } else {
      Tile::fetch(kb, a.k_stride, keys.key(t), keys.upto(t), a.D, a.vec, kr);
      Tile::fetch(vb, a.v_stride, keys.key(t), keys.upto(t), a.D, a.vec, vr);
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
    const int j0 = keys.key(t), window = keys.window(t, a.window);
    const unsigned char* const kl = lds[t & 1];
    const unsigned char* const vl = kl + Tile::kBytes;
    const bool some = j0 <= p1 && i0 < sq.nq && (j0 + BN - 1 > p0 - window || j0 < a.sinks);
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
      const bool whole = j0 + BN - 1 <= p0 && (j0 > p1 - window || j0 + BN <= a.sinks);
      if (!whole) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int p = p0 + 16 * m + c;
#pragma unroll
          for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = j0 + 16 * k + 4 * g + i;
              s[m][k][i] = j <= p && (j > p - window || j < a.sinks) ? s[m][k][i] : -INFINITY;
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
    if (a.o_rest) {
#pragma unroll
      for (int d = 0; d < NT; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[m][d][r] = rest_of(o[m][d][r]);
      attn_store_row<NT>(a.o_rest, row * a.D, o[m], a.D, g, 1, a.vec);
    }
  }
}

// The same of bf16 rows of aligned 16-byte groups in 32 x 32 tiles, which take half the instructions: 128
// queries a workgroup, 32 a wave, and tiles of 32 keys, with which three workgroups share a CU (64 keys and
// two: 233 instead of 218 us on a prompt of 8192, 32 heads of 128, window 1024).
// 8192 x 32 heads of 128 without a window: 700 us, 785 TFLOP/s of the 1235 that a library product reaches; the
// low parts of P make it 1180.  Zeros take 530: the card's clock follows the products' power.
template <int DQ, int NP>
__global__ __launch_bounds__(256, 3) void attn_fwd_wide_kernel(const AttnArgs a, int o_bf16) {
  constexpr int BN = 32, KT = BN / 32, KS = DQ / 16, NT = DQ / 32, BM = 128;
  using Tile = AttnTile<bf16s, BN, DQ, true>;
  using W = Wide<Tile>;
  __shared__ __align__(16) unsigned char lds[4][Tile::kBytes];  // keys, keys, values, values

  const AttnWork w = attn_work(a, blockIdx.x, BM, false, a.h / a.hk);
  if (w.tile < 0) return;
  const AttnSeq sq = w.seq;
  const int wave = uniform(threadIdx.x / 64), lane = threadIdx.x % 64, h = lane / 32, c = lane % 32;
  const int kh = w.head / (a.h / a.hk);
  const int off = sq.nk - sq.nq;              // position of query 0
  const int i0 = w.tile * BM + wave * 32;     // the wave's first query
  const bf16s* const kb = static_cast<const bf16s*>(a.k) + sq.k0 * a.k_stride + static_cast<long>(kh) * a.D;
  const bf16s* const vb = static_cast<const bf16s*>(a.v) + sq.k0 * a.v_stride + static_cast<long>(kh) * a.D;

  uint4 q[KS];
  {
    const int i = i0 + c;
    const bf16s* const row = static_cast<const bf16s*>(a.q) + (sq.q0 + i) * a.q_stride + static_cast<long>(w.head) * a.D;
#pragma unroll
    for (int u = 0; u < KS; ++u) q[u] = load16_if(row + 16 * u + 8 * h, i < sq.nq && 16 * u + 8 * h < a.D);
  }

  // tiles that some query of the workgroup sees
  const int last = off + min(w.tile * BM + BM, sq.nq) - 1;  // its last position
  const AttnKeys<BN> keys(a, off + w.tile * BM, last);
  const int n = keys.n;

  f32x16 o[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) o[t] = f32x16{};
  float mx = -INFINITY, l = 0.0f;
  const float cs = attn_log2_scale(a.scale);
  const int p0 = off + i0, p1 = p0 + 31;  // the wave's positions

  const typename Tile::Source ks = Tile::source(a.k_stride, a.D), vs = Tile::source(a.v_stride, a.D);
  const uint32_t lds0 = lds_address(lds[0]), k0 = W::rows_at(lds[0], lane), v0 = W::cols_at(lds[2], lane);
  const auto load = [&](int t) {
    Tile::load(lds0 + (t & 1) * Tile::kBytes, ks, kb, a.k_stride, keys.key(t), keys.upto(t), a.D);
    Tile::load(lds0 + (2 + (t & 1)) * Tile::kBytes, vs, vb, a.v_stride, keys.key(t), keys.upto(t), a.D);
  };
  if (n > 0) load(0);
  for (int t = 0; t < n; ++t) {
    loads_done();
    lds_barrier();  // tile t is there, and nobody reads the tile before it any more
    if (t + 1 < n) load(t + 1);
    const int j0 = keys.key(t), window = keys.window(t, a.window);
    if (!(j0 <= p1 && i0 < sq.nq && (j0 + BN - 1 > p0 - window || j0 < a.sinks))) continue;
    // The operands of a step of products are read during the step before it; the order is held, as the
    // compiler would read each right ahead of its use.
    const uint32_t kl = k0 + (t & 1) * Tile::kBytes, vl = v0 + (t & 1) * Tile::kBytes;
    constexpr int NK = KT * KS / 4;  // steps of four products
    f32x16 s[KT];
    uint4 kf[2][4], vf[2][NT];
    const auto read_k = [&](int st) {
#pragma unroll
      for (int x = 0; x < 4; ++x) kf[st & 1][x] = W::rows(kl, 32 * ((4 * st + x) % KT), (4 * st + x) / KT);
    };
    const auto read_v = [&](int st) {
#pragma unroll
      for (int d = 0; d < NT; ++d) vf[st & 1][d] = W::cols(vl, 16 * st, d);
    };
#pragma unroll
    for (int k = 0; k < KT; ++k) s[k] = f32x16{};
    if constexpr (NK == 0) {  // (two units)
      kf[0][0] = W::rows(kl, 0, 0);
      kf[0][1] = W::rows(kl, 0, 1);
      s[0] = mma32(kf[0][0], q[0], s[0]);
      s[0] = mma32(kf[0][1], q[1], s[0]);
    } else {
      read_k(0);
#pragma unroll
      for (int st = 0; st < NK; ++st) {
        if (st + 1 < NK) read_k(st + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int x = 0; x < 4; ++x) s[x % KT] = mma32(kf[st & 1][x], q[(4 * st + x) / KT], s[x % KT]);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (KS * KT % 4 != 0) {
        kf[0][0] = W::rows(kl, 0, KS - 2);
        kf[0][1] = W::rows(kl, 0, KS - 1);
        s[0] = mma32(kf[0][0], q[KS - 2], s[0]);
        s[0] = mma32(kf[0][1], q[KS - 1], s[0]);
      }
    }
    wide_hide<KT>(s, j0, p0, p0 + c, h, window, a.sinks);
    float top = s[0][0];
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, s[k][e]);
    top = half_max(top) * cs;  // (scale is not negative)
    if (__any(top > mx + 8.0f)) {
      const float to = fmaxf(mx, top);
      const float f = mx == -INFINITY ? 0.0f : exp2_fast(mx - to);
      mx = to;
      l *= f;
#pragma unroll
      for (int d = 0; d < NT; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] *= f;
    }
    read_v(0);
    const float sub = mx == -INFINITY ? 0.0f : mx;
    Frag<NP> p[KT][2];
#pragma unroll
    for (int k = 0; k < KT; ++k) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        s[k][e] = exp2_fast(fmaf(s[k][e], cs, -sub));
        l += s[k][e];
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) p[k][u] = wide_operand<NP>(s[k], u);
    }
#pragma unroll
    for (int st = 0; st < 2 * KT; ++st) {
      if (st + 1 < 2 * KT) read_v(st + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int e = NP - 1; e >= 0; --e)
#pragma unroll
        for (int d = 0; d < NT; ++d) o[d] = mma32(vf[st & 1][d], p[st / 2][st % 2].p[e], o[d]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  const int i = i0 + c;
  const float sum = half_sum(l);
  const float f = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;  // (nothing visible: zeros)
  if (i >= sq.nq) return;
  const size_t row = static_cast<size_t>(sq.q0 + i) * a.h + w.head;
  if (a.lse && h == 0) a.lse[row] = sum > 0.0f || sum != sum ? (mx + log2_fast(sum)) * kLn2 : -INFINITY;
#pragma unroll
  for (int d = 0; d < NT; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] *= f;
  wide_store_o<NT>(a, row * a.D, o, h, o_bf16);
}

// The same for few queries that see many keys: one workgroup of 128 queries on a CU has eight waves, two on
// each SIMD: waves w and w + 4 hold the same 32 queries, and waves 0-3 and 4-7 take the tiles of
// keys in turn (tile 2 i, tile 2 i + 1); their sums are joined at the end.
// A wave alternates between a phase of matrix products (scores of its next tile, P v of its present one) and
// one of vector instructions (the softmax), and the halves are one phase apart, held there by a barrier
// between phases: one half's products go beside the other's softmax.
//   phase 2 i:      waves 0-3 products of tile i,     waves 4-7 softmax of tile i  (numbers of the half's own)
//   phase 2 i + 1:  waves 0-3 softmax of tile i + 1,  waves 4-7 products of tile i
// Products of i read the keys of i + 1 and the values of i; a half asks for the keys of i + 3 and the values of
// i + 2 in the softmax phase behind them, over those, three phases ahead of their use.
template <int DQ, int NP>
__global__ __launch_bounds__(512, 2) void attn_fwd_long_kernel(const AttnArgs a, int o_bf16) {
  constexpr int BN = 64, KT = BN / 32, KS = DQ / 16, NT = DQ / 32, BM = 128;
  using Tile = AttnTile<bf16s, BN, DQ, true, 256>;  // loaded by the four waves of a half
  using W = Wide<Tile>;
  // [half][keys, keys, values, values]; at the end [wave][sums of 64 lanes, NT 16 of each]
  __shared__ __align__(16) unsigned char lds[2][4][Tile::kBytes];
  static_assert(sizeof(lds) >= 4 * 64 * (NT * 16 + 2) * 4, "room for the join");

  const AttnWork w = attn_work(a, blockIdx.x, BM, false, a.h / a.hk);
  if (w.tile < 0) return;
  const AttnSeq sq = w.seq;
  const int wave = uniform(threadIdx.x / 64), half = wave / 4, lane = threadIdx.x % 64, h = lane / 32, c = lane % 32;
  const int kh = w.head / (a.h / a.hk);
  const int off = sq.nk - sq.nq;                  // position of query 0
  const int i0 = w.tile * BM + wave % 4 * 32;     // the wave's first query
  const bf16s* const kb = static_cast<const bf16s*>(a.k) + sq.k0 * a.k_stride + static_cast<long>(kh) * a.D;
  const bf16s* const vb = static_cast<const bf16s*>(a.v) + sq.k0 * a.v_stride + static_cast<long>(kh) * a.D;

  uint4 q[KS];
  {
    const int i = i0 + c;
    const bf16s* const row = static_cast<const bf16s*>(a.q) + (sq.q0 + i) * a.q_stride + static_cast<long>(w.head) * a.D;
#pragma unroll
    for (int u = 0; u < KS; ++u) q[u] = load16_if(row + 16 * u + 8 * h, i < sq.nq && 16 * u + 8 * h < a.D);
  }

  // tiles that some query of the workgroup sees
  const int last = off + min(w.tile * BM + BM, sq.nq) - 1;  // its last position
  const AttnKeys<BN> keys(a, off + w.tile * BM, last);
  const int from = static_cast<int>(static_cast<long>(keys.n) * blockIdx.y / a.nsplit);  // the part's tiles
  const int n = static_cast<int>(static_cast<long>(keys.n) * (blockIdx.y + 1) / a.nsplit) - from;

  f32x16 o[NT], s[KT];
  Frag<NP> p[KT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) o[t] = f32x16{};
  float mx = -INFINITY, l = 0.0f;
  const float cs = attn_log2_scale(a.scale);
  const int p0 = off + i0, p1 = p0 + 31;  // the wave's positions

  const typename Tile::Source ks = Tile::source(a.k_stride, a.D), vs = Tile::source(a.v_stride, a.D);
  unsigned char(&mine)[4][Tile::kBytes] = lds[half];
  // the half's tile i (none: zeros, so that the number of loads in flight stays)
  const auto load_k = [&](int i) {
    const int t = 2 * i + half;
    Tile::load(lds_address(mine[i & 1]), ks, kb, a.k_stride, t < n ? keys.key(t + from) : 0, t < n ? keys.upto(t + from) : 0, a.D);
  };
  const auto load_v = [&](int i) {
    const int t = 2 * i + half;
    Tile::load(lds_address(mine[2 + (i & 1)]), vs, vb, a.v_stride, t < n ? keys.key(t + from) : 0, t < n ? keys.upto(t + from) : 0, a.D);
  };
  // The operands of a step of products are read during the step before it; the order is held, as the
  // compiler would read each right ahead of its use.
  // scores of tile i + 1 (with kScores), P v of tile i (with kOut)
  const auto products = [&](int i, auto scores_too, auto out_too) {
    constexpr bool kScores = decltype(scores_too)::value, kOut = decltype(out_too)::value;
    const uint32_t kl = W::rows_at(mine[(i + 1) & 1], lane), vl = W::cols_at(mine[2 + (i & 1)], lane);
    uint4 kf[2][4], vf[2][NT];
    const auto read_k = [&](int st, uint4 (&f)[4]) {
#pragma unroll
      for (int x = 0; x < 4; ++x) f[x] = W::rows(kl, 32 * (x % 2), 2 * st + x / 2);
    };
    const auto read_v = [&](int st, uint4 (&f)[NT]) {
#pragma unroll
      for (int d = 0; d < NT; ++d) f[d] = W::cols(vl, 16 * st, d);
    };
    if constexpr (kScores) {
      read_k(0, kf[0]);
#pragma unroll
      for (int k = 0; k < KT; ++k) s[k] = f32x16{};
#pragma unroll
      for (int st = 0; st < KS / 2; ++st) {
        if (st + 1 < KS / 2) read_k(st + 1, kf[(st + 1) & 1]);
        else if (kOut) read_v(0, vf[0]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int x = 0; x < 4; ++x) s[x % 2] = mma32(kf[st & 1][x], q[2 * st + x / 2], s[x % 2]);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      read_v(0, vf[0]);
    }
    if constexpr (kOut) {
#pragma unroll
      for (int st = 0; st < 4; ++st) {
        if (st < 3) read_v(st + 1, vf[(st + 1) & 1]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int e = NP - 1; e >= 0; --e)
#pragma unroll
          for (int d = 0; d < NT; ++d) o[d] = mma32(vf[st & 1][d], p[st / 2][st % 2].p[e], o[d]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  const auto softmax = [&](int i) {
    const int t = 2 * i + half, j0 = t < n ? keys.key(t + from) : wide_none(p0);
    wide_hide<KT>(s, j0, p0, p0 + c, h, keys.window(t + from, a.window), a.sinks);
    float top = s[0][0];
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, s[k][e]);
    top = half_max(top) * cs;  // (scale is not negative)
    if (__any(top > mx + 8.0f)) {
      const float to = fmaxf(mx, top);
      const float f = mx == -INFINITY ? 0.0f : exp2_fast(mx - to);
      mx = to;
      l *= f;
#pragma unroll
      for (int d = 0; d < NT; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] *= f;
    }
    const float sub = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        s[k][e] = exp2_fast(fmaf(s[k][e], cs, -sub));
        l += s[k][e];
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        p[k][u] = wide_operand<NP>(s[k], u);
#pragma unroll
        for (int e = 0; e < NP; ++e)  // (formed in this phase, not where it is used)
          asm volatile("" : "+v"(p[k][u].p[e].x), "+v"(p[k][u].p[e].y), "+v"(p[k][u].p[e].z), "+v"(p[k][u].p[e].w));
      }
    }
    asm volatile("" : "+v"(l));
  };
  const auto next_phase = [&] {
    __builtin_amdgcn_sched_barrier(0);
    lds_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  const auto vector_phase = [&](int i) {  // softmax of tile i; loads for the products two tiles on
    load_k(i + 2);
    load_v(i + 1);
    softmax(i);
    loads_left<2 * Tile::kPer>();  // (the ones before these)
    next_phase();
  };
  if (n > 0) {
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    load_k(0);
    load_v(0);
    load_k(1);
    loads_done();
    lds_barrier();
    products(-1, yes, no);
    next_phase();  // the keys of tile 0 are read
    const int pairs = (n + 1) / 2;
    // Every wave passes the same 2 pairs + 1 barriers.
    if (half == 0) {
      vector_phase(0);
      for (int i = 0; i + 1 < pairs; ++i) {
        products(i, yes, yes);
        next_phase();
        vector_phase(i + 1);
      }
      products(pairs - 1, no, yes);
      next_phase();
      next_phase();
    } else {
      next_phase();
      for (int i = 0; i + 1 < pairs; ++i) {
        vector_phase(i);
        products(i, yes, yes);
        next_phase();
      }
      vector_phase(pairs - 1);
      products(pairs - 1, no, yes);
      next_phase();
    }
  }

  // the halves' sums
  loads_done();
  __syncthreads();
  float* const red = reinterpret_cast<float*>(lds) + wave % 4 * (NT * 16 + 2) * 64 + lane;
  l = half_sum(l);
  if (half == 1) {
#pragma unroll
    for (int d = 0; d < NT; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) red[(d * 16 + e) * 64] = o[d][e];
    red[NT * 16 * 64] = mx;
    red[(NT * 16 + 1) * 64] = l;
  }
  __syncthreads();
  const int i = i0 + c;
  if (half == 1 || i >= sq.nq) return;
  const float mo = red[NT * 16 * 64], to = fmaxf(mx, mo), sub = to == -INFINITY ? 0.0f : to;
  const float f0 = exp2_fast(mx - sub), f1 = exp2_fast(mo - sub);
  const float sum = l * f0 + red[(NT * 16 + 1) * 64] * f1;
  const float inv = a.nsplit > 1 ? 1.0f : sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;  // (nothing visible: zeros)
  const size_t row = static_cast<size_t>(sq.q0 + i) * a.h + w.head;
#pragma unroll
  for (int d = 0; d < NT; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = (o[d][e] * f0 + red[(d * 16 + e) * 64] * f1) * inv;
  if (a.nsplit > 1) {
    const size_t at = row * a.nsplit + blockIdx.y;
    wide_store_row<NT>(a.part, at * DQ, o, a.D, h, 0, a.vec);
    float* const stats = a.part + static_cast<size_t>(a.rows_q) * a.h * a.nsplit * DQ + 2 * at;
    if (h == 0) stats[0] = to;
    else stats[1] = sum;
    return;
  }
  if (a.lse && h == 0) a.lse[row] = sum > 0.0f || sum != sum ? (to + log2_fast(sum)) * kLn2 : -INFINITY;
  wide_store_o<NT>(a, row * a.D, o, h, o_bf16);
}

template <int DQ, int NP>
hipError_t attn_fwd_wide_go(const AttnLaunch& l, bool few, hipStream_t s) {
  const unsigned blocks = static_cast<unsigned>(attn_tiles(l.a, 128, false) * l.a.h);
  return timed_launch(s, [&] {
    if (few) hipLaunchKernelGGL((attn_fwd_long_kernel<DQ, NP>), dim3(blocks, l.a.nsplit), dim3(512), 0, s, l.a, l.o_dtype == kBF16);
    else hipLaunchKernelGGL((attn_fwd_wide_kernel<DQ, NP>), dim3(blocks), dim3(256), 0, s, l.a, l.o_dtype == kBF16);
  });
}
template <int NP>
hipError_t attn_fwd_wide(const AttnLaunch& l, bool few, hipStream_t s) {
  switch (attn_dq(l.a.D)) {
    case 32: return attn_fwd_wide_go<32, NP>(l, few, s);
    case 64: return attn_fwd_wide_go<64, NP>(l, few, s);
    case 96: return attn_fwd_wide_go<96, NP>(l, few, s);
    default: return attn_fwd_wide_go<128, NP>(l, few, s);
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
