// Backward of the window attention for gfx950 (no atomics, sums in a fixed order).
//
//   delta_p = sum_d do_pd o_pd
//   P_pj = 2^(scale log2(e) q_p.k_j - log2(e) lse_p),  dS_pj = P_pj (do_p.v_j - delta_p)
//   dq_p = scale sum_j dS_pj k_j   (attn_dq, attn_dq_wide: queries as columns, as in the forward)
//   dk_j = scale sum_p dS_pj q_p,  dv_j = sum_p P_pj do_p   (attn_dkv, attn_dkv_wide: keys as columns)
// Both form S and dP again: 7 products where one walk would take 5, which would have to add dq up
// with atomics.  A query that sees one key has P = 1 and no gradient of S: dS = 0 there, and not the
// rounding of do.v - do.o.
//
// P and dS enter their products in two bf16 parts for gradients in bf16 (one would add an error as large as the
// gradients' own rounding), in three for f32 ones of bf16 inputs.
//
// Bound by the matrix cores, the vector instructions beside them and the reads from LDS: 4 x 2048 tokens, 16/4 heads
// of 128, window 1024, bf16: 320-350 us, 129 GFLOP by the formulas, 258 with
// both walks and the parts (matrix cores busy 43 % of the time, vector instructions 31 %).
#pragma once
#include "attn_device.h"

namespace ssm {

__device__ __forceinline__ float attn_lse2(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }

// Bytes of LDS: two tiles of queries and dout, with their statistics, for each half of a workgroup of keys
template <typename T, int DQ>
constexpr int kNarrowBwdLds = 4 * (2 * AttnTile<T, AttnEl<T>::kTile, DQ, true>::kBytes + 8 * AttnEl<T>::kTile);

// The queries' gradients: a wave takes 16 queries as columns; the two halves of the workgroup 64 queries of two
// heads that share their keys, or 128 of one head.
template <typename T, int DQ, int NP, bool VEC>
__device__ __forceinline__ void attn_dq(const AttnArgs& a, unsigned char* mem, unsigned block) {
  using E = AttnEl<T>;
  constexpr int MT = 1, BN = E::kTile, KS = DQ / E::kUnit, NT = DQ / 16;
  constexpr int PU = sizeof(T) == 2 ? 2 : 1, UN = BN / 16 / PU;
  using Tile = AttnTile<T, BN, DQ, VEC, 512>;
  unsigned char(&lds)[2][2 * Tile::kBytes] = *reinterpret_cast<unsigned char(*)[2][2 * Tile::kBytes]>(mem);  // keys, values

  const int heads = a.h / a.hk;
  const bool two = heads % 2 == 0;  // heads, else tiles
  const int BM = two ? 64 : 128;
  const AttnWork w = attn_work(a, block, BM, false, two ? heads / 2 : heads);
  if (w.tile < 0) return;
  const AttnSeq sq = w.seq;
  const int wave = uniform(threadIdx.x / 64), lane = threadIdx.x % 64, g = lane / 16, c = lane % 16;
  const int head = two ? 2 * w.head + wave / 4 : w.head, kh = head / heads;
  const int off = sq.nk - sq.nq;
  const int i0 = w.tile * BM + (two ? wave % 4 : wave) * 16;
  const T* const kb = static_cast<const T*>(a.k) + sq.k0 * a.k_stride + static_cast<long>(kh) * a.D;
  const T* const vb = static_cast<const T*>(a.v) + sq.k0 * a.v_stride + static_cast<long>(kh) * a.D;

  uint4 q[MT][KS], dO[MT][KS];
  float lse[MT], delta[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int i = i0 + 16 * m + c;
    const long row = (sq.q0 + i) * a.h + head;
    const T* qrow = static_cast<const T*>(a.q) + (sq.q0 + i) * a.q_stride + static_cast<long>(head) * a.D;
    const T* drow = static_cast<const T*>(a.dout) + row * a.D;
    lse[m] = INFINITY;
    delta[m] = 0.0f;
    if (i < sq.nq) {
      lse[m] = attn_lse2(a.lse[row]);
      delta[m] = a.delta[row];
    }
#pragma unroll
    for (int u = 0; u < KS; ++u) {
      q[m][u] = dO[m][u] = make_uint4(0u, 0u, 0u, 0u);
      if (i < sq.nq) {
        q[m][u] = attn_chunk<T>(qrow, u * E::kUnit + g * E::kVec, a.D, a.vec);
        dO[m][u] = attn_chunk<T>(drow, u * E::kUnit + g * E::kVec, a.D, a.vec);
      }
    }
  }

  const int last = off + min(w.tile * BM + BM, sq.nq) - 1;
  const AttnKeys<BN> keys(a, off + w.tile * BM, last);
  const int n = keys.n;

  f32x4 dq[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) dq[m][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const float cs = a.scale * kLog2e;
  const int p0 = off + i0, p1 = p0 + 16 * MT - 1;
  const bool lone_all = a.window == 1 && a.sinks == 0;

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
      const bool whole = j0 + BN - 1 <= p0 && (j0 > p1 - window || j0 + BN <= a.sinks);
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        f32x4 s[MT][PU], dp[MT][PU];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int e = 0; e < PU; ++e) s[m][e] = dp[m][e] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int x = 0; x < KS; ++x)
#pragma unroll
          for (int e = 0; e < PU; ++e) {
            const uint4 kf = Tile::rows(kl, 16 * (PU * u + e), x, lane);
            const uint4 vf = Tile::rows(vl, 16 * (PU * u + e), x, lane);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              s[m][e] = attn_mma<T>(kf, q[m][x], s[m][e]);
              dp[m][e] = attn_mma<T>(vf, dO[m][x], dp[m][e]);
            }
          }
        Frag<NP> f[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
          for (int e = 0; e < PU; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[m][e][i] = exp2_fast(fmaf(s[m][e][i], cs, -lse[m])) * (dp[m][e][i] - delta[m]);
          if (!whole) {
            const int p = p0 + 16 * m + c;
            const bool lone = p == 0 || lone_all;
#pragma unroll
            for (int e = 0; e < PU; ++e)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int j = j0 + 16 * (PU * u + e) + 4 * g + i;
                s[m][e][i] = j <= p && (j > p - window || j < a.sinks) && !lone ? s[m][e][i] : 0.0f;
              }
          }
          f[m] = attn_operand<T, NP>(s[m]);
        }
#pragma unroll
        for (int d = 0; d < NT; ++d) {
          const uint4 x = Tile::cols(kl, 16 * PU * u, 16 * d, lane);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = NP - 1; e >= 0; --e) dq[m][d] = attn_mma<T>(x, f[m].p[e], dq[m][d]);
        }
      }
    }
    if (t + 1 < n) put(t + 1);
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int i = i0 + 16 * m + c;
    if (i >= sq.nq) continue;
#pragma unroll
    for (int d = 0; d < NT; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) dq[m][d][r] *= a.scale;
    attn_store_row<NT>(a.dq, (static_cast<size_t>(sq.q0 + i) * a.h + head) * a.D, dq[m], a.D, g, a.grad_bf16, a.vec);
  }
}

// The keys' and values' gradients: a workgroup takes 64 keys of one key head, a wave 16 of them as columns, and
// walks the tiles of queries that see them, head by head of the key head's (their sum stays in registers); each
// half of the workgroup takes every second tile, and their sums are added in LDS at the end.
// The tiles that hold sinks are seen by every later query.  Where they are few (a.sink_tiles), the queries
// are cut into pieces of a.span for them, the first workgroups of the launch, whose partial sums
// attn_sink_kernel adds up.
template <typename T, int DQ, int NP, bool VEC>
__device__ __forceinline__ void attn_dkv(const AttnArgs& a, unsigned char* mem, unsigned block, unsigned sink_blocks) {
  using E = AttnEl<T>;
  constexpr int MT = 1, BN = E::kTile, KS = DQ / E::kUnit, NT = DQ / 16, BM = kSinkRows;
  constexpr int PU = sizeof(T) == 2 ? 2 : 1, UN = BN / 16 / PU;
  using Tile = AttnTile<T, BN, DQ, VEC, 256>;  // loaded by a half
  constexpr int kBuf = 2 * Tile::kBytes + 8 * BN;  // queries, dout, lse, delta
  static_assert(4 * kBuf <= kNarrowBwdLds<T, DQ> && 8 * BM * DQ <= kNarrowBwdLds<T, DQ>, "room for the tiles, for the sums");
  const int wave = uniform(threadIdx.x / 64), half = wave / 4, x256 = threadIdx.x % 256;
  unsigned char(&lds)[2][kBuf] = reinterpret_cast<unsigned char(*)[2][kBuf]>(mem)[half];

  const int heads = a.h / a.hk;
  const bool sink = block < sink_blocks;
  AttnWork w;
  long slot = 0;
  int piece = 0;
  if (sink) {
    const unsigned per = static_cast<unsigned>(a.hk) * a.sink_tiles;
    slot = block / per;
    const unsigned r = block % per;
    w.head = r / a.sink_tiles;
    w.tile = r % a.sink_tiles;
    if (a.cu_q) {
      piece = attn_slot(a.cu_q, a.nseq, a.rows_q, a.span, slot, &w.seq, a, false);
    } else {
      const int pieces = (a.lq + a.span - 1) / a.span;
      w.seq = attn_seq(a, static_cast<int>(slot / pieces));
      piece = static_cast<int>(slot % pieces);
    }
    if (piece < 0) return;
  } else {
    w = attn_work(a, block - sink_blocks, BM, true, 1);
    if (w.tile < a.sink_tiles) return;  // (also an unused slot)
  }
  const AttnSeq sq = w.seq;
  const int lane = threadIdx.x % 64, g = lane / 16, c = lane % 16;
  const int kh = w.head;
  const int off = sq.nk - sq.nq;
  const int jt = w.tile * BM, j0 = jt + wave % 4 * 16, j1 = j0 + 16 * MT - 1;

  uint4 k[MT][KS], v[MT][KS];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int j = j0 + 16 * m + c;
    const T* krow = static_cast<const T*>(a.k) + (sq.k0 + j) * a.k_stride + static_cast<long>(kh) * a.D;
    const T* vrow = static_cast<const T*>(a.v) + (sq.k0 + j) * a.v_stride + static_cast<long>(kh) * a.D;
#pragma unroll
    for (int u = 0; u < KS; ++u) {
      k[m][u] = v[m][u] = make_uint4(0u, 0u, 0u, 0u);
      if (j < sq.nk) {
        k[m][u] = attn_chunk<T>(krow, u * E::kUnit + g * E::kVec, a.D, a.vec);
        v[m][u] = attn_chunk<T>(vrow, u * E::kUnit + g * E::kVec, a.D, a.vec);
      }
    }
  }

  // queries that see some key of the workgroup: others, in whose rows a NaN would not vanish beside P = 0, are not loaded
  long lo = max(0, jt - off), hi = sq.nq - 1L;
  if (a.window != kAttnAll && jt >= a.sinks) hi = min(hi, static_cast<long>(min(jt + BM, sq.nk)) + a.window - 2 - off);
  if (sink) {
    lo = max(lo, static_cast<long>(piece) * a.span);
    hi = min(hi, static_cast<long>(piece) * a.span + a.span - 1);
  }
  if (jt >= sq.nk) hi = -1;
  const int first = static_cast<int>(lo), upto = static_cast<int>(hi) + 1;  // (rows from upto on: zeros, and P = 0)
  const int per = upto <= first ? 0 : (upto - first + BN - 1) / BN;         // tiles of a head
  const int n = per * heads, steps = (n + 1) / 2;  // of both halves, of one

  f32x4 dk[MT][NT], dv[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) dk[m][t] = dv[m][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const float cs = a.scale * kLog2e;
  const bool lone_all = a.window == 1 && a.sinks == 0;

  uint4 qr[VEC ? 1 : Tile::kPer], dr[VEC ? 1 : Tile::kPer];
  float st = 0.0f;
  const long dstride = static_cast<long>(a.h) * a.D;
  const typename Tile::Source qs = Tile::source(a.q_stride, a.D), ds = Tile::source(dstride, a.D);
  int head = kh * heads, row0 = first;  // of the tile asked for next
  const int stop = first + per * BN;
  const auto skip = [&](int by) {
    for (row0 += by * BN; row0 >= stop && per > 0; row0 -= per * BN) ++head;
  };
  const auto load = [&](int t) {
    const int i0 = row0;
    const T* const qb = static_cast<const T*>(a.q) + sq.q0 * a.q_stride + static_cast<long>(head) * a.D;
    const T* const db = static_cast<const T*>(a.dout) + (sq.q0 * a.h + head) * a.D;
    if constexpr (VEC) {
      Tile::load(lds_address(lds[t & 1]), qs, qb, a.q_stride, i0, upto, a.D);
      Tile::load(lds_address(lds[t & 1]) + Tile::kBytes, ds, db, dstride, i0, upto, a.D);
    } else {
      Tile::fetch(qb, a.q_stride, i0, upto, a.D, a.vec, qr);
      Tile::fetch(db, dstride, i0, upto, a.D, a.vec, dr);
    }
    if (x256 < 2 * BN) {  // lse, then delta
      const int i = i0 + x256 % BN;
      const long row = (sq.q0 + i) * a.h + head;
      st = x256 < BN ? INFINITY : 0.0f;
      if (i < upto) st = x256 < BN ? attn_lse2(a.lse[row]) : a.delta[row];
    }
  };
  const auto put = [&](int t) {
    unsigned char* const to = lds[t & 1];
    if constexpr (!VEC) {
      Tile::put(to, qr);
      Tile::put(to + Tile::kBytes, dr);
    }
    if (x256 < 2 * BN) reinterpret_cast<float*>(to + 2 * Tile::kBytes)[x256] = st;
  };
  skip(half);
  int now = row0;  // of the tile at hand
  if (half < n) {
    load(0);
    put(0);
  }
  for (int t = 0; t < steps; ++t) {
    if constexpr (VEC) loads_done();
    lds_barrier();
    const bool more = 2 * (t + 1) + half < n;
    const int i0 = now, p0 = off + i0, p1 = p0 + BN - 1;
    if (more) {
      skip(2);
      now = row0;
      load(t + 1);
    }
    const unsigned char* const ql = lds[t & 1];
    const unsigned char* const dl = ql + Tile::kBytes;
    const float* const sl = reinterpret_cast<const float*>(ql + 2 * Tile::kBytes);
    const bool some = 2 * t + half < n && j0 <= p1 && j0 < sq.nk && (j1 > p0 - a.window || j0 < a.sinks);
    if (some) {
      const bool whole = j1 <= p0 && (j0 > p1 - a.window || j1 < a.sinks) && i0 + BN <= upto;
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        f32x4 s[MT][PU], dp[MT][PU];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int e = 0; e < PU; ++e) s[m][e] = dp[m][e] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int x = 0; x < KS; ++x)
#pragma unroll
          for (int e = 0; e < PU; ++e) {
            const uint4 qf = Tile::rows(ql, 16 * (PU * u + e), x, lane);
            const uint4 df = Tile::rows(dl, 16 * (PU * u + e), x, lane);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              s[m][e] = attn_mma<T>(qf, k[m][x], s[m][e]);
              dp[m][e] = attn_mma<T>(df, v[m][x], dp[m][e]);
            }
          }
#pragma unroll
        for (int e = 0; e < PU; ++e) {
          const f32x4 lse = *reinterpret_cast<const f32x4*>(sl + 16 * (PU * u + e) + 4 * g);
          const f32x4 delta = *reinterpret_cast<const f32x4*>(sl + BN + 16 * (PU * u + e) + 4 * g);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              s[m][e][i] = exp2_fast(fmaf(s[m][e][i], cs, -lse[i]));
              dp[m][e][i] = s[m][e][i] * (dp[m][e][i] - delta[i]);
            }
            if (!whole) {
              const int j = j0 + 16 * m + c;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int r = i0 + 16 * (PU * u + e) + 4 * g + i, p = off + r;
                const bool see = j <= p && (j > p - a.window || j < a.sinks) && r < upto;
                s[m][e][i] = see ? s[m][e][i] : 0.0f;
                dp[m][e][i] = see && p != 0 && !lone_all ? dp[m][e][i] : 0.0f;
              }
            }
          }
        }
        Frag<NP> fp[MT], fs[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          fp[m] = attn_operand<T, NP>(s[m]);
          fs[m] = attn_operand<T, NP>(dp[m]);
        }
#pragma unroll
        for (int d = 0; d < NT; ++d) {
          const uint4 x = Tile::cols(dl, 16 * PU * u, 16 * d, lane);
          const uint4 y = Tile::cols(ql, 16 * PU * u, 16 * d, lane);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = NP - 1; e >= 0; --e) {
              dv[m][d] = attn_mma<T>(x, fp[m].p[e], dv[m][d]);
              dk[m][d] = attn_mma<T>(y, fs[m].p[e], dk[m][d]);
            }
        }
      }
    }
    if (more) put(t + 1);
  }

  // the second half's sums in LDS: [wave][dk, dv][tile of channels][lane]
  f32x4* const sums = reinterpret_cast<f32x4*>(mem) + wave % 4 * (2 * NT * 64) + lane;
  lds_barrier();
  if (half == 1) {
#pragma unroll
    for (int d = 0; d < NT; ++d) {
      sums[d * 64] = dk[0][d];
      sums[(NT + d) * 64] = dv[0][d];
    }
  }
  lds_barrier();
  if (half == 1) return;
#pragma unroll
  for (int d = 0; d < NT; ++d) {
    dk[0][d] = (dk[0][d] + sums[d * 64]) * a.scale;
    dv[0][d] += sums[(NT + d) * 64];
  }
  const int j = j0 + c;
  if (j >= sq.nk) return;
  if (sink) {
    const size_t at = (((static_cast<size_t>(slot) * a.hk + kh) * a.sink_tiles + w.tile) * BM + (j - jt)) * a.D;
    attn_store_row<NT>(a.dk_part, at, dk[0], a.D, g, 0, a.vec);
    attn_store_row<NT>(a.dv_part, at, dv[0], a.D, g, 0, a.vec);
  } else {
    const size_t at = (static_cast<size_t>(sq.k0 + j) * a.hk + kh) * a.D;
    if (a.dk) attn_store_row<NT>(a.dk, at, dk[0], a.D, g, a.grad_bf16, a.vec);
    if (a.dv) attn_store_row<NT>(a.dv, at, dv[0], a.D, g, a.grad_bf16, a.vec);
  }
}

// One launch of both, so that queries' workgroups fill the compute units that the keys' leave (with the halves above
// 113 -> 80 us for a step of 3 packed sequences of 1000 tokens in f32, 6/2 heads of 64)
template <typename T, int DQ, int NP, bool VEC>
__global__ __launch_bounds__(512, 2) void attn_bwd_kernel(const AttnArgs a, unsigned sink_blocks, unsigned key_blocks) {
  __shared__ __align__(16) unsigned char lds[kNarrowBwdLds<T, DQ>];
  if (blockIdx.x < key_blocks) attn_dkv<T, DQ, NP, VEC>(a, lds, blockIdx.x, sink_blocks);
  else attn_dq<T, DQ, NP, VEC>(a, lds, blockIdx.x - key_blocks);
}

constexpr int wide_bwd_lds(int dq) {  // bytes: keys' workgroups need the more
  const int row = (dq == 96 ? 128 : dq) * 2;
  return 4 * 4 * 32 * row + 64 * row + 4 * 2 * 64 * 4;
}

// A wave's vector work goes between its own products (training step 407 -> 396 us)
template <int n>
__device__ __forceinline__ void beside_products() {
#pragma unroll
  for (int i = 0; i < n; ++i) {
    __builtin_amdgcn_sched_group_barrier(8, 1, 0);  // a product
    __builtin_amdgcn_sched_group_barrier(2, 4, 0);  // vector instructions
  }
}
// Ahead of a branch between products and the first use of their results: there the compiler counts the wait
// states (11 behind a product of 32 x 32 x 16) along one path only.
__device__ __forceinline__ void products_done() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 10");
  __builtin_amdgcn_sched_barrier(0);
}
// The gradients of bf16 rows of aligned 16-byte groups in 32 x 32 tiles by eight waves.  Operands are read from
// LDS two products ahead, in an order that is held (three ahead, the keys' walk needs more than its 256 registers).
// The queries': 32 a wave, tiles of 32 keys; the two halves of the workgroup take 128 queries of two heads that
// share their keys, or 256 of one head.
template <int DQ, int NP>
__device__ __forceinline__ void attn_dq_wide(const AttnArgs& a, unsigned char* mem, unsigned block) {
  constexpr int BN = 32, KS = DQ / 16, NT = DQ / 32;
  using Tile = AttnTile<bf16s, BN, DQ, true, 512>;
  using W = Wide<Tile>;
  unsigned char(&lds)[4][Tile::kBytes] = *reinterpret_cast<unsigned char(*)[4][Tile::kBytes]>(mem);  // keys, keys, values, values

  const int heads = a.h / a.hk;
  const bool two = heads % 2 == 0;  // heads, else tiles
  const int BM = two ? 128 : 256;
  const AttnWork w = attn_work(a, block, BM, false, two ? heads / 2 : heads);
  if (w.tile < 0) return;
  const AttnSeq sq = w.seq;
  const int wave = uniform(threadIdx.x / 64), lane = threadIdx.x % 64, h = lane / 32, c = lane % 32;
  const int head = two ? 2 * w.head + wave / 4 : w.head, kh = head / heads;
  const int off = sq.nk - sq.nq;
  const int i0 = w.tile * BM + (two ? wave % 4 : wave) * 32;
  const bf16s* const kb = static_cast<const bf16s*>(a.k) + sq.k0 * a.k_stride + static_cast<long>(kh) * a.D;
  const bf16s* const vb = static_cast<const bf16s*>(a.v) + sq.k0 * a.v_stride + static_cast<long>(kh) * a.D;

  uint4 q[KS], dO[KS];
  float lse = INFINITY, delta = 0.0f;
  {
    const int i = i0 + c;
    const long at = (sq.q0 + i) * a.h + head;
    const bf16s* const qrow = static_cast<const bf16s*>(a.q) + (sq.q0 + i) * a.q_stride + static_cast<long>(head) * a.D;
    const bf16s* const drow = static_cast<const bf16s*>(a.dout) + at * a.D;
#pragma unroll
    for (int u = 0; u < KS; ++u) {
      const bool in = i < sq.nq && 16 * u + 8 * h < a.D;
      q[u] = load16_if(qrow + 16 * u + 8 * h, in);
      dO[u] = load16_if(drow + 16 * u + 8 * h, in);
    }
    if (i < sq.nq) {
      lse = attn_lse2(a.lse[at]);
      delta = a.delta[at];
    }
  }

  const int last = off + min(w.tile * BM + BM, sq.nq) - 1;
  const AttnKeys<BN> keys(a, off + w.tile * BM, last);
  const int n = keys.n;

  f32x16 dq[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) dq[t] = f32x16{};
  const float cs = a.scale * kLog2e;
  const int p0 = off + i0, p1 = p0 + 31;
  const bool lone_all = a.window == 1 && a.sinks == 0;

  const typename Tile::Source ks = Tile::source(a.k_stride, a.D), vs = Tile::source(a.v_stride, a.D);
  const uint32_t lds0 = lds_address(lds[0]), k0 = W::rows_at(lds[0], lane), v0 = W::rows_at(lds[2], lane), c0 = W::cols_at(lds[0], lane);
  const auto load = [&](int t) {
    Tile::load(lds0 + (t & 1) * Tile::kBytes, ks, kb, a.k_stride, keys.key(t), keys.upto(t), a.D);
    Tile::load(lds0 + (2 + (t & 1)) * Tile::kBytes, vs, vb, a.v_stride, keys.key(t), keys.upto(t), a.D);
  };
  if (n > 0) load(0);
  for (int t = 0; t < n; ++t) {
    loads_done();
    lds_barrier();
    if (t + 1 < n) load(t + 1);
    const int j0 = keys.key(t), window = keys.window(t, a.window);
    if (!(j0 <= p1 && i0 < sq.nq && (j0 + BN - 1 > p0 - window || j0 < a.sinks))) continue;
    const uint32_t kl = k0 + (t & 1) * Tile::kBytes, vl = v0 + (t & 1) * Tile::kBytes, cl = c0 + (t & 1) * Tile::kBytes;
    f32x16 s = {}, dp = {};
    uint4 kf[3][2], cf[2][NT];
    const auto read = [&](int st) {  // keys, then values
#pragma unroll
      for (int x = 0; x < 2; ++x) kf[st % 3][x] = st < KS / 2 ? W::rows(kl, 0, 2 * st + x) : W::rows(vl, 0, 2 * (st - KS / 2) + x);
    };
    const auto read_c = [&](int u) {
#pragma unroll
      for (int d = 0; d < NT; ++d) cf[u][d] = W::cols(cl, 16 * u, d);
    };
    read(0);
    read(1);
#pragma unroll
    for (int st = 0; st < KS; ++st) {
      if (st + 2 < KS) read(st + 2);
      if (st == KS - 1) read_c(0);
      __builtin_amdgcn_sched_barrier(0);
      if (st < KS / 2) {
#pragma unroll
        for (int x = 0; x < 2; ++x) s = mma32(kf[st % 3][x], q[2 * st + x], s);
      } else {
        const int u = st - KS / 2;
#pragma unroll
        for (int x = 0; x < 2; ++x) dp = mma32(kf[st % 3][x], dO[2 * u + x], dp);
#pragma unroll
        for (int e = 16 * u / (KS / 2); e < 16 * (u + 1) / (KS / 2); ++e) {
          s[e] = exp2_fast(fmaf(s[e], cs, -lse));
          asm volatile("" : "+v"(s[e]));  // (here, not where it is used)
        }
        beside_products<2>();
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    products_done();
    if (!(j0 + BN - 1 <= p0 && (j0 > p1 - window || j0 + BN <= a.sinks))) {
      const int pos = p0 + c;
      const auto [d, v, f] = wide_mask(pos, j0, h, window, a.sinks);
      const bool lone = pos == 0 || lone_all;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int j = 8 * (e / 4) + e % 4;
        const bool see = j <= d && (j > v || j < f) && !lone;
        s[e] = see ? s[e] : 0.0f;
        dp[e] = see ? dp[e] : 0.0f;
      }
    }
    Frag<NP> p[2];
    const auto form = [&](int u) {
#pragma unroll
      for (int e = 8 * u; e < 8 * u + 8; ++e) s[e] *= dp[e] - delta;
      p[u] = wide_operand<NP>(s, u);
    };
    form(0);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (u == 0) read_c(1);
      __builtin_amdgcn_sched_barrier(0);
      if (u == 0) form(1);
#pragma unroll
      for (int e = NP - 1; e >= 0; --e)
#pragma unroll
        for (int d = 0; d < NT; ++d) dq[d] = mma32(cf[u][d], p[u].p[e], dq[d]);
      beside_products<NP * NT>();
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  const int i = i0 + c;
  if (i >= sq.nq) return;
#pragma unroll
  for (int d = 0; d < NT; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) dq[d][e] *= a.scale;
  wide_store_row<NT>(a.dq, (static_cast<size_t>(sq.q0 + i) * a.h + head) * a.D, dq, a.D, h, a.grad_bf16, a.vec);
}

// The keys' and values' gradients: 64 keys a workgroup, 32 a wave as columns, four pairs of waves that take every
// fourth tile of 32 queries.  The keys are held in registers; the values, for which there is no room beside both
// sums, in LDS.  The pairs' sums are added in LDS at the end.  (128 keys a workgroup and no pairs leave a wave per
// SIMD: 412 instead of 244 us for this part.)  Scores start from -lse / scale, dP from -delta, read from LDS into the
// accumulators.
template <int DQ, int NP>
__device__ __forceinline__ void attn_dkv_wide(const AttnArgs& a, unsigned char* mem, unsigned block, unsigned sink_blocks) {
  constexpr int BN = 32, KS = DQ / 16, NT = DQ / 32, BM = 64, G = 4;
  constexpr int CT = NT == 4 ? 2 : NT, CS = NT / CT;  // channels' tiles of a step of products
  using Tile = AttnTile<bf16s, BN, DQ, true, 128>;    // loaded by a pair of waves
  using VTile = AttnTile<bf16s, BM, DQ, true, 512>;
  using W = Wide<Tile>;
  struct Lds {
    unsigned char tiles[G][4][Tile::kBytes];  // queries, queries, dout, dout; at the end sums
    unsigned char values[VTile::kBytes];
    float stats[G][2][2 * BN];  // -lse / scale, -delta: what the products start from
  };
  static_assert(sizeof(Lds) <= wide_bwd_lds(DQ) && sizeof(Lds::tiles) >= G * BM * DQ * 4, "room for the sums");
  auto& lds = reinterpret_cast<Lds*>(mem)->tiles;
  auto& vlds = reinterpret_cast<Lds*>(mem)->values;
  auto& stats = reinterpret_cast<Lds*>(mem)->stats;

  const int heads = a.h / a.hk;
  const bool sink = block < sink_blocks;
  AttnWork w;
  long slot = 0;
  int piece = 0;
  if (sink) {
    const unsigned per = static_cast<unsigned>(a.hk) * a.sink_tiles;
    slot = block / per;
    const unsigned r = block % per;
    w.head = r / a.sink_tiles;
    w.tile = r % a.sink_tiles;
    if (a.cu_q) {
      piece = attn_slot(a.cu_q, a.nseq, a.rows_q, a.span, slot, &w.seq, a, false);
    } else {
      const int pieces = (a.lq + a.span - 1) / a.span;
      w.seq = attn_seq(a, static_cast<int>(slot / pieces));
      piece = static_cast<int>(slot % pieces);
    }
    if (piece < 0) return;
  } else {
    w = attn_work(a, block - sink_blocks, BM, true, 1);
    if (w.tile < a.sink_tiles) return;  // (also an unused slot)
  }
  const AttnSeq sq = w.seq;
  const int wave = uniform(threadIdx.x / 64), g = wave / 2, lane = threadIdx.x % 64, h = lane / 32, c = lane % 32;
  const int kh = w.head;
  const int off = sq.nk - sq.nq;
  const int jt = w.tile * BM, j0 = jt + wave % 2 * 32, j1 = j0 + 31;

  VTile::load(lds_address(vlds), VTile::source(a.v_stride, a.D), static_cast<const bf16s*>(a.v) + sq.k0 * a.v_stride + static_cast<long>(kh) * a.D,
              a.v_stride, jt, sq.nk, a.D);
  uint4 k[KS];
  {
    const int j = j0 + c;
    const bf16s* const row = static_cast<const bf16s*>(a.k) + (sq.k0 + j) * a.k_stride + static_cast<long>(kh) * a.D;
#pragma unroll
    for (int u = 0; u < KS; ++u) k[u] = load16_if(row + 16 * u + 8 * h, j < sq.nk && 16 * u + 8 * h < a.D);
  }

  // queries that see some key of the workgroup: others, in whose rows a NaN would not vanish beside P = 0, are not loaded
  long lo = max(0, jt - off), hi = sq.nq - 1L;
  if (a.window != kAttnAll && jt >= a.sinks) hi = min(hi, static_cast<long>(min(jt + BM, sq.nk)) + a.window - 2 - off);
  if (sink) {
    lo = max(lo, static_cast<long>(piece) * a.span);
    hi = min(hi, static_cast<long>(piece) * a.span + a.span - 1);
  }
  if (jt >= sq.nk) hi = -1;
  const int first = static_cast<int>(lo), upto = static_cast<int>(hi) + 1;  // (rows from upto on: zeros, and P = 0)
  const int per = upto <= first ? 0 : (upto - first + BN - 1) / BN;         // tiles of a head
  const int n = per * heads, steps = (n + G - 1) / G;

  f32x16 dk[NT], dv[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) dk[t] = dv[t] = f32x16{};
  const float cs = attn_log2_scale(a.scale), inv = 1.0f / cs;
  const bool lone_all = a.window == 1 && a.sinks == 0;

  const long dstride = static_cast<long>(a.h) * a.D;
  const typename Tile::Source qs = Tile::source(a.q_stride, a.D), ds = Tile::source(dstride, a.D);
  unsigned char(&mine)[4][Tile::kBytes] = lds[g];
  const uint32_t lds0 = lds_address(mine[0]), q0 = W::rows_at(mine[0], lane), qc0 = W::cols_at(mine[0], lane);
  const uint32_t vl = Wide<VTile>::rows_at(vlds + wave % 2 * 32 * VTile::kStride, lane);
  const bool stater = threadIdx.x % 128 < 2 * BN;
  float st = 0.0f;
  int head = kh * heads, row = first;  // of the tile asked for next
  const int stop = first + per * BN;
  const auto skip = [&](int by) {
    for (row += by * BN; row >= stop && per > 0; row -= per * BN) ++head;
  };
  const auto load = [&](int t) {
    const int i0 = row;
    Tile::load(lds0 + (t & 1) * Tile::kBytes, qs, static_cast<const bf16s*>(a.q) + sq.q0 * a.q_stride + static_cast<long>(head) * a.D, a.q_stride,
               i0, upto, a.D);
    Tile::load(lds0 + (2 + (t & 1)) * Tile::kBytes, ds, static_cast<const bf16s*>(a.dout) + (sq.q0 * a.h + head) * a.D, dstride, i0, upto, a.D);
    if (stater) {
      const int x = threadIdx.x % (2 * BN), i = i0 + x % BN;
      const long row = (sq.q0 + i) * a.h + head;
      st = x < BN ? -INFINITY : 0.0f;
      if (i < upto) st = x < BN ? attn_lse2(a.lse[row]) * -inv : -a.delta[row];
    }
  };
  skip(g);
  int now = row;  // of the tile at hand
  if (g < n) {
    load(0);
    if (stater) stats[g][0][threadIdx.x % (2 * BN)] = st;
  }
  for (int t = 0; t < steps; ++t) {
    loads_done();
    lds_barrier();
    const bool more = G * (t + 1) + g < n;
    const int i0 = now, p0 = off + i0, p1 = p0 + BN - 1;
    if (more) {
      skip(G);
      now = row;
      load(t + 1);
    }
    if (G * t + g < n && j0 <= p1 && j0 < sq.nk && (j1 > p0 - a.window || j0 < a.sinks)) {
      const uint32_t ql = q0 + (t & 1) * Tile::kBytes, dl = ql + 2 * Tile::kBytes;
      const uint32_t qc = qc0 + (t & 1) * Tile::kBytes, dc = qc + 2 * Tile::kBytes;
      f32x16 s, dp;
      uint4 qf[3], df[2], vf[2], cf[2][CT];
      const auto read_q = [&](int u) { qf[u % 3] = W::rows(ql, 0, u); };
      const auto read_d = [&](int u) {
        df[u & 1] = W::rows(dl, 0, u);
        vf[u & 1] = Wide<VTile>::rows(vl, 0, u);
      };
      const auto read_c = [&](int z) {  // dout's two units of 16 queries, then the queries', CT tiles of channels each
        const int x = z / CS;
#pragma unroll
        for (int d = 0; d < CT; ++d) cf[z & 1][d] = W::cols(x < 2 ? dc : qc, 16 * (x & 1), z % CS * CT + d);
      };
      const auto read_stats = [&](int of, f32x16& to) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const f32x4 r = *reinterpret_cast<const f32x4*>(&stats[g][t & 1][of * BN + 8 * x + 4 * h]);
#pragma unroll
          for (int i = 0; i < 4; ++i) to[4 * x + i] = r[i];
        }
      };
      read_stats(0, s);
#pragma unroll
      for (int u = 0; u < 2; ++u) read_q(u);
#pragma unroll
      for (int u = 0; u < KS; ++u) {
        if (u + 2 < KS) read_q(u + 2);
        if (u == KS - 1) {
          read_d(0);
          read_stats(1, dp);
        }
        __builtin_amdgcn_sched_barrier(0);
        s = mma32(qf[u % 3], k[u], s);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int u = 0; u < KS; ++u) {
        if (u + 1 < KS) read_d(u + 1);
        if (u == KS - 1) read_c(0);
        __builtin_amdgcn_sched_barrier(0);
        dp = mma32(df[u & 1], vf[u & 1], dp);
#pragma unroll
        for (int e = 16 * u / KS; e < 16 * (u + 1) / KS; ++e) {
          s[e] = exp2_fast(s[e] * cs);
          asm volatile("" : "+v"(s[e]));  // (here, not where it is used)
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      products_done();
      if (!(j1 <= p0 && (j0 > p1 - a.window || j1 < a.sinks) && i0 + BN <= upto)) {
        const int j = j0 + c, d = j - p0 - 4 * h, end = upto - i0 - 4 * h;  // rows from d on, before d + window (or a sink), before end
        const long far = j < a.sinks ? static_cast<long>(kAttnAll) * 2 : static_cast<long>(d) + a.window;
        const int past = static_cast<int>(min(static_cast<long>(end), far)), zero = -p0 - 4 * h;  // the row at position 0
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int r = 8 * (e / 4) + e % 4;
          const bool see = r >= d && r < past;
          s[e] = see ? s[e] : 0.0f;
          dp[e] = see && r != zero && !lone_all ? dp[e] : 0.0f;
        }
      }
      uint32_t pw[2][NP][4];
      const auto form = [&](int x, int from, int to) {  // pairs of P's units, then dS's
#pragma unroll
        for (int i = from; i < to; ++i) {
          const int e = 8 * (x & 1) + 2 * i;
          uint32_t w2[NP];
          if (x < 2) split2<NP>(s[e], s[e + 1], w2);
          else split2<NP>(s[e] * dp[e], s[e + 1] * dp[e + 1], w2);
#pragma unroll
          for (int y = 0; y < NP; ++y) pw[x & 1][y][i] = w2[y];
        }
      };
      form(0, 0, 4);
#pragma unroll
      for (int z = 0; z < 4 * CS; ++z) {
        const int x = z / CS, y = z % CS * CT;
        if (z + 1 < 4 * CS) read_c(z + 1);
        __builtin_amdgcn_sched_barrier(0);
        if (x < 3) form(x + 1, 4 * (z % CS) / CS, 4 * (z % CS + 1) / CS);
#pragma unroll
        for (int e = NP - 1; e >= 0; --e) {
          const uint4 p = make_uint4(pw[x & 1][e][0], pw[x & 1][e][1], pw[x & 1][e][2], pw[x & 1][e][3]);
#pragma unroll
          for (int d = 0; d < CT; ++d) {
            if (x < 2) dv[y + d] = mma32(cf[z & 1][d], p, dv[y + d]);
            else dk[y + d] = mma32(cf[z & 1][d], p, dk[y + d]);
          }
        }
        beside_products<NP * CT>();
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (more && stater) stats[g][(t + 1) & 1][threadIdx.x % (2 * BN)] = st;
  }
  loads_done();  // (the values, where no query sees a key)

  // each pair adds every fourth tile of channels, in the pairs' order
  const int j = j0 + c;
  float* const sums = reinterpret_cast<float*>(lds);
  const auto join = [&](f32x16(&x)[NT], float f, void* out, float* part) {
    lds_barrier();
#pragma unroll
    for (int d = 0; d < NT; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f32x4*>(sums + (((wave * NT + d) * 4 + i) * 64 + lane) * 4) = f32x4{x[d][4 * i], x[d][4 * i + 1], x[d][4 * i + 2], x[d][4 * i + 3]};
    lds_barrier();
    if (j >= sq.nk) return;
    for (int d = g; d < NT; d += G) {
      f32x16 r[1] = {};
#pragma unroll
      for (int y = 0; y < G; ++y)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 add = *reinterpret_cast<const f32x4*>(sums + ((((2 * y + wave % 2) * NT + d) * 4 + i) * 64 + lane) * 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) r[0][4 * i + e] += add[e];
        }
#pragma unroll
      for (int e = 0; e < 16; ++e) r[0][e] *= f;
      if (sink) {
        const size_t at = (((static_cast<size_t>(slot) * a.hk + kh) * a.sink_tiles + w.tile) * BM + (j - jt)) * a.D;
        wide_store_row<1>(part, at + 32 * d, r, a.D - 32 * d, h, 0, a.vec);
      } else if (out) {
        wide_store_row<1>(out, (static_cast<size_t>(sq.k0 + j) * a.hk + kh) * a.D + 32 * d, r, a.D - 32 * d, h, a.grad_bf16, a.vec);
      }
    }
  };
  join(dk, a.scale, a.dk, a.dk_part);
  join(dv, 1.0f, a.dv, a.dv_part);
}

// One launch of both, so that queries' workgroups fill the compute units that the keys' leave (training step 440 ->
// 407 us)
template <int DQ, int NP>
__global__ __launch_bounds__(512, 2) void attn_bwd_wide_kernel(const AttnArgs a, unsigned sink_blocks, unsigned key_blocks) {
  __shared__ __align__(16) unsigned char lds[wide_bwd_lds(DQ)];
  if (blockIdx.x < key_blocks) attn_dkv_wide<DQ, NP>(a, lds, blockIdx.x, sink_blocks);
  else attn_dq_wide<DQ, NP>(a, lds, blockIdx.x - key_blocks);
}

struct KeyBlocks {
  unsigned sinks, all;  // workgroups: of the sinks' pieces, with those of 64 keys
};
inline KeyBlocks key_blocks(const AttnArgs& a) {
  if (!(a.dk || a.dv) || a.rows_k == 0) return {0, 0};
  const long sinks = a.sink_tiles > 0 ? attn_pieces(a) * a.hk * a.sink_tiles : 0;
  return {static_cast<unsigned>(sinks), static_cast<unsigned>(sinks + attn_tiles(a, kSinkRows, true) * a.hk)};
}

// One launch of a kernel whose query workgroups take `rows` queries, and of the sinks' pieces
template <typename K>
hipError_t attn_bwd_launch(const AttnArgs& a, int rows, K* kernel, hipStream_t s) {
  const KeyBlocks b = key_blocks(a);
  const long blocks = b.all + (a.dq && a.rows_q > 0 ? attn_query_blocks(a, rows) : 0);
  if (blocks == 0) return hipSuccess;
  const hipError_t e =
      timed_launch(s, [&] { hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks)), dim3(512), 0, s, a, b.sinks, b.all); });
  return e == hipSuccess && b.sinks > 0 ? launch_attn_sinks(a, s) : e;
}

template <typename T, int NP, bool VEC>
hipError_t attn_bwd_vec(const AttnArgs& a, hipStream_t s) {
  switch (attn_dq(a.D)) {
    case 32: return attn_bwd_launch(a, 64, attn_bwd_kernel<T, 32, NP, VEC>, s);
    case 64: return attn_bwd_launch(a, 64, attn_bwd_kernel<T, 64, NP, VEC>, s);
    case 96: return attn_bwd_launch(a, 64, attn_bwd_kernel<T, 96, NP, VEC>, s);
    default: return attn_bwd_launch(a, 64, attn_bwd_kernel<T, 128, NP, VEC>, s);
  }
}
template <typename T, int NP>
hipError_t attn_bwd_d(const AttnArgs& a, hipStream_t s) {
  return a.vec == 2 ? attn_bwd_vec<T, NP, true>(a, s) : attn_bwd_vec<T, NP, false>(a, s);
}

template <int NP>
hipError_t attn_bwd_wide(const AttnArgs& a, hipStream_t s) {
  switch (attn_dq(a.D)) {
    case 32: return attn_bwd_launch(a, 128, attn_bwd_wide_kernel<32, NP>, s);
    case 64: return attn_bwd_launch(a, 128, attn_bwd_wide_kernel<64, NP>, s);
    case 96: return attn_bwd_launch(a, 128, attn_bwd_wide_kernel<96, NP>, s);
    default: return attn_bwd_launch(a, 128, attn_bwd_wide_kernel<128, NP>, s);
  }
}

hipError_t attn_bwd_bf16(const AttnArgs& a, hipStream_t s);
hipError_t attn_bwd_bf16_f32(const AttnArgs& a, hipStream_t s);
hipError_t attn_bwd_f32(const AttnArgs& a, hipStream_t s);

}  // namespace ssm
