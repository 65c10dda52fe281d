// Backward of the window attention for gfx950 (no atomics, sums in a fixed order).
//
//   delta_p = sum_d do_pd o_pd
//   P_pj = 2^(scale log2(e) q_p.k_j - log2(e) lse_p),  dS_pj = P_pj (do_p.v_j - delta_p)
//   dq_p = scale sum_j dS_pj k_j   (attn_dq_kernel, queries as columns, as in the forward)
//   dk_j = scale sum_p dS_pj q_p,  dv_j = sum_p P_pj do_p   (attn_dkv_kernel, keys as columns)
// Both form S and dP again: 7 products where one kernel would take 5, which would have to add dq up
// with atomics.  A query that sees one key has P = 1 and no gradient of S: dS = 0 there, and not the
// rounding of do.v - do.o.
#pragma once
#include "attn_device.h"

namespace ssm {

__device__ __forceinline__ float attn_lse2(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }

template <typename T, int DQ, int MT, int NP, bool VEC>
__global__ __launch_bounds__(256, 2) void attn_dq_kernel(const AttnArgs a) {
  using E = AttnEl<T>;
  constexpr int BN = E::kTile, KS = DQ / E::kUnit, NT = DQ / 16, BM = 64 * MT;
  constexpr int PU = sizeof(T) == 2 ? 2 : 1, UN = BN / 16 / PU;
  using Tile = AttnTile<T, BN, DQ, VEC>;
  __shared__ __align__(16) unsigned char lds[2][2 * Tile::kBytes];  // keys, values

  const AttnWork w = attn_work(a, blockIdx.x, BM, false, a.h / a.hk);
  if (w.tile < 0) return;
  const AttnSeq sq = w.seq;
  const int lane = threadIdx.x % 64, g = lane / 16, c = lane % 16;
  const int kh = w.head / (a.h / a.hk);
  const int off = sq.nk - sq.nq;
  const int i0 = w.tile * BM + threadIdx.x / 64 * (16 * MT);
  const T* const kb = static_cast<const T*>(a.k) + sq.k0 * a.k_stride + static_cast<long>(kh) * a.D;
  const T* const vb = static_cast<const T*>(a.v) + sq.k0 * a.v_stride + static_cast<long>(kh) * a.D;

  uint4 q[MT][KS], dO[MT][KS];
  float lse[MT], delta[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int i = i0 + 16 * m + c;
    const long row = (sq.q0 + i) * a.h + w.head;
    const T* qrow = static_cast<const T*>(a.q) + (sq.q0 + i) * a.q_stride + static_cast<long>(w.head) * a.D;
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
  const int lo = max(0, off + w.tile * BM - a.window + 1);
  const int first = lo / BN;
  const int ns = min((a.sinks + BN - 1) / BN, first);
  const int n = last < 0 ? 0 : ns + max(0, last / BN + 1 - first);

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
  const auto key = [&](int t) { return (t < ns ? t : t - ns + first) * BN; };  // first key of tile t
  const auto load = [&](int t) {
    if constexpr (VEC) {
      Tile::load(lds_address(lds[t & 1]), ks, kb, a.k_stride, key(t), sq.nk, a.D);
      Tile::load(lds_address(lds[t & 1]) + Tile::kBytes, vs, vb, a.v_stride, key(t), sq.nk, a.D);
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
      const bool whole = j0 + BN - 1 <= p0 && (j0 > p1 - a.window || j0 + BN <= a.sinks);
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
                s[m][e][i] = j <= p && (j > p - a.window || j < a.sinks) && !lone ? s[m][e][i] : 0.0f;
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
    attn_store_row<NT>(a.dq, (static_cast<size_t>(sq.q0 + i) * a.h + w.head) * a.D, dq[m], a.D, g, a.grad_bf16, a.vec);
  }
}

// A workgroup takes 64 MT keys of one key head, a wave 16 MT of them as columns, and walks the tiles of
// queries that see them, head by head of the key head's (their sum stays in registers).
// The tiles that hold sinks are seen by every later query.  Where they are few (a.sink_tiles), the queries
// are cut into pieces of a.span for them, the first workgroups of the launch, whose partial sums
// attn_sink_kernel adds up.
template <typename T, int DQ, int MT, int NP, bool VEC>
__global__ __launch_bounds__(256, 2) void attn_dkv_kernel(const AttnArgs a, unsigned sink_blocks) {
  using E = AttnEl<T>;
  constexpr int BN = E::kTile, KS = DQ / E::kUnit, NT = DQ / 16, BM = 64 * MT;
  constexpr int PU = sizeof(T) == 2 ? 2 : 1, UN = BN / 16 / PU;
  using Tile = AttnTile<T, BN, DQ, VEC>;
  __shared__ __align__(16) unsigned char lds[2][2 * Tile::kBytes + 8 * BN];

  const int heads = a.h / a.hk;
  const bool sink = blockIdx.x < sink_blocks;
  AttnWork w;
  long slot = 0;
  int piece = 0;
  if (sink) {
    const unsigned per = static_cast<unsigned>(a.hk) * a.sink_tiles;
    slot = blockIdx.x / per;
    const unsigned r = blockIdx.x % per;
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
    w = attn_work(a, blockIdx.x - sink_blocks, BM, true, 1);
    if (w.tile < a.sink_tiles) return;  // (also an unused slot)
  }
  const AttnSeq sq = w.seq;
  const int lane = threadIdx.x % 64, g = lane / 16, c = lane % 16;
  const int kh = w.head;
  const int off = sq.nk - sq.nq;
  const int jt = w.tile * BM, j0 = jt + threadIdx.x / 64 * (16 * MT), j1 = j0 + 16 * MT - 1;

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

  // queries that see some key of the workgroup
  long lo = max(0, jt - off), hi = sq.nq - 1L;
  if (a.window != kAttnAll && jt >= a.sinks) hi = min(hi, static_cast<long>(min(jt + BM, sq.nk)) + a.window - 2 - off);
  if (sink) {
    lo = max(lo, static_cast<long>(piece) * a.span);
    hi = min(hi, static_cast<long>(piece) * a.span + a.span - 1);
  }
  if (jt >= sq.nk) hi = -1;
  const int first = static_cast<int>(lo / BN);
  const int per = hi < lo ? 0 : static_cast<int>(hi / BN) + 1 - first;  // tiles of a head
  const int n = per * heads;

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
  const auto load = [&](int t) {
    const int head = kh * heads + t / per, i0 = (first + t % per) * BN;
    const T* const qb = static_cast<const T*>(a.q) + sq.q0 * a.q_stride + static_cast<long>(head) * a.D;
    const T* const db = static_cast<const T*>(a.dout) + (sq.q0 * a.h + head) * a.D;
    if constexpr (VEC) {
      Tile::load(lds_address(lds[t & 1]), qs, qb, a.q_stride, i0, sq.nq, a.D);
      Tile::load(lds_address(lds[t & 1]) + Tile::kBytes, ds, db, dstride, i0, sq.nq, a.D);
    } else {
      Tile::fetch(qb, a.q_stride, i0, sq.nq, a.D, a.vec, qr);
      Tile::fetch(db, dstride, i0, sq.nq, a.D, a.vec, dr);
    }
    if (threadIdx.x < 2 * BN) {  // lse, then delta
      const int i = i0 + threadIdx.x % BN;
      const long row = (sq.q0 + i) * a.h + head;
      st = threadIdx.x < BN ? INFINITY : 0.0f;
      if (i < sq.nq) st = threadIdx.x < BN ? attn_lse2(a.lse[row]) : a.delta[row];
    }
  };
  const auto put = [&](int t) {
    unsigned char* const to = lds[t & 1];
    if constexpr (!VEC) {
      Tile::put(to, qr);
      Tile::put(to + Tile::kBytes, dr);
    }
    if (threadIdx.x < 2 * BN) reinterpret_cast<float*>(to + 2 * Tile::kBytes)[threadIdx.x] = st;
  };
  if (n > 0) {
    load(0);
    put(0);
  }
  for (int t = 0; t < n; ++t) {
    if constexpr (VEC) loads_done();
    lds_barrier();
    if (t + 1 < n) load(t + 1);
    const unsigned char* const ql = lds[t & 1];
    const unsigned char* const dl = ql + Tile::kBytes;
    const float* const sl = reinterpret_cast<const float*>(ql + 2 * Tile::kBytes);
    const int i0 = (first + t % per) * BN, p0 = off + i0, p1 = p0 + BN - 1;
    const bool some = j0 <= p1 && j0 < sq.nk && (j1 > p0 - a.window || j0 < a.sinks);
    if (some) {
      const bool whole = j1 <= p0 && (j0 > p1 - a.window || j1 < a.sinks) && i0 + BN <= sq.nq;
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
                const bool see = j <= p && (j > p - a.window || j < a.sinks) && r < sq.nq;
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
    if (t + 1 < n) put(t + 1);
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int j = j0 + 16 * m + c;
    if (j >= sq.nk) continue;
#pragma unroll
    for (int d = 0; d < NT; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) dk[m][d][r] *= a.scale;
    if (sink) {
      const size_t at = (((static_cast<size_t>(slot) * a.hk + kh) * a.sink_tiles + w.tile) * BM + (j - jt)) * a.D;
      attn_store_row<NT>(a.dk_part, at, dk[m], a.D, g, 0, a.vec);
      attn_store_row<NT>(a.dv_part, at, dv[m], a.D, g, 0, a.vec);
    } else {
      const size_t at = (static_cast<size_t>(sq.k0 + j) * a.hk + kh) * a.D;
      if (a.dk) attn_store_row<NT>(a.dk, at, dk[m], a.D, g, a.grad_bf16, a.vec);
      if (a.dv) attn_store_row<NT>(a.dv, at, dv[m], a.D, g, a.grad_bf16, a.vec);
    }
  }
}

template <typename T, int DQ, int MT, int NP, bool VEC>
hipError_t attn_bwd_go(const AttnLaunch& l, hipStream_t s) {
  const AttnArgs& a = l.a;
  if (a.dq && a.rows_q > 0) {
    const long blocks = attn_tiles(a, 64 * MT, false) * a.h;
    hipLaunchKernelGGL((attn_dq_kernel<T, DQ, MT, NP, VEC>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!(a.dk || a.dv) || a.rows_k == 0) return hipSuccess;
  const long sinks = a.sink_tiles > 0 ? attn_pieces(a) * a.hk * a.sink_tiles : 0;
  const long blocks = sinks + attn_tiles(a, 64, true) * a.hk;
  hipError_t e = timed_launch(s, [&] {
    hipLaunchKernelGGL((attn_dkv_kernel<T, DQ, 1, NP, VEC>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a,
                       static_cast<unsigned>(sinks));
  });
  if (e == hipSuccess && a.sink_tiles > 0) e = launch_attn_sinks(a, s);
  return e;
}

template <typename T, int MT, int NP, bool VEC>
hipError_t attn_bwd_vec(const AttnLaunch& l, hipStream_t s) {
  switch (attn_dq(l.a.D)) {
    case 32: return attn_bwd_go<T, 32, MT, NP, VEC>(l, s);
    case 64: return attn_bwd_go<T, 64, MT, NP, VEC>(l, s);
    case 96: return attn_bwd_go<T, 96, MT, NP, VEC>(l, s);
    default: return attn_bwd_go<T, 128, MT, NP, VEC>(l, s);
  }
}
template <typename T, int MT, int NP>
hipError_t attn_bwd_d(const AttnLaunch& l, hipStream_t s) {
  return l.a.vec == 2 ? attn_bwd_vec<T, MT, NP, true>(l, s) : attn_bwd_vec<T, MT, NP, false>(l, s);
}

hipError_t attn_bwd_bf16(const AttnLaunch& l, hipStream_t s);
hipError_t attn_bwd_bf16_f32(const AttnLaunch& l, hipStream_t s);
hipError_t attn_bwd_f32(const AttnLaunch& l, hipStream_t s);

}  // namespace ssm
