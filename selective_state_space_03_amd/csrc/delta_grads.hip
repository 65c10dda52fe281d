// The gradients of a chunk of the gated delta rule, all chunks in parallel,
// from what the two walks kept: the state S entering the chunk and the gradient
// D of the state leaving it, the corrections u and dR = T^T dU (delta_pass.hip).
// With k^ = rk k, q^ = scale rq q, E_ts = e^{G_t - G_s}, and per chunk
//   dP = do u^T,  dL = -dR u^T,  W = dP E (s <= t),  M = dL beta_t E (s < t):
//   dv = beta dR
//   dq^_t = e^{G_t} S do_t + sum_s W_ts k^_s
//   dk^_t = -beta_t e^{G_t} S dR_t + e^{G_C-G_t} D u_t + sum_s W_st q^_s + sum_s (M_ts + M_st) k^_s
//   dbeta_t = dR_t.v_t - e^{G_t} k^_t.(S dR_t) + sum_s dL_ts E_ts k^_t.k^_s
//   dG_t = every term's part of the exponent; dg_t = sum of dG from t to the chunk's end
// and through the norm, dq = scale rq (dq^ - q~ (q~.dq^)), q~ = rq q.
//
// One workgroup takes a (chunk, value head); where value heads share a key head,
// their dq and dk are added up by a second kernel in a fixed order (holding the sums
// in registers over a workgroup's heads instead cost 212 bytes of scratch per lane
// and left a third of the workgroups).  Wave w owns
// the key channels 16 w .. 16 w + 15 for the products with S and D, so those are
// read and split into bf16 parts once, and a share of the tokens of row tile
// rt = w % 4 for everything else; the rows do, dR and u of 32 value channels at a
// time are split by their token's waves and handed round through LDS, two buffers
// in turn, with the next step's loads in flight.  4 x 2048 tokens, 16 heads of 128:
// 254 us for 2048 workgroups, one to a CU, a third of it reading S, D, u and dR
// (230 KB a workgroup) at the HBM rate.  64 x 64 products that meet a triangle
// take only the halves inside it.
#include "delta_device.h"

namespace ssm {
namespace {

constexpr int kLP = 68;  // floats per LDS row of a 64 x 64 matrix

// 8 consecutive values of such a row as an operand
__device__ __forceinline__ Frag<1> row_frag(const bf16s* p) {
  Frag<1> f;
  f.p[0] = *reinterpret_cast<const uint4*>(p);
  return f;
}
__device__ __forceinline__ Frag<3> row_frag(const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  return split8<3>(v);
}

// A k and a q value, in their own type
template <typename IN>
struct KQ;
template <>
struct KQ<bf16s> {
  uint32_t v;
  __device__ __forceinline__ void set(bf16s k, bf16s q) {
    v = static_cast<uint32_t>(k.bits) | static_cast<uint32_t>(q.bits) << 16;
  }
  __device__ __forceinline__ float k() const { return __uint_as_float(v << 16); }
  __device__ __forceinline__ float q() const { return __uint_as_float(v & 0xffff0000u); }
};
template <>
struct KQ<float> {
  float a, b;
  __device__ __forceinline__ void set(float k, float q) {
    a = k;
    b = q;
  }
  __device__ __forceinline__ float k() const { return a; }
  __device__ __forceinline__ float q() const { return b; }
};

// Sum over the 16 lanes of a row, in every lane of it
__device__ __forceinline__ float sum16(float x) {
  x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x128, 0xf, 0xf, false));
  x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x124, 0xf, 0xf, false));
  x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x122, 0xf, 0xf, false));
  x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x121, 0xf, 0xf, false));
  return x;
}
__device__ __forceinline__ float exp_of(double x) { return exp2_fast(static_cast<float>(x * 1.4426950408889634)); }

// 8 gradients from element i on; vec: all inside and aligned, else the first `left`
__device__ __forceinline__ void store8(void* p, size_t i, int dtype, bool vec, int left, const float (&v)[8]) {
  if (dtype == kBF16) {
    uint16_t* o = static_cast<uint16_t*>(p) + i;
    const uint32_t w[4] = {pack_rne(v[0], v[1]), pack_rne(v[2], v[3]), pack_rne(v[4], v[5]), pack_rne(v[6], v[7])};
    if (vec) {
      *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) o[e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
    }
  } else {
    float* o = static_cast<float*>(p) + i;
    if (vec) {
      reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) o[e] = v[e];
    }
  }
}

// VEC: rows of q, k, v, do, dq, dk and dv take 16-byte accesses (else element by element).
template <typename IN, int KP, bool VEC>
__global__ __launch_bounds__(KP * 4, KP / 64) void delta_grads_kernel(DeltaArgs a, int grad_dtype) {
  using Parts = DeltaParts<IN>;
  constexpr int NI = Parts::in, NS = Parts::state;
  constexpr int ND = KP / 32, NW = KP / 16, NT = 64 * NW;  // a wave per 16 key channels
  constexpr int JT = 16 / NW;                              // column tiles (and, halved, token steps) per wave of a row tile
  constexpr int kDo = 4 * NI * kDeltaFrag, kRow = 4 * NS * kDeltaFrag;
  constexpr int kStage = kDo + 2 * kRow;
  __shared__ __align__(16) unsigned char stage[2 * kStage];
  __shared__ __align__(16) float WM[2 * kDeltaC * kLP];
  float* const Wm = WM;
  float* const Mm = WM + kDeltaC * kLP;
  __shared__ float kkq[2][kDeltaC * kLP];   // k k^T, scale q k^T, with the norms
  __shared__ float rowp[NW][2][kDeltaC];
  __shared__ float colx[4][kDeltaC];
  __shared__ __align__(16) float sc[kDeltaSc];  // the head's coefficients
  __shared__ float rowx[NW / 4][kDeltaC], rowb[NW / 4][kDeltaC], rowv[kDeltaC], sdots[NW], csums[NW];
  // after the last step the staging holds W and M as operands
  unsigned char* const wf = stage;                                     // rows of W: lower triangle
  unsigned char* const cf = stage + kDeltaTri * NS * kDeltaFrag;       // columns of W: upper triangle
  unsigned char* const nf = stage;                                     // M + M^T, all 8

  const long slot = blockIdx.x / a.h;
  const int head = static_cast<int>(blockIdx.x - slot * a.h);
  const int rep = a.h / a.hk, kh = head / rep;
  long t0 = 0;
  const int n = delta_chunk(a, slot, &t0);
  if (n == 0) return;
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6), r = lane & 15, q = lane >> 4;
  const int rt = w & 3, hf = w >> 2;  // this wave's row tile, and its share of that tile's work
  const int vp = delta_vp(a.V), steps = vp / 32;
  const size_t kc = static_cast<size_t>(slot) * a.hk + kh;
  const size_t kbytes = 4 * ND * NI * kDeltaFrag;
  const unsigned char* ktf = a.ktf + kc * kbytes;
  const unsigned char* qtf = a.qtf + kc * kbytes;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};

  // the chunk's q and k rows, through the staging (zeros past the ends)
  constexpr int pitch = KP + 16 / static_cast<int>(sizeof(IN));
  static_assert(2 * kDeltaC * pitch * static_cast<int>(sizeof(IN)) <= 2 * kStage, "q and k rows fit the staging");
  IN* const Ks = reinterpret_cast<IN*>(stage);
  IN* const Qs = Ks + kDeltaC * pitch;
  {
    constexpr int per = KP / 8, each = kDeltaC * per / NT;
    Row8<IN> rk[each], rq[each];
#pragma unroll
    for (int i = 0; i < each; ++i) {
      const int p = tid + NT * i, t = p / per, d = (p % per) * 8;
      const long tt = t0 + (t < n ? t : 0), off = static_cast<long>(kh) * a.K;
      rk[i].load(static_cast<const IN*>(a.k) + tt * a.k_stride + off, d, a.K, VEC);
      rq[i].load(static_cast<const IN*>(a.q) + tt * a.q_stride + off, d, a.K, VEC);
    }
#pragma unroll
    for (int i = 0; i < each; ++i) {
      const int p = tid + NT * i, t = p / per, d = (p % per) * 8;
      float v[8];
      rk[i].get(t < n ? a.K - d : 0, v);
      put8(Ks + t * pitch + d, v);
      rq[i].get(t < n ? a.K - d : 0, v);
      put8(Qs + t * pitch + d, v);
    }
  }
  __syncthreads();
  // q and k at this wave's channels, all tokens, in the accumulators' layout
  KQ<IN> kq[4][4];
  f32x4 dqa[4], dka[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    dqa[i] = dka[i] = zero;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int at = (16 * i + 4 * q + e) * pitch + 16 * w + r;
      kq[i][e].set(Ks[at], Qs[at]);
    }
  }
  {  // the products of k and q with k wait in LDS for their use
    const float* nrm = a.sc + (static_cast<size_t>(slot) * a.h + head) * kDeltaSc;
    f32x4 kk[JT], qk[JT];
#pragma unroll
    for (int j = 0; j < JT; ++j) kk[j] = qk[j] = zero;
#pragma unroll
    for (int c = 0; c < ND; ++c) {
      const int off = 32 * c + 8 * q;
      const Frag<NI> fk = row_frag(Ks + (16 * rt + r) * pitch + off), fq = row_frag(Qs + (16 * rt + r) * pitch + off);
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        const Frag<NI> b = row_frag(Ks + (16 * (hf * JT + j) + r) * pitch + off);
        kk[j] = mma(fk, b, kk[j]);
        qk[j] = mma(fq, b, qk[j]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * rt + 4 * q + i;
      const float rk = nrm[kScRk * kDeltaC + t], rq = a.scale * nrm[kScRq * kDeltaC + t];
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        const int s = 16 * (hf * JT + j) + r;
        const float rks = nrm[kScRk * kDeltaC + s];
        kkq[0][t * kLP + s] = rk * rks * kk[j][i];
        kkq[1][t * kLP + s] = rq * rks * qk[j][i];
      }
    }
  }
  __syncthreads();

  {
    const size_t hc = static_cast<size_t>(slot) * a.h + head;
    constexpr int kScEach = (kDeltaSc + NT - 1) / NT;
    float scr[kScEach];
#pragma unroll
    for (int i = 0; i < kScEach; ++i) scr[i] = a.sc[hc * kDeltaSc + min(tid + NT * i, kDeltaSc - 1)];
    const double* G = reinterpret_cast<const double*>(sc + kScG * kDeltaC);
    const int trow = 16 * rt + r;  // this lane's token as an operand's row
    const bool live = trow < n;
    const size_t orow = (static_cast<size_t>(t0 + (live ? trow : 0)) * a.h + head) * a.V;
    const IN* const dorow = static_cast<const IN*>(a.dout) + orow;
    const IN* const vrow = static_cast<const IN*>(a.v) + (t0 + (live ? trow : 0)) * a.v_stride + static_cast<long>(head) * a.V;
    const float* const urow = a.u_chunk + (hc * kDeltaC + trow) * vp;
    const float* const rrow = NW == 4 || hf == 0 ? a.dr_chunk + (hc * kDeltaC + trow) * vp : urow;
    const float* const srow = a.s_chunk + (hc * KP + 16 * w + r) * vp;
    const float* const grow = a.ds_chunk + (hc * KP + 16 * w + r) * vp;

    f32x4 sdo[4], sdr[4], dsu[4], dp[JT], dl[JT];
#pragma unroll
    for (int i = 0; i < 4; ++i) sdo[i] = sdr[i] = dsu[i] = zero;
#pragma unroll
    for (int j = 0; j < JT; ++j) dp[j] = dl[j] = zero;
    float sdot = 0.0f, drv = 0.0f;
    const float brow = a.sc[hc * kDeltaSc + kScBeta * kDeltaC + trow];

    // the rows of a tile: do, dR and v by its first wave, u by its last
    const bool first = hf == 0;
    Row8<IN> ldo, lv;
    Row8<float> lr, lu, ls, ld;  // (with two waves to a tile lr holds dR in one, u in the other)
    auto load_step = [&](int c) {
      const int vc = 32 * c + 8 * q;
      if (first) {
        ldo.load(dorow, vc, a.V, VEC);
        lv.load(vrow, vc, a.V, VEC);
      }
      lr.load(rrow, vc, vp, true);
      if (NW == 4) lu.load(urow, vc, vp, true);
      ls.load(srow, vc, vp, true);
      ld.load(grow, vc, vp, true);
    };
    load_step(0);
#pragma unroll
    for (int i = 0; i < kScEach; ++i)  // (seen by all after the first step's barrier)
      if (tid + NT * i < kDeltaSc) sc[tid + NT * i] = scr[i];
#pragma unroll 1
    for (int c = 0; c < steps; ++c) {
      unsigned char* const sdf = stage + (c & 1) * kStage;
      unsigned char* const srf = sdf + kDo;
      unsigned char* const suf = srf + kRow;
      const int vc = 32 * c + 8 * q, left = live ? a.V - vc : 0;
      float x8[8], y8[8];
      if (first) {
        ldo.get(left, x8);
        store_frag<NI>(sdf, rt, lane, split8<NI>(x8));
      }
      lr.get(8, x8);
      store_frag<NS>(NW == 4 || hf == 0 ? srf : suf, rt, lane, split8<NS>(x8));
      if (first) {
        lv.get(left, y8);
#pragma unroll
        for (int i = 0; i < 8; ++i) drv = fmaf(x8[i], y8[i], drv);
        if (a.dv && left > 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x8[i] *= brow;
          store8(a.dv, orow + vc, grad_dtype, VEC, left, x8);
        }
      }
      if (NW == 4) {
        lu.get(8, x8);
        store_frag<NS>(suf, rt, lane, split8<NS>(x8));
      }
      ls.get(8, x8);
      ld.get(8, y8);
#pragma unroll
      for (int i = 0; i < 8; ++i) sdot = fmaf(x8[i], y8[i], sdot);
      const Frag<NS> fs = split8<NS>(x8), fd = split8<NS>(y8);
      load_step(min(c + 1, steps - 1));
      lds_barrier();
      const Frag<NI> mydo = load_frag<NI>(sdf, rt, lane);
      const Frag<NS> mydr = load_frag<NS>(srf, rt, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sdo[i] = mma(load_frag<NI>(sdf, i, lane), fs, sdo[i]);
        sdr[i] = mma(load_frag<NS>(srf, i, lane), fs, sdr[i]);
        dsu[i] = mma(load_frag<NS>(suf, i, lane), fd, dsu[i]);
      }
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        const Frag<NS> fu = load_frag<NS>(suf, hf * JT + j, lane);
        dp[j] = mma(mydo, fu, dp[j]);
        dl[j] = mma(mydr, fu, dl[j]);
      }
    }
    drv += __shfl_xor(drv, 16);
    drv += __shfl_xor(drv, 32);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) sdot += __shfl_xor(sdot, o);
    if (lane == 0) sdots[w] = sdot;
    if (first && q == 0) rowv[trow] = drv;

    {  // W, M and the exponents' parts in the 64 x 64 products: row tile rt
      float bt[4], rx[4] = {0, 0, 0, 0}, rb[4] = {0, 0, 0, 0};
      double Gt[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * rt + 4 * q + i;
        Gt[i] = G[t];
        bt[i] = sc[kScBeta * kDeltaC + t];
      }
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        const int s = 16 * (hf * JT + j) + r;
        const double Gs = G[s];
        float cx = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 16 * rt + 4 * q + i;
          const double diff = s <= t ? Gt[i] - Gs : -1e4;  // 0 above the diagonal, where e^{G_t - G_s} may overflow
          const float e = exp_of(diff);
          const float wv = s <= t ? dp[j][i] * e : 0.0f;
          const float le = s < t ? -dl[j][i] * e : 0.0f;  // dL E
          const float kkv = kkq[0][t * kLP + s];
          const float xv = wv * kkq[1][t * kLP + s] + le * bt[i] * kkv;
          Wm[t * kLP + s] = wv;
          Mm[t * kLP + s] = le * bt[i];
          rx[i] += xv;
          rb[i] = fmaf(le, kkv, rb[i]);
          cx += xv;
        }
        cx += __shfl_xor(cx, 16);
        cx += __shfl_xor(cx, 32);
        if (q == 0) colx[rt][s] = cx;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = sum16(rx[i]), y = sum16(rb[i]);
        if (r == 0) {
          rowx[hf][16 * rt + 4 * q + i] = x;
          rowb[hf][16 * rt + 4 * q + i] = y;
        }
      }
    }
    // the terms that meet the states, and their parts of the exponents
    float cs = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * i + 4 * q + e;
        const float gt = sc[kScEg * kDeltaC + t], el = sc[kScEl * kDeltaC + t], bt = sc[kScBeta * kDeltaC + t];
        const float rk = sc[kScRk * kDeltaC + t], rq = a.scale * sc[kScRq * kDeltaC + t];
        const float xq = gt * sdo[i][e], xr = gt * sdr[i][e], xu = el * dsu[i][e];
        float sa = kq[i][e].q() * xq, sb = kq[i][e].k() * xr;
        const float su = kq[i][e].k() * xu;
        dqa[i][e] += xq;
        dka[i][e] += xu - bt * xr;
        cs = fmaf(rk, su, cs);
        sa = sum16(rq * sa - rk * fmaf(bt, sb, su));
        sb = sum16(rk * sb);
        if (r == 0) {
          rowp[w][0][t] = sa;
          rowp[w][1][t] = sb;
        }
      }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) cs += __shfl_xor(cs, o);
    if (lane == 0) csums[w] = cs;
    __syncthreads();
    constexpr int SW = JT / 2;  // token steps of this wave's row tile
    float nn[SW][8];
#pragma unroll
    for (int x = 0; x < SW; ++x) {
      const int s = SW == 2 ? x : hf;
      float wr[8], wc[8];
      const int t = 16 * rt + r, k0 = 32 * s + 8 * q;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float rk = sc[kScRk * kDeltaC + k0 + i], rq = sc[kScRq * kDeltaC + k0 + i];
        wr[i] = Wm[t * kLP + k0 + i] * rk;
        wc[i] = Wm[(k0 + i) * kLP + t] * (a.scale * rq);
        nn[x][i] = (Mm[t * kLP + k0 + i] + Mm[(k0 + i) * kLP + t]) * rk;
      }
      if (s == 0 || rt >= 2) store_frag<NS>(wf, low_frag(rt, s), lane, split8<NS>(wr));
      if (s == 1 || rt < 2) store_frag<NS>(cf, up_frag(rt, s), lane, split8<NS>(wc));
    }
    Frag<NI> bk[2], bq[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      bk[s] = load_frag<NI>(ktf, 2 * w + s, lane);
      bq[s] = load_frag<NI>(qtf, 2 * w + s, lane);
    }
    // dbeta, and dg as the running sum from the chunk's end
    if (w == 3) {
      float av = 0.0f, bv = 0.0f, rx = 0.0f, rb = 0.0f;
      double cs = 0.0, sd = 0.0;
#pragma unroll
      for (int x = 0; x < NW; ++x) {
        av += rowp[x][0][lane];
        bv += rowp[x][1][lane];
        cs += csums[x];
        sd += sdots[x];
      }
#pragma unroll
      for (int x = 0; x < NW / 4; ++x) {
        rx += rowx[x][lane];
        rb += rowb[x][lane];
      }
      double g = static_cast<double>(av) + rx -
                 (static_cast<double>(colx[0][lane]) + colx[1][lane] + colx[2][lane] + colx[3][lane]);
      if (lane == kDeltaC - 1)
        g += cs + static_cast<double>(sc[kScGamma * kDeltaC]) * sd;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const double up = __shfl_down(g, o);
        if (lane + o < 64) g += up;
      }
      if (lane < n) {
        const size_t at = static_cast<size_t>(t0 + lane) * a.h + head;
        if (a.dg) a.dg[at] = static_cast<float>(g);
        if (a.dbeta) a.dbeta[at] = rowv[lane] + rb - bv;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (s <= i / 2) dqa[i] = mma(load_frag<NS>(wf, low_frag(i, s), lane), bk[s], dqa[i]);
        if (s >= i / 2) dka[i] = mma(load_frag<NS>(cf, up_frag(i, s), lane), bq[s], dka[i]);
      }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < SW; ++x) store_frag<NS>(nf, 2 * rt + (SW == 2 ? x : hf), lane, split8<NS>(nn[x]));
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s) dka[i] = mma(load_frag<NS>(nf, 2 * i + s, lane), bk[s], dka[i]);
    __syncthreads();
  }

  // through the norms, and out by whole rows; where heads share q and k, as they are
  // (per value head) for the kernel that adds them up
  if (rep == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float dq = sum16(kq[i][e].q() * dqa[i][e]), dk = sum16(kq[i][e].k() * dka[i][e]);
        if (r == 0) {
          rowp[w][0][16 * i + 4 * q + e] = dq;
          rowp[w][1][16 * i + 4 * q + e] = dk;
        }
      }
    __syncthreads();
  }
  constexpr int opitch = KP + 4;
  static_assert(kDeltaC * opitch <= 2 * kDeltaC * kLP, "a gradient's rows fit W and M");
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * i + 4 * q + e;
        float g = which ? dka[i][e] : dqa[i][e];
        if (rep == 1) {
          const float rr = sc[(which ? kScRk : kScRq) * kDeltaC + t];
          float dot = 0.0f;
#pragma unroll
          for (int x = 0; x < NW; ++x) dot += rowp[x][which][t];
          dot = a.qk_norm ? dot * rr * rr : 0.0f;
          g = (which ? 1.0f : a.scale) * rr * (g - (which ? kq[i][e].k() : kq[i][e].q()) * dot);
        }
        WM[t * opitch + 16 * w + r] = g;
      }
    __syncthreads();
    constexpr int per = KP / 8;
#pragma unroll
    for (int p = tid; p < kDeltaC * per; p += NT) {
      const int t = p / per, d = (p % per) * 8;
      const float4 x = *reinterpret_cast<const float4*>(WM + t * opitch + d);
      const float4 y = *reinterpret_cast<const float4*>(WM + t * opitch + d + 4);
      const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      if (t < n && d < a.K) {
        if (rep == 1) {
          void* const dst = which ? a.dk : a.dq;
          if (dst) store8(dst, (static_cast<size_t>(t0 + t) * a.hk + kh) * a.K + d, grad_dtype, VEC, a.K - d, v);
        } else {
          float* const dst = which ? a.dk_part : a.dq_part;  // rows padded to KP
          store8(dst, (static_cast<size_t>(t0 + t) * a.h + head) * KP + d, kF32, true, 8, v);
        }
      }
    }
    __syncthreads();
  }
}

// dq and dk of heads that share them: the sum over a key head's value heads, in their
// order, and through the norms.  KP / 8 lanes per row, q's rows and then k's.
template <typename IN, int KP>
__global__ __launch_bounds__(256) void delta_heads_kernel(DeltaArgs a, int grad_dtype) {
  constexpr int LPR = KP / 8;
  const long row = (static_cast<long>(blockIdx.x) * 256 + threadIdx.x) / LPR;  // (token, key head)
  if (row >= a.tokens * a.hk) return;  // whole rows leave together
  const bool of_k = blockIdx.y != 0;
  void* const dst = of_k ? a.dk : a.dq;
  if (!dst) return;
  const long t = row / a.hk;
  if (a.cu && !delta_inside(a, t)) return;
  const int kh = static_cast<int>(row - t * a.hk), rep = a.h / a.hk, d = (threadIdx.x % LPR) * 8;
  const float* part = (of_k ? a.dk_part : a.dq_part) + (t * a.h + static_cast<long>(kh) * rep) * KP + d;
  float g[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (d < a.K)
    for (int h = 0; h < rep; ++h) {
      const float4 x = reinterpret_cast<const float4*>(part + static_cast<long>(h) * KP)[0];
      const float4 y = reinterpret_cast<const float4*>(part + static_cast<long>(h) * KP)[1];
      g[0] += x.x; g[1] += x.y; g[2] += x.z; g[3] += x.w;
      g[4] += y.x; g[5] += y.y; g[6] += y.z; g[7] += y.w;
    }
  float rr = 1.0f;
  if (a.qk_norm) {
    const IN* src = static_cast<const IN*>(of_k ? a.k : a.q) + t * (of_k ? a.k_stride : a.q_stride) + static_cast<long>(kh) * a.K;
    Row8<IN> raw;
    raw.load(src, d, a.K, a.vec_qk);
    float x[8], ss = 0.0f, dot = 0.0f;
    raw.get(a.K - d, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (d + i >= a.K) g[i] = 0.0f;  // (the padded columns hold zeros, or nothing)
      ss = fmaf(x[i], x[i], ss);
      dot = fmaf(x[i], g[i], dot);
    }
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) {
      ss += __shfl_xor(ss, o);
      dot += __shfl_xor(dot, o);
    }
    rr = 1.0f / sqrtf(ss + a.eps);
    dot *= rr * rr;
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = fmaf(-x[i], dot, g[i]);
  }
  const float f = of_k ? rr : a.scale * rr;
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] *= f;
  const bool vec = a.K % 8 == 0 && (reinterpret_cast<uintptr_t>(dst) & 15) == 0;
  if (d < a.K) store8(dst, static_cast<size_t>(row) * a.K + d, grad_dtype, vec, a.K - d, g);
}

template <typename IN, int KP>
hipError_t go(const DeltaLaunch& l, hipStream_t s) {
  const DeltaArgs& a = l.a;
  auto al16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const bool vec = a.vec_qk && a.V % 8 == 0 && a.v_stride % 8 == 0 && al16(a.v) && al16(a.dout) && al16(a.dv) &&
                   al16(a.dq) && al16(a.dk);
  const dim3 grid(static_cast<unsigned>(a.slots * a.h)), block(KP * 4);
  const hipError_t e = timed_launch(s, [&] {
    if (vec) hipLaunchKernelGGL((delta_grads_kernel<IN, KP, true>), grid, block, 0, s, a, l.grad_dtype);
    else hipLaunchKernelGGL((delta_grads_kernel<IN, KP, false>), grid, block, 0, s, a, l.grad_dtype);
  });
  if (e != hipSuccess || a.h == a.hk || (!a.dq && !a.dk)) return e;
  const long rows = 256 / (KP / 8);
  hipLaunchKernelGGL((delta_heads_kernel<IN, KP>), dim3(static_cast<unsigned>((a.tokens * a.hk + rows - 1) / rows), 2),
                     dim3(256), 0, s, a, l.grad_dtype);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_grads(const DeltaLaunch& l, hipStream_t s) {
  if (l.a.slots == 0) return hipSuccess;
  const bool small = delta_kp(l.a.K) == 64;
  if (l.in_dtype == kBF16) return small ? go<bf16s, 64>(l, s) : go<bf16s, 128>(l, s);
  return small ? go<float, 64>(l, s) : go<float, 128>(l, s);
}

}  // namespace ssm
