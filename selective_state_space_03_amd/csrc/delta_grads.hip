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
// One workgroup takes a (chunk, key head) and its value heads in turn, so the
// shared heads' dq and dk are summed in registers in a fixed order.  Wave w
// computes the tokens 16 w .. 16 w + 15.  Bound by the splitting of the 32-bit
// operands (S, D, u, dR) into bf16 parts and the matrix products on them.
#include "delta_device.h"

namespace ssm {
namespace {

constexpr int kLP = 68;

// 8 consecutive values from column c of a row of `width` 32-bit values
__device__ __forceinline__ void row8f(const float* row, int c, int width, bool ok, bool vec, float (&v)[8]) {
  if (vec) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 r = load16_if(row + c + 4 * h, ok && c + 4 * h < width);
      v[4 * h] = __uint_as_float(r.x); v[4 * h + 1] = __uint_as_float(r.y);
      v[4 * h + 2] = __uint_as_float(r.z); v[4 * h + 3] = __uint_as_float(r.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = ok && c + i < width ? row[c + i] : 0.0f;
  }
}
// the same of the inputs' type, 4-element accesses where vec
__device__ __forceinline__ void row8i(const float* row, int c, int width, bool ok, bool vec, float (&v)[8]) {
  row8f(row, c, width, ok, vec, v);
}
__device__ __forceinline__ void row8i(const bf16s* row, int c, int width, bool ok, bool vec, float (&v)[8]) {
  if (vec) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint2 r = make_uint2(0u, 0u);
      if (ok && c + 4 * h < width) r = *reinterpret_cast<const uint2*>(row + c + 4 * h);
      v[4 * h] = __uint_as_float(r.x << 16); v[4 * h + 1] = __uint_as_float(r.x & 0xffff0000u);
      v[4 * h + 2] = __uint_as_float(r.y << 16); v[4 * h + 3] = __uint_as_float(r.y & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = ok && c + i < width ? to_f32(row[c + i]) : 0.0f;
  }
}

__device__ __forceinline__ float sum16(float x) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) x += __shfl_xor(x, o);
  return x;
}
__device__ __forceinline__ float exp_of(double x) { return exp2_fast(static_cast<float>(x * 1.4426950408889634)); }

__device__ __forceinline__ void put_grad(void* p, size_t i, int dtype, float v) {
  if (dtype == kBF16) st<bf16s>(p, i, v);
  else st<float>(p, i, v);
}

template <typename IN, int KP>
__global__ __launch_bounds__(256) void delta_grads_kernel(DeltaArgs a, int grad_dtype, int vec_v, int vec_in) {
  using Parts = DeltaParts<IN>;
  constexpr int NI = Parts::in, NS = Parts::state;
  constexpr int ND = KP / 32, NT = KP / 16;
  __shared__ __align__(16) float Wm[kDeltaC * kLP];
  __shared__ __align__(16) float Mm[kDeltaC * kLP];
  __shared__ float colx[4][kDeltaC];
  __shared__ float rowg[kDeltaC], rowb[kDeltaC], rowv[kDeltaC], rowc[kDeltaC];
  __shared__ float sdots[4];

  const long slot = blockIdx.x / a.hk;
  const int kh = static_cast<int>(blockIdx.x - slot * a.hk);
  const int rep = a.h / a.hk;
  long t0 = 0;
  const int n = delta_chunk(a, slot, &t0);
  if (n == 0) return;
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6), r = lane & 15, q = lane >> 4;
  const size_t kc = static_cast<size_t>(slot) * a.hk + kh;
  const unsigned char* kf = a.kf + kc * (4 * ND * NI * kDeltaFrag);
  const unsigned char* qf = a.qf + kc * (4 * ND * NI * kDeltaFrag);
  const unsigned char* ktf = a.ktf + kc * (4 * ND * NI * kDeltaFrag);
  const unsigned char* qtf = a.qtf + kc * (4 * ND * NI * kDeltaFrag);
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};

  // q, k in the accumulators' layout, and the products of k and q with k
  f32x4 kC[NT], qC[NT], dqa[NT], dka[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    dqa[j] = dka[j] = zero;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * w + 4 * q + i, d = 16 * j + r;
      const bool ok = t < n && d < a.K;
      const long tt = t0 + (ok ? t : 0);
      const long off = static_cast<long>(kh) * a.K + (ok ? d : 0);
      kC[j][i] = ok ? to_f32(static_cast<const IN*>(a.k)[tt * a.k_stride + off]) : 0.0f;
      qC[j][i] = ok ? to_f32(static_cast<const IN*>(a.q)[tt * a.q_stride + off]) : 0.0f;
    }
  }
  f32x4 kk[4], qk[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) kk[j] = qk[j] = zero;
#pragma unroll
  for (int c = 0; c < ND; ++c) {
    const Frag<NI> fk = load_frag<NI>(kf, w * ND + c, lane), fq = load_frag<NI>(qf, w * ND + c, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j <= w) {
        const Frag<NI> b = load_frag<NI>(kf, j * ND + c, lane);
        kk[j] = mma(fk, b, kk[j]);
        qk[j] = mma(fq, b, qk[j]);
      }
  }

  for (int hr = 0; hr < rep; ++hr) {
    const int head = kh * rep + hr;
    const size_t hc = static_cast<size_t>(slot) * a.h + head;
    const float* sc = a.sc + hc * kDeltaSc;
    const double* G = reinterpret_cast<const double*>(sc + kScG * kDeltaC);
    const float* Sg = a.s_chunk + hc * a.K * a.V;
    const float* Dg = a.ds_chunk + hc * a.K * a.V;
    const float* Ug = a.u_chunk + hc * kDeltaC * a.V;
    const float* Rg = a.dr_chunk + hc * kDeltaC * a.V;
    const int trow = 16 * w + r;  // this lane's token as an operand's row
    const size_t orow = (static_cast<size_t>(t0 + (trow < n ? trow : 0)) * a.h + head) * a.V;
    const IN* vrow = static_cast<const IN*>(a.v) + (t0 + (trow < n ? trow : 0)) * a.v_stride + static_cast<long>(head) * a.V;

    f32x4 sdo[NT], sdr[NT], dsu[NT], dp[4], dl[4];
#pragma unroll
    for (int j = 0; j < NT; ++j) sdo[j] = sdr[j] = dsu[j] = zero;
#pragma unroll
    for (int j = 0; j < 4; ++j) dp[j] = dl[j] = zero;
    float sdot = 0.0f, drv = 0.0f;
    const float brow = sc[kScBeta * kDeltaC + trow];
#pragma unroll 1
    for (int c = 0; c < a.V; c += 32) {
      const int vc = c + 8 * q;
      float x[8], y[8];
      row8i(static_cast<const IN*>(a.dout) + orow, vc, a.V, trow < n, vec_in, x);
      const Frag<NI> fdo = split8<NI>(x);
      row8f(Rg + static_cast<size_t>(trow) * a.V, vc, a.V, true, vec_v, x);
      const Frag<NS> fdr = split8<NS>(x);
      row8i(vrow, vc, a.V, trow < n, vec_in, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        drv = fmaf(x[i], y[i], drv);
        if (a.dv && trow < n && vc + i < a.V) put_grad(a.dv, orow + vc + i, grad_dtype, brow * x[i]);
      }
      row8f(Ug + static_cast<size_t>(trow) * a.V, vc, a.V, true, vec_v, x);
      const Frag<NS> fu = split8<NS>(x);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= w) {
          row8f(Ug + static_cast<size_t>(16 * j + r) * a.V, vc, a.V, true, vec_v, x);
          const Frag<NS> b = split8<NS>(x);
          dp[j] = mma(fdo, b, dp[j]);
          dl[j] = mma(fdr, b, dl[j]);
        }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int d = 16 * j + r;
        row8f(Sg + static_cast<size_t>(d) * a.V, vc, a.V, d < a.K, vec_v, x);
        row8f(Dg + static_cast<size_t>(d) * a.V, vc, a.V, d < a.K, vec_v, y);
        if ((j & 3) == w)
#pragma unroll
          for (int i = 0; i < 8; ++i) sdot = fmaf(x[i], y[i], sdot);
        const Frag<NS> fs = split8<NS>(x), fd = split8<NS>(y);
        sdo[j] = mma(fdo, fs, sdo[j]);
        sdr[j] = mma(fdr, fs, sdr[j]);
        dsu[j] = mma(fu, fd, dsu[j]);
      }
    }
    drv += __shfl_xor(drv, 16);
    drv += __shfl_xor(drv, 32);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) sdot += __shfl_xor(sdot, o);
    if (lane == 0) sdots[w] = sdot;
    if (q == 0) rowv[trow] = drv;

    // W, M and the exponents' parts in the 64 x 64 products
    float gt[4], bt[4], rkt[4], rqt[4], rx[4] = {0, 0, 0, 0}, rb[4] = {0, 0, 0, 0};
    double Gt[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * w + 4 * q + i;
      Gt[i] = G[t];
      gt[i] = exp_of(Gt[i]);
      bt[i] = sc[kScBeta * kDeltaC + t];
      rkt[i] = sc[kScRk * kDeltaC + t];
      rqt[i] = sc[kScRq * kDeltaC + t];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int s = 16 * j + r;
      const double Gs = G[s];
      const float rks = sc[kScRk * kDeltaC + s];
      float cx = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * w + 4 * q + i;
        const float e = s <= t ? exp_of(Gt[i] - Gs) : 0.0f;
        const float wv = s <= t ? dp[j][i] * e : 0.0f;
        const float le = s < t ? -dl[j][i] * e : 0.0f;  // dL E
        const float kkv = rkt[i] * rks * kk[j][i];
        const float xv = wv * (a.scale * rqt[i] * rks * qk[j][i]) + le * bt[i] * kkv;
        Wm[t * kLP + s] = wv;
        Mm[t * kLP + s] = le * bt[i];
        rx[i] += xv;
        rb[i] = fmaf(le, kkv, rb[i]);
        cx += xv;
      }
      cx += __shfl_xor(cx, 16);
      cx += __shfl_xor(cx, 32);
      if (q == 0) colx[w][s] = cx;
    }
    // the terms that meet the states, and their parts of the exponents
    const double GC = G[kDeltaC - 1];
    float sa[4] = {0, 0, 0, 0}, sb[4] = {0, 0, 0, 0}, scx[4] = {0, 0, 0, 0};
    float el[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) el[i] = exp_of(GC - Gt[i]);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float xq = gt[i] * sdo[j][i], xr = gt[i] * sdr[j][i], xu = el[i] * dsu[j][i];
        sa[i] = fmaf(qC[j][i], xq, sa[i]);
        sb[i] = fmaf(kC[j][i], xr, sb[i]);
        scx[i] = fmaf(kC[j][i], xu, scx[i]);
        dqa[j][i] += xq;
        dka[j][i] += xu - bt[i] * xr;
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * w + 4 * q + i;
      const float av = sum16(sa[i]) * rqt[i] * a.scale, bv = sum16(sb[i]) * rkt[i], cv = sum16(scx[i]) * rkt[i];
      const float x = sum16(rx[i]), y = sum16(rb[i]);
      if (r == 0) {
        rowg[t] = av - bt[i] * bv - cv + x;
        rowc[t] = cv;
        rowb[t] = y - bv;
      }
    }
    __syncthreads();
    // products of W and M with the rows of k and q
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float wr[8], wc[8], nn[8];
      const int t = 16 * w + r, k0 = 32 * s + 8 * q;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float rk = sc[kScRk * kDeltaC + k0 + i], rq = sc[kScRq * kDeltaC + k0 + i];
        wr[i] = Wm[t * kLP + k0 + i] * rk;
        wc[i] = Wm[(k0 + i) * kLP + t] * (a.scale * rq);
        nn[i] = (Mm[t * kLP + k0 + i] + Mm[(k0 + i) * kLP + t]) * rk;
      }
      const Frag<NS> fw = split8<NS>(wr), fc = split8<NS>(wc), fn = split8<NS>(nn);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const Frag<NI> bk = load_frag<NI>(ktf, 2 * j + s, lane), bq = load_frag<NI>(qtf, 2 * j + s, lane);
        if (s == 0 || w >= 2) dqa[j] = mma(fw, bk, dqa[j]);
        if (s == 1 || w < 2) dka[j] = mma(fc, bq, dka[j]);
        dka[j] = mma(fn, bk, dka[j]);
      }
    }
    // dbeta, and dg as the running sum from the chunk's end
    if (w == 0) {
      double g = static_cast<double>(rowg[lane]) -
                 (static_cast<double>(colx[0][lane]) + colx[1][lane] + colx[2][lane] + colx[3][lane]);
      double cs = rowc[lane];
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) cs += __shfl_xor(cs, o);
      if (lane == kDeltaC - 1)
        g += cs + static_cast<double>(sc[kScGamma * kDeltaC]) * (static_cast<double>(sdots[0]) + sdots[1] + sdots[2] + sdots[3]);
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const double up = __shfl_down(g, o);
        if (lane + o < 64) g += up;
      }
      if (lane < n) {
        const size_t at = static_cast<size_t>(t0 + lane) * a.h + head;
        if (a.dg) a.dg[at] = static_cast<float>(g);
        if (a.dbeta) a.dbeta[at] = rowv[lane] + rowb[lane];
      }
    }
    __syncthreads();
  }

  // through the norms
  const float* sc = a.sc + (static_cast<size_t>(slot) * a.h + kh * rep) * kDeltaSc;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 16 * w + 4 * q + i;
    const float rq = sc[kScRq * kDeltaC + t], rk = sc[kScRk * kDeltaC + t];
    float dq = 0.0f, dk = 0.0f;
    if (a.qk_norm) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        dq = fmaf(qC[j][i], dqa[j][i], dq);
        dk = fmaf(kC[j][i], dka[j][i], dk);
      }
      dq = sum16(dq) * rq * rq;
      dk = sum16(dk) * rk * rk;
    }
    if (t < n) {
      const size_t at = (static_cast<size_t>(t0 + t) * a.hk + kh) * a.K;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int d = 16 * j + r;
        if (d < a.K) {
          if (a.dq) put_grad(a.dq, at + d, grad_dtype, a.scale * rq * (dqa[j][i] - qC[j][i] * dq));
          if (a.dk) put_grad(a.dk, at + d, grad_dtype, rk * (dka[j][i] - kC[j][i] * dk));
        }
      }
    }
  }
}

template <typename IN, int KP>
hipError_t go(const DeltaLaunch& l, hipStream_t s) {
  const DeltaArgs& a = l.a;
  const int vec_v = a.V % 4 == 0;
  const uintptr_t need = l.in_dtype == kBF16 ? 7 : 15;
  const int vec_in = vec_v && a.v_stride % 4 == 0 &&
                     ((reinterpret_cast<uintptr_t>(a.v) | reinterpret_cast<uintptr_t>(a.dout)) & need) == 0;
  hipLaunchKernelGGL((delta_grads_kernel<IN, KP>), dim3(static_cast<unsigned>(a.slots * a.hk)), dim3(256), 0, s, a,
                     l.grad_dtype, vec_v, vec_in);
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
