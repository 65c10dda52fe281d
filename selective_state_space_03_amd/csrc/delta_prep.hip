// The part of the chunked gated delta rule that does not depend on the state:
// per chunk of 64 tokens and value head, T = (I + L)^-1 and P (delta.h), and the
// chunk's q and k rows, all written as matrix operands in the order in which the
// walking kernels' lanes read them (1 KB per fragment and load), so those read
// operands straight into registers without staging, transposing or masking.
//
// Running sums of g are taken in 64 bits (differences G_t - G_s of a chunk that
// holds a reset, g very negative, would lose their digits in 32); the inverse in
// 32 bits: the four 16 x 16 diagonal blocks by substitution, one wave each, the
// blocks below them as T_ij = -T_ii sum_m L_im T_mj with 32-bit matrix
// instructions, first within the two halves, then between them.  q and k enter the products
// unscaled (bf16 rows are exact operands); the reciprocal norms, decays, gates
// and the readout scale are folded into L, P and per-token coefficients.
//
// Bound by latency (seven barriers and two substitutions' lengths a head) and by what
// it writes, 39.7 kB per chunk and head.  12289 packed tokens, 80 heads on 8 key heads,
// K 64: 222 us (671 MB written, 3.0 TB/s); 8192 tokens, 32 heads on 16, K 128: 83 us.
#include "delta_device.h"

namespace ssm {
namespace {

constexpr int kLP = 68;  // floats per LDS row of a 64 x 64 matrix
constexpr int kHeads = 8;  // value heads of a workgroup at most

// 8 values of an LDS tile as an operand: `lo` and `hi` point at 4 consecutive ones each
__device__ __forceinline__ Frag<1> frag44(const bf16s* lo, const bf16s* hi) {
  const uint2 a = *reinterpret_cast<const uint2*>(lo), b = *reinterpret_cast<const uint2*>(hi);
  Frag<1> f;
  f.p[0] = make_uint4(a.x, a.y, b.x, b.y);
  return f;
}
__device__ __forceinline__ Frag<3> frag44(const float* lo, const float* hi) {
  const float4 a = *reinterpret_cast<const float4*>(lo), b = *reinterpret_cast<const float4*>(hi);
  const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  return split8<3>(v);
}
// 8 values down a column
__device__ __forceinline__ Frag<1> frag_col(const bf16s* p, int pitch) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = static_cast<uint32_t>(p[2 * i * pitch].bits) | (static_cast<uint32_t>(p[(2 * i + 1) * pitch].bits) << 16);
  Frag<1> f;
  f.p[0] = make_uint4(w[0], w[1], w[2], w[3]);
  return f;
}
__device__ __forceinline__ Frag<3> frag_col(const float* p, int pitch) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = p[i * pitch];
  return split8<3>(v);
}

template <int NP>
__device__ __forceinline__ Frag<NP> frag_row(const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  return split8<NP>(v);
}
template <int NP>
__device__ __forceinline__ Frag<NP> frag_fcol(const float* p) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = p[i * kLP];
  return split8<NP>(v);
}

// C = A B of 16 x 16 blocks in LDS, 32-bit matrix instructions
__device__ __forceinline__ f32x4 mma16(const float* A, const float* B, int r, int q, f32x4 acc) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(A[r * kLP + 4 * k + q], B[(4 * k + q) * kLP + r], acc, 0, 0, 0);
  return acc;
}

__device__ __forceinline__ float exp_of(double x) { return exp2_fast(static_cast<float>(x * 1.4426950408889634)); }

template <typename IN, int KP, bool BWD>
__global__ __launch_bounds__(256, 2) void delta_prep_kernel(DeltaArgs a, int parts) {
  using Parts = DeltaParts<IN>;
  constexpr int NI = Parts::in, NS = Parts::state;
  constexpr int ND = KP / 32;                              // 32-channel steps
  constexpr int pitch = KP + 16 / static_cast<int>(sizeof(IN));
  constexpr int tile = kDeltaC * pitch * static_cast<int>(sizeof(IN));
  constexpr int mat = kDeltaC * kLP * 4;
  __shared__ __align__(16) unsigned char qk_raw[2 * tile > mat ? 2 * tile : mat];
  __shared__ __align__(16) float Lm[kDeltaC * kLP];
  __shared__ double Gs[kHeads][kDeltaC];
  __shared__ float bs[kHeads][kDeltaC], rks[kDeltaC], rqs[kDeltaC];
  IN* const Ks = reinterpret_cast<IN*>(qk_raw);
  IN* const Qs = reinterpret_cast<IN*>(qk_raw + tile);
  // after the last use of Ks and Qs their room holds a head's P, then its T
  float* const Pm = reinterpret_cast<float*>(qk_raw);
  float* const Tm = Pm;

  const unsigned groups = static_cast<unsigned>(a.hk) * parts;
  const long slot = blockIdx.x / groups;
  const int kp = static_cast<int>(blockIdx.x - slot * groups);
  const int kh = kp / parts, part = kp - kh * parts;
  const int rep = a.h / a.hk;
  const int h0 = kh * rep + static_cast<int>(static_cast<long>(part) * rep / parts);
  const int h1 = kh * rep + static_cast<int>(static_cast<long>(part + 1) * rep / parts);
  long t0 = 0;
  const int n = delta_chunk(a, slot, &t0);
  if (n == 0) return;
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6), r = lane & 15, q = lane >> 4;

  // the heads' running sums of g, in 64 bits, a head per wave at a time
  const size_t grow = static_cast<size_t>(t0 + (lane < n ? lane : 0)) * a.h;
  for (int head = h0 + w; head < h1; head += 4) {
    const float gl = a.g[grow + head], bl = a.beta[grow + head];
    double g = lane < n ? static_cast<double>(gl) : 0.0;
    g = g < -1e4 ? -1e4 : g;  // e^-10000 is 0 in 32 bits already; -inf would make differences NaN
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const double up = __shfl_up(g, o);
      if (lane >= o) g += up;
    }
    Gs[head - h0][lane] = g;
    bs[head - h0][lane] = lane < n ? bl : 0.0f;
  }
  // the chunk's q and k rows, zeros past its end and past K
  {
    constexpr int per = KP / 8, each = kDeltaC * per / 256;
    Row8<IN> rk[each], rq[each];
#pragma unroll
    for (int i = 0; i < each; ++i) {
      const int p = tid + 256 * i, t = p / per, d = (p % per) * 8;
      const long tt = t0 + (t < n ? t : 0), off = static_cast<long>(kh) * a.K;
      rk[i].load(static_cast<const IN*>(a.k) + tt * a.k_stride + off, d, a.K, a.vec_qk);
      rq[i].load(static_cast<const IN*>(a.q) + tt * a.q_stride + off, d, a.K, a.vec_qk);
    }
#pragma unroll
    for (int i = 0; i < each; ++i) {
      const int p = tid + 256 * i, t = p / per, d = (p % per) * 8;
      float v[8], u[8], sk = 0.0f, sq = 0.0f;
      rk[i].get(t < n ? a.K - d : 0, v);
      rq[i].get(t < n ? a.K - d : 0, u);
      put8(Ks + t * pitch + d, v);
      put8(Qs + t * pitch + d, u);
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        sk = fmaf(v[x], v[x], sk);
        sq = fmaf(u[x], u[x], sq);
      }
#pragma unroll
      for (int o = 1; o < per; o <<= 1) {
        sk += __shfl_xor(sk, o);
        sq += __shfl_xor(sq, o);
      }
      if (d == 0) {
        // (0 past the chunk's end: with eps = 0 a row of zeros has no reciprocal norm)
        rks[t] = t >= n ? 0.0f : a.qk_norm ? 1.0f / sqrtf(sk + a.eps) : 1.0f;
        rqs[t] = t >= n ? 0.0f : a.qk_norm ? 1.0f / sqrtf(sq + a.eps) : 1.0f;
      }
    }
  }
  __syncthreads();

  // k k^T and q k^T on the ten 16 x 16 tiles of the lower triangle: three for waves 0
  // and 1, two for waves 2 and 3 (whose third repeats their first, unused: no branch
  // among the products)
  const int nt = w < 2 ? 3 : 2;
  const int ti[3] = {w, w < 3 ? w + 1 : 2, w < 2 ? 3 : w}, tj[3] = {w, w < 3 ? w : 0, w};
  f32x4 kk[3], qk[3];
#pragma unroll
  for (int j = 0; j < 3; ++j) kk[j] = qk[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int c = 0; c < ND; ++c) {
    const int off = 32 * c + 8 * q;
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const IN* rk = Ks + (16 * ti[j] + r) * pitch + off;
      const IN* rq = Qs + (16 * ti[j] + r) * pitch + off;
      const IN* rb = Ks + (16 * tj[j] + r) * pitch + off;
      const Frag<NI> b = frag44(rb, rb + 4);
      kk[j] = mma(frag44(rk, rk + 4), b, kk[j]);
      qk[j] = mma(frag44(rq, rq + 4), b, qk[j]);
    }
  }
  // norms and the readout scale go into the products, which every head shares
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const float rs = rks[16 * tj[j] + r];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * ti[j] + 4 * q + i;
      kk[j][i] *= rks[t] * rs;
      qk[j][i] *= a.scale * rqs[t] * rs;
    }
  }
  // operands shared by the key head's value heads
  if (part == 0) {
    const size_t at = static_cast<size_t>(slot) * a.hk + kh;
    constexpr size_t bytes = 4 * ND * NI * kDeltaFrag;
#pragma unroll
    for (int c = 0; c < ND; ++c) {
      const int o = (16 * w + r) * pitch + 32 * c + 4 * q;
      store_frag<NI>(a.kf + at * bytes, w * ND + c, lane, frag44(Ks + o, Ks + o + 16));
      if (!BWD) store_frag<NI>(a.qf + at * bytes, w * ND + c, lane, frag44(Qs + o, Qs + o + 16));
    }
#pragma unroll
    for (int ct = w; ct < KP / 16; ct += 4)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int o = (32 * s + 8 * q) * pitch + 16 * ct + r;
        store_frag<NI>(a.ktf + at * bytes, 2 * ct + s, lane, frag_col(Ks + o, pitch));
        if (BWD) store_frag<NI>(a.qtf + at * bytes, 2 * ct + s, lane, frag_col(Qs + o, pitch));
      }
  }

#pragma unroll 1
  for (int head = h0; head < h1; ++head) {
    const size_t at = static_cast<size_t>(slot) * a.h + head;
    const double* const Gh = Gs[head - h0];
    const float* const bh = bs[head - h0];
    if (w == 3) {
      float* const sc = a.sc + at * kDeltaSc;
      const double g = Gh[lane], GC = Gh[kDeltaC - 1];
      const float eg = exp_of(g), el = exp_of(GC - g), rk = rks[lane], rq = rqs[lane], b = bh[lane];
      sc[kScBeta * kDeltaC + lane] = b;
      sc[kScR * kDeltaC + lane] = b * eg * rk;
      sc[kScO * kDeltaC + lane] = a.scale * eg * rq;
      sc[kScU * kDeltaC + lane] = el * rk;
      sc[kScEg * kDeltaC + lane] = eg;
      sc[kScEl * kDeltaC + lane] = el;
      sc[kScRk * kDeltaC + lane] = rk;
      sc[kScRq * kDeltaC + lane] = rq;
      reinterpret_cast<double*>(sc + kScG * kDeltaC)[lane] = g;
      if (lane == 0) sc[kScGamma * kDeltaC] = exp_of(GC);
    }
    __syncthreads();  // the room of q and k (or of the head before) is free
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (j < nt) {
        const int s = 16 * tj[j] + r;
        const double Gsv = Gh[s];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 16 * ti[j] + 4 * q + i;
          // 0 above the diagonal, where the decay may overflow
          const float dec = exp_of(s <= t ? Gh[t] - Gsv : -1e4);
          Lm[t * kLP + s] = s < t ? bh[t] * dec * kk[j][i] : 0.0f;
          Pm[t * kLP + s] = s <= t ? dec * qk[j][i] : 0.0f;
        }
      }
    // tiles above the diagonal that an operand's step spans: (0, 1) and (2, 3)
    if (w >= 2)
#pragma unroll
      for (int i = 0; i < 4; ++i) Pm[(32 * (w - 2) + 4 * q + i) * kLP + 32 * (w - 2) + 16 + r] = 0.0f;
    __syncthreads();
    if (!BWD) {
      unsigned char* pf = a.pf + at * (kDeltaTri * NS * kDeltaFrag);
      for (int s = 0; s <= (w >> 1); ++s)
        store_frag<NS>(pf, low_frag(w, s), lane, frag_row<NS>(Pm + (16 * w + r) * kLP + 32 * s + 8 * q));
    } else {
      unsigned char* ptf = a.ptf + at * (kDeltaTri * NS * kDeltaFrag);
      for (int s = w >> 1; s < 2; ++s)
        store_frag<NS>(ptf, up_frag(w, s), lane, frag_fcol<NS>(Pm + (32 * s + 8 * q) * kLP + 16 * w + r));
    }
    // the diagonal blocks of T by substitution: column r of block w's inverse in
    // every 16-lane row of the wave; x[m] leaves the later rows' sums as soon as it is known
    float x[16];
    {
      const float* Lw = Lm + 16 * w * kLP + 16 * w;
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = i == r ? 1.0f : 0.0f;
#pragma unroll
      for (int m4 = 0; m4 < 4; ++m4) {  // four of L's columns at a time
        float Lr[16][4];
#pragma unroll
        for (int i = 1; i < 16; ++i)
          if (i > 4 * m4) {
            const float4 f = *reinterpret_cast<const float4*>(Lw + i * kLP + 4 * m4);
            Lr[i][0] = f.x; Lr[i][1] = f.y; Lr[i][2] = f.z; Lr[i][3] = f.w;
          }
#pragma unroll
        for (int mm = 0; mm < 4; ++mm)
#pragma unroll
          for (int i = 1; i < 16; ++i)
            if (i > 4 * m4 + mm) x[i] = fmaf(-Lr[i][mm], x[4 * m4 + mm], x[i]);
        __builtin_amdgcn_sched_barrier(0);  // keeps the next columns' loads out of these registers
      }
    }
    __syncthreads();  // P is out
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((i >> 2) == q) Tm[(16 * w + i) * kLP + 16 * w + r] = x[i];
    // blocks above the diagonal are read as operands where a step spans them
#pragma unroll
    for (int j = 1; j < 4; ++j)
      if (j > w)
#pragma unroll
        for (int i = 0; i < 4; ++i) Tm[(16 * w + 4 * q + i) * kLP + 16 * j + r] = 0.0f;
    __syncthreads();
    // then T_ij = -T_ii sum_m L_im T_mj: the blocks (1, 0) and (3, 2), then the
    // 32 x 32 block below the two halves, a wave per 16 x 16 block
    const f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
    {
      const int i = w | 1, j = i - 1;  // waves 0, 1: block (1, 0); waves 2, 3: block (3, 2)
      const f32x4 sum = mma16(Lm + 16 * i * kLP + 16 * j, Tm + 16 * j * kLP + 16 * j, r, q, z);
      // (L's own block holds the sum now: both waves of a block write the same values)
#pragma unroll
      for (int e = 0; e < 4; ++e) Tm[(16 * i + 4 * q + e) * kLP + 16 * j + r] = -sum[e];
      __syncthreads();
      const f32x4 t = mma16(Tm + 16 * i * kLP + 16 * i, Tm + 16 * i * kLP + 16 * j, r, q, z);
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 4; ++e) Tm[(16 * i + 4 * q + e) * kLP + 16 * j + r] = t[e];
      __syncthreads();
    }
    {
      const int i = 2 + (w >> 1), j = w & 1;
      f32x4 sum = mma16(Lm + 16 * i * kLP, Tm + 16 * j, r, q, z);
      sum = mma16(Lm + 16 * i * kLP + 16, Tm + 16 * kLP + 16 * j, r, q, sum);
#pragma unroll
      for (int e = 0; e < 4; ++e) Tm[(16 * i + 4 * q + e) * kLP + 16 * j + r] = -sum[e];
      __syncthreads();
      f32x4 t = mma16(Tm + 16 * i * kLP + 32, Tm + 32 * kLP + 16 * j, r, q, z);
      t = mma16(Tm + 16 * i * kLP + 48, Tm + 48 * kLP + 16 * j, r, q, t);
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 4; ++e) Tm[(16 * i + 4 * q + e) * kLP + 16 * j + r] = t[e];
      __syncthreads();
    }
    unsigned char* tf = a.tf + at * (kDeltaTri * NS * kDeltaFrag);
    for (int s = 0; s <= (w >> 1); ++s)
      store_frag<NS>(tf, low_frag(w, s), lane, frag_row<NS>(Tm + (16 * w + r) * kLP + 32 * s + 8 * q));
    if (BWD) {
      unsigned char* ttf = a.ttf + at * (kDeltaTri * NS * kDeltaFrag);
      for (int s = w >> 1; s < 2; ++s)
        store_frag<NS>(ttf, up_frag(w, s), lane, frag_fcol<NS>(Tm + (32 * s + 8 * q) * kLP + 16 * w + r));
    }
  }
}

// Workgroups per (chunk, key head): the value heads share the rows and their
// products, so a workgroup takes as many (up to kHeads) as leave the GPU's CUs eight
// workgroups each (five heads each at the packed call above 222 us, one 351 us; two
// at the prompt 83 us, one 107 us).
int head_parts(const DeltaArgs& a) {
  const long rep = a.h / a.hk, want = 8L * 256, have = a.slots * a.hk;
  const long parts = (want + have - 1) / have, least = (rep + kHeads - 1) / kHeads;
  return static_cast<int>(parts > rep ? rep : parts < least ? least : parts);
}

template <typename IN, int KP>
hipError_t go(const DeltaLaunch& l, bool bwd, hipStream_t s) {
  const int parts = head_parts(l.a);
  const dim3 grid(static_cast<unsigned>(l.a.slots * l.a.hk * parts));
  if (bwd)
    hipLaunchKernelGGL((delta_prep_kernel<IN, KP, true>), grid, dim3(256), 0, s, l.a, parts);
  else
    hipLaunchKernelGGL((delta_prep_kernel<IN, KP, false>), grid, dim3(256), 0, s, l.a, parts);
  return hipGetLastError();
}

template <typename IN>
hipError_t pick(const DeltaLaunch& l, bool bwd, hipStream_t s) {
  return delta_kp(l.a.K) == 64 ? go<IN, 64>(l, bwd, s) : go<IN, 128>(l, bwd, s);
}

}  // namespace

hipError_t launch_delta_prep(const DeltaLaunch& l, bool backward, hipStream_t s) {
  if (l.a.slots == 0) return hipSuccess;
  return l.in_dtype == kBF16 ? pick<bf16s>(l, backward, s) : pick<float>(l, backward, s);
}

}  // namespace ssm
