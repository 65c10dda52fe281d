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
// instructions, one diagonal after the other.  q and k enter the products
// unscaled (bf16 rows are exact operands); the reciprocal norms, decays, gates
// and the readout scale are folded into L, P and per-token coefficients.
#include "delta_device.h"

namespace ssm {
namespace {

constexpr int kLP = 68;  // floats per LDS row of a 64 x 64 matrix

template <typename IN>
__device__ __forceinline__ void row8(const IN* row, int d0, int K, bool vec, float (&v)[8]);

template <>
__device__ __forceinline__ void row8<bf16s>(const bf16s* row, int d0, int K, bool vec, float (&v)[8]) {
  if (vec) {
    const uint4 r = load16_if(row + d0, d0 < K);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = d0 + i < K ? to_f32(row[d0 + i]) : 0.0f;
  }
}
template <>
__device__ __forceinline__ void row8<float>(const float* row, int d0, int K, bool vec, float (&v)[8]) {
  if (vec) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 r = load16_if(row + d0 + 4 * h, d0 < K);
      v[4 * h] = __uint_as_float(r.x); v[4 * h + 1] = __uint_as_float(r.y);
      v[4 * h + 2] = __uint_as_float(r.z); v[4 * h + 3] = __uint_as_float(r.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = d0 + i < K ? row[d0 + i] : 0.0f;
  }
}

__device__ __forceinline__ void put8(bf16s* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_hi(v[0], v[1]), pack_hi(v[2], v[3]), pack_hi(v[4], v[5]), pack_hi(v[6], v[7]));
}
__device__ __forceinline__ void put8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

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
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaArgs a) {
  using Parts = DeltaParts<IN>;
  constexpr int NI = Parts::in, NS = Parts::state, NO = Parts::out;
  constexpr int ND = KP / 32;                              // 32-channel steps
  constexpr int pitch = KP + 16 / static_cast<int>(sizeof(IN));
  constexpr int tile = kDeltaC * pitch * static_cast<int>(sizeof(IN));
  constexpr int mat = kDeltaC * kLP * 4;
  __shared__ __align__(16) unsigned char qk_raw[2 * tile > mat ? 2 * tile : mat];
  __shared__ __align__(16) float Lm[kDeltaC * kLP];
  __shared__ __align__(16) float Tm[kDeltaC * kLP];
  __shared__ double Gs[kDeltaC];
  __shared__ float bs[kDeltaC], rks[kDeltaC], rqs[kDeltaC];
  IN* const Ks = reinterpret_cast<IN*>(qk_raw);
  IN* const Qs = reinterpret_cast<IN*>(qk_raw + tile);
  float* const Pm = reinterpret_cast<float*>(qk_raw);  // after the last use of Ks and Qs

  const long slot = blockIdx.x / a.h;
  const int head = static_cast<int>(blockIdx.x - slot * a.h);
  const int kh = head / (a.h / a.hk);
  long t0 = 0;
  const int n = delta_chunk(a, slot, &t0);
  if (n == 0) return;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, r = lane & 15, q = lane >> 4;
  float* const sc = a.sc + (slot * a.h + head) * kDeltaSc;

  if (w == 0) {
    const size_t at = static_cast<size_t>(t0 + lane) * a.h + head;
    double g = lane < n ? static_cast<double>(a.g[at]) : 0.0;
    g = g < -1e4 ? -1e4 : g;  // e^-10000 is 0 in 32 bits already; -inf would make differences NaN
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const double up = __shfl_up(g, o);
      if (lane >= o) g += up;
    }
    Gs[lane] = g;
    bs[lane] = lane < n ? a.beta[at] : 0.0f;
  }
  {  // the chunk's q and k rows, zeros past its end and past K
    constexpr int per = KP / 8;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const IN* src = static_cast<const IN*>(which ? a.q : a.k);
      const long stride = which ? a.q_stride : a.k_stride;
      IN* dst = which ? Qs : Ks;
      float* rs = which ? rqs : rks;
#pragma unroll
      for (int p = tid; p < kDeltaC * per; p += 256) {
        const int t = p / per, d0 = (p % per) * 8;
        float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (t < n) row8<IN>(src + (t0 + t) * stride + static_cast<long>(kh) * a.K, d0, a.K, a.vec_qk, v);
        put8(dst + t * pitch + d0, v);
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
        for (int o = 1; o < per; o <<= 1) ss += __shfl_xor(ss, o);
        if (d0 == 0) rs[t] = a.qk_norm ? 1.0f / sqrtf(ss + a.eps) : 1.0f;
      }
    }
  }
  __syncthreads();

  // k k^T and q k^T, row tile w against the column tiles up to it
  f32x4 kk[4], qk[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) kk[j] = qk[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int c = 0; c < ND; ++c) {
    const int off = 32 * c + 8 * q;
    const Frag<NI> fk = frag44(Ks + (16 * w + r) * pitch + off, Ks + (16 * w + r) * pitch + off + 4);
    const Frag<NI> fq = frag44(Qs + (16 * w + r) * pitch + off, Qs + (16 * w + r) * pitch + off + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j <= w) {
        const Frag<NI> b = frag44(Ks + (16 * j + r) * pitch + off, Ks + (16 * j + r) * pitch + off + 4);
        kk[j] = mma(fk, b, kk[j]);
        qk[j] = mma(fq, b, qk[j]);
      }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * w + 4 * q + i, s = 16 * j + r;
      const bool in = s <= t;  // above the diagonal the decay may overflow: never formed
      const float dec = in ? exp_of(Gs[t] - Gs[s]) * rks[s] : 0.0f;
      Lm[t * kLP + s] = s < t ? bs[t] * rks[t] * dec * kk[j][i] : 0.0f;
      qk[j][i] = in ? a.scale * rqs[t] * dec * qk[j][i] : 0.0f;
    }
  }
  // operands shared by the key head's value heads
  if (head % (a.h / a.hk) == 0) {
    const size_t at = static_cast<size_t>(slot) * a.hk + kh;
    unsigned char* kf = a.kf + at * (4 * ND * NI * kDeltaFrag);
    unsigned char* qf = a.qf + at * (4 * ND * NI * kDeltaFrag);
#pragma unroll
    for (int c = 0; c < ND; ++c) {
      const int o = (16 * w + r) * pitch + 32 * c + 4 * q;
      store_frag<NI>(kf, w * ND + c, lane, frag44(Ks + o, Ks + o + 16));
      store_frag<NI>(qf, w * ND + c, lane, frag44(Qs + o, Qs + o + 16));
    }
    unsigned char* ktf = a.ktf + at * (4 * ND * NI * kDeltaFrag);
    unsigned char* qtf = BWD ? a.qtf + at * (4 * ND * NI * kDeltaFrag) : nullptr;
#pragma unroll
    for (int ct = w; ct < KP / 16; ct += 4)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int o = (32 * s + 8 * q) * pitch + 16 * ct + r;
        store_frag<NI>(ktf, 2 * ct + s, lane, frag_col(Ks + o, pitch));
        if (BWD) store_frag<NI>(qtf, 2 * ct + s, lane, frag_col(Qs + o, pitch));
      }
  }
  if (tid < kDeltaC) {
    const double G = Gs[tid], GC = Gs[kDeltaC - 1];
    const float eg = exp_of(G), el = exp_of(GC - G);
    sc[kScBeta * kDeltaC + tid] = bs[tid];
    sc[kScR * kDeltaC + tid] = bs[tid] * eg * rks[tid];
    sc[kScO * kDeltaC + tid] = a.scale * eg * rqs[tid];
    sc[kScU * kDeltaC + tid] = el * rks[tid];
    sc[kScEg * kDeltaC + tid] = eg;
    sc[kScEl * kDeltaC + tid] = el;
    sc[kScRk * kDeltaC + tid] = rks[tid];
    sc[kScRq * kDeltaC + tid] = rqs[tid];
    reinterpret_cast<double*>(sc + kScG * kDeltaC)[tid] = G;
    if (tid == 0) sc[kScGamma * kDeltaC] = exp_of(GC);
  }
  __syncthreads();

  // P takes the rows' place; the diagonal blocks of T by substitution
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) Pm[(16 * w + 4 * q + i) * kLP + 16 * j + r] = qk[j][i];
  {
    float x[16];  // column r of block w's inverse (every 16-lane row of the wave alike)
    const float* Lw = Lm + 16 * w * kLP + 16 * w;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == r ? 1.0f : 0.0f;
#pragma unroll
      for (int m = 0; m < i; ++m) s = fmaf(-Lw[i * kLP + m], x[m], s);
      x[i] = s;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((i >> 2) == q) Tm[(16 * w + i) * kLP + 16 * w + r] = x[i];
    // blocks above the diagonal are read as operands where a step spans them
    for (int j = w + 1; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) Tm[(16 * w + 4 * q + i) * kLP + 16 * j + r] = 0.0f;
  }
  __syncthreads();
#pragma unroll 1
  for (int dist = 1; dist < 4; ++dist) {
    const int i = w, j = w - dist;  // one block of this diagonal per wave
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    if (j >= 0) {
      for (int m = j; m < i; ++m)
        sum = mma16(Lm + 16 * i * kLP + 16 * m, Tm + 16 * m * kLP + 16 * j, r, q, sum);
#pragma unroll
      for (int e = 0; e < 4; ++e) Tm[(16 * i + 4 * q + e) * kLP + 16 * j + r] = -sum[e];
    }
    __syncthreads();
    if (j >= 0) {
      const f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
      sum = mma16(Tm + 16 * i * kLP + 16 * i, Tm + 16 * i * kLP + 16 * j, r, q, z);
      // this wave alone reads and writes block (i, j) between the barriers
#pragma unroll
      for (int e = 0; e < 4; ++e) Tm[(16 * i + 4 * q + e) * kLP + 16 * j + r] = sum[e];
    }
    __syncthreads();
  }

  const size_t at = static_cast<size_t>(slot) * a.h + head;
  unsigned char* tf = a.tf + at * (kDeltaTri * NS * kDeltaFrag);
  unsigned char* pf = BWD ? nullptr : a.pf + at * (kDeltaTri * NO * kDeltaFrag);
  for (int s = 0; s <= (w >> 1); ++s) {
    const int o = (16 * w + r) * kLP + 32 * s + 8 * q;
    store_frag<NS>(tf, low_frag(w, s), lane, frag_row<NS>(Tm + o));
    if (!BWD) store_frag<NO>(pf, low_frag(w, s), lane, frag_row<NO>(Pm + o));
  }
  if (BWD) {
    unsigned char* ttf = a.ttf + at * (kDeltaTri * NS * kDeltaFrag);
    unsigned char* ptf = a.ptf + at * (kDeltaTri * NS * kDeltaFrag);
    for (int s = w >> 1; s < 2; ++s) {
      const int o = (32 * s + 8 * q) * kLP + 16 * w + r;
      store_frag<NS>(ttf, up_frag(w, s), lane, frag_fcol<NS>(Tm + o));
      store_frag<NS>(ptf, up_frag(w, s), lane, frag_fcol<NS>(Pm + o));
    }
  }
}

template <typename IN, int KP>
hipError_t go(const DeltaLaunch& l, bool bwd, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(l.a.slots * l.a.h));
  if (bwd)
    hipLaunchKernelGGL((delta_prep_kernel<IN, KP, true>), grid, dim3(256), 0, s, l.a);
  else
    hipLaunchKernelGGL((delta_prep_kernel<IN, KP, false>), grid, dim3(256), 0, s, l.a);
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
