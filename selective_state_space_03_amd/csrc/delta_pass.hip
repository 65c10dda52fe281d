// The walk of the gated delta rule over the chunks of a sequence, forward and in
// reverse (equations in delta.h).
//
// One workgroup of four waves holds NV slices of 16 value channels of one
// (sequence, head): S is K x 16 NV in accumulator tiles, K / 64 tiles of 16 key
// channels per wave and slice.  A chunk has three dependent products (k S^T,
// T R, the state update); between them the waves exchange their tiles through
// LDS, each split once, by the wave that made it, into bf16 parts:
//   1. R = beta v - (beta e^G rk) (K S)       wave w: tokens 16 w .. 16 w + 15
//   2. u = T R                                same tokens
//   3. S <- e^{G_C} S + K^T (e^{G_C-G} rk u)  wave w: its own key channels
//      o = (scale e^G rq) (Q S) + P u         its own tokens, transposed, so a
//                                             lane stores 4 neighbouring channels
// Every operand that does not depend on the state comes from the prep kernel in
// the lanes' order, so it goes from memory to registers, asked for as soon as its
// registers are free of the chunk before.
//
// Bound by a chunk's length in time where there is one workgroup per CU (8192 tokens,
// 32 heads of 128: 128 chunks in 295 us, 2.3 us each; reading ahead halved it), and by
// vector ALU (43 % of the SIMD cycles) and matrix cores (29 %) at two waves per SIMD
// where there are many (12289 packed tokens, 80 heads, K 64, V 96: 480 us; LDS 34 %
// busy, 9 % more in bank conflicts).  Training, 4 x 2048 tokens, 16 heads of 128: 120 us
// forward, 154 us in reverse.
#include "delta_device.h"

namespace ssm {
namespace {

constexpr int kTile = 16 * kDeltaC;  // 16-bit words of an exchanged tile's part in LDS

// 4 consecutive outputs of a row, any dtype; vec: they are all inside and aligned
__device__ __forceinline__ void store4(void* p, size_t i, bool bf16, bool vec, int left, f32x4 v) {
  if (bf16) {
    uint16_t* o = static_cast<uint16_t*>(p) + i;
    const uint32_t a = pack_rne(v[0], v[1]), b = pack_rne(v[2], v[3]);
    if (vec) {
      *reinterpret_cast<uint2*>(o) = make_uint2(a, b);
    } else {
      if (left > 0) o[0] = static_cast<uint16_t>(a);
      if (left > 1) o[1] = static_cast<uint16_t>(a >> 16);
      if (left > 2) o[2] = static_cast<uint16_t>(b);
      if (left > 3) o[3] = static_cast<uint16_t>(b >> 16);
    }
  } else {
    float* o = static_cast<float*>(p) + i;
    if (vec) {
      *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (left > e) o[e] = v[e];
    }
  }
}

// state rows (V, K): 4 consecutive key channels from d of row v
__device__ __forceinline__ f32x4 load_state4(const float* s, long row, int d, int K, bool ok, bool vec) {
  f32x4 r = {0.0f, 0.0f, 0.0f, 0.0f};
  if (!ok) return r;
  const float* p = s + row * K + d;
  if (vec) {
    if (d < K) r = *reinterpret_cast<const f32x4*>(p);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (d + e < K) r[e] = p[e];
  }
  return r;
}
__device__ __forceinline__ void store_state4(float* s, long row, int d, int K, bool ok, bool vec, f32x4 v) {
  if (!ok) return;
  float* p = s + row * K + d;
  if (vec) {
    if (d < K) *reinterpret_cast<f32x4*>(p) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (d + e < K) p[e] = v[e];
  }
}

// A wave's tile (tokens t .. t + 3 = 16 w + 4 q .., channel r) as NP parts into the
// operands' order, [part][step][lane] 16 bytes: reads are whole lines
template <int NP>
__device__ __forceinline__ void put_tile(uint16_t* dst, int r, int t, f32x4 v) {
  uint32_t a[NP], b[NP];
  split2<NP>(v[0], v[1], a);
  split2<NP>(v[2], v[3], b);
  uint16_t* at = dst + ((t >> 5) * 64 + ((t >> 3) & 3) * 16 + r) * 8 + (t & 4);
#pragma unroll
  for (int p = 0; p < NP; ++p) *reinterpret_cast<uint2*>(at + p * kTile) = make_uint2(a[p], b[p]);
}
// The operand of token step s from such a tile
template <int NP>
__device__ __forceinline__ Frag<NP> get_tile(const uint16_t* src, int r, int q, int s) {
  Frag<NP> f;
#pragma unroll
  for (int p = 0; p < NP; ++p)
    f.p[p] = *reinterpret_cast<const uint4*>(src + p * kTile + (s * 64 + q * 16 + r) * 8);
  return f;
}

// State tiles -> operand parts: [slab of 32 key channels][part][lane] 16 bytes, a
// tile filling half of each lane's 8 slots.
template <int NP, int ND>
__device__ __forceinline__ void put_state(unsigned char* dst, int ct, int lane, f32x4 v) {
  uint32_t a[NP], b[NP];
  split2<NP>(v[0], v[1], a);
  split2<NP>(v[2], v[3], b);
#pragma unroll
  for (int p = 0; p < NP; ++p)
    *reinterpret_cast<uint2*>(dst + (((ct >> 1) * NP + p) * 64 + lane) * 16 + (ct & 1) * 8) = make_uint2(a[p], b[p]);
}

// The two tiles of a slab at once
template <int NP>
__device__ __forceinline__ void put_slab(unsigned char* dst, int slab, int lane, f32x4 v, f32x4 x) {
  uint32_t a[NP], b[NP], c[NP], d[NP];
  split2<NP>(v[0], v[1], a);
  split2<NP>(v[2], v[3], b);
  split2<NP>(x[0], x[1], c);
  split2<NP>(x[2], x[3], d);
#pragma unroll
  for (int p = 0; p < NP; ++p)
    *reinterpret_cast<uint4*>(dst + ((slab * NP + p) * 64 + lane) * 16) = make_uint4(a[p], b[p], c[p], d[p]);
}
// A wave's CT state tiles
template <int NP, int ND, int CT, int NV>
__device__ __forceinline__ void put_states(unsigned char* dst, int w, int lane, int e, const f32x4 (&S)[CT][NV]) {
  if (CT == 2) {
    put_slab<NP>(dst, w, lane, S[0][e], S[CT - 1][e]);
  } else {
    put_state<NP, ND>(dst, w, lane, S[0][e]);
  }
}

template <typename IN, int KP, int NV, bool SAVE>
__global__ __launch_bounds__(256) void delta_pass_kernel(DeltaArgs a, int slices, int o_bf16, int vec_o) {
  using Parts = DeltaParts<IN>;
  constexpr int NI = Parts::in, NS = Parts::state;
  constexpr int ND = KP / 32, CT = KP / 64;
  constexpr int kState = ND * NS * kDeltaFrag;
  __shared__ __align__(16) unsigned char Ssh[NV * kState];
  __shared__ __align__(16) uint16_t Rsh[NV][NS * kTile];
  __shared__ __align__(16) uint16_t Ush[NV][NS * kTile];
  __shared__ __align__(16) uint16_t Wsh[SAVE ? 1 : NV][SAVE ? 8 : NS * kTile];

  long group;
  unsigned slice;
  xcd_group(blockIdx.x, slices, &group, &slice);
  if (group >= static_cast<long>(a.nseq) * a.h) return;
  const int seq = static_cast<int>(group / a.h), head = static_cast<int>(group - static_cast<long>(seq) * a.h);
  const int kh = head / (a.h / a.hk);
  const DeltaSeq sq = delta_seq(a, seq);
  const int nch = (sq.len + kDeltaC - 1) / kDeltaC;
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6), r = lane & 15, q = lane >> 4;
  const int v0 = static_cast<int>(slice) * 16 * NV;
  [[maybe_unused]] const int vp = delta_vp(a.V);

  f32x4 S[CT][NV];
#pragma unroll
  for (int i = 0; i < CT; ++i)
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      const int v = v0 + 16 * e + r, d = 16 * (w * CT + i) + 4 * q;
      S[i][e] = a.state_in ? load_state4(a.state_in, group * a.V + v, d, a.K, v < a.V, a.vec_state)
                           : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
  for (int e = 0; e < NV; ++e) put_states<NS, ND, CT, NV>(Ssh + e * kState, w, lane, e, S);

  // operands of the chunk at hand; each is asked for again, for the next chunk, right
  // after its last use, so a chunk's loads have the rest of the chunk before to arrive
  Frag<NI> fk[ND], fq[SAVE ? 1 : ND], fkt[CT][2];
  Frag<NS> ft[2];
  Frag<NS> fp[2];
  // Waves 0 and 1 have no second step of the triangles: theirs stays zero, which costs
  // nothing beside waves 2 and 3 (skipping it measured the same) and keeps the products
  // free of branches: between a matrix instruction and the first use of its result the
  // compiler's wait states are counted along one path only.
  zero_frag(ft[1]);
  zero_frag(fp[1]);
  f32x4 beta, cr, cu;
  IN vv[NV][4];  // as loaded: a conversion here would wait for the load
  float co = 0.0f, gamma = 0.0f;
  const size_t kstep = static_cast<size_t>(a.hk) * (4 * ND * NI * kDeltaFrag);
  const size_t khead = (static_cast<size_t>(sq.slot0) * a.hk + kh) * (4 * ND * NI * kDeltaFrag);
  const size_t hc0 = static_cast<size_t>(sq.slot0) * a.h + head;
  auto load_rows = [&](int c) {  // what the first product uses
    const float* sc = a.sc + (hc0 + static_cast<size_t>(c) * a.h) * kDeltaSc;
#pragma unroll
    for (int s = 0; s < ND; ++s) {
      fk[s] = load_frag<NI>(a.kf + khead + c * kstep, w * ND + s, lane);
      if (!SAVE) fq[s] = load_frag<NI>(a.qf + khead + c * kstep, w * ND + s, lane);
    }
    beta = *reinterpret_cast<const f32x4*>(sc + kScBeta * kDeltaC + 16 * w + 4 * q);
    cr = *reinterpret_cast<const f32x4*>(sc + kScR * kDeltaC + 16 * w + 4 * q);
    const long t0 = sq.t0 + static_cast<long>(c) * kDeltaC;
    const int n = min(kDeltaC, sq.len - c * kDeltaC);
#pragma unroll
    for (int e = 0; e < NV; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // (rows and channels past the end read others and are dropped at their use)
        const int t = 16 * w + 4 * q + i, v = v0 + 16 * e + r;
        const long row = t0 + (t < n ? t : 0);
        vv[e][i] = static_cast<const IN*>(a.v)[row * a.v_stride + static_cast<long>(head) * a.V + min(v, a.V - 1)];
      }
  };
  auto load_tri = [&](int c) {  // T and the coefficients of u
    const size_t hc = hc0 + static_cast<size_t>(c) * a.h;
    const unsigned char* tf = a.tf + hc * (kDeltaTri * NS * kDeltaFrag);
    ft[0] = load_frag<NS>(tf, low_frag(w, 0), lane);
    if (w >= 2) ft[1] = load_frag<NS>(tf, low_frag(w, 1), lane);
    cu = *reinterpret_cast<const f32x4*>(a.sc + hc * kDeltaSc + kScU * kDeltaC + 16 * w + 4 * q);
  };
  auto load_update = [&](int c) {
    const size_t hc = hc0 + static_cast<size_t>(c) * a.h;
    const float* sc = a.sc + hc * kDeltaSc;
#pragma unroll
    for (int i = 0; i < CT; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s) fkt[i][s] = load_frag<NI>(a.ktf + khead + c * kstep, 2 * (w * CT + i) + s, lane);
    gamma = sc[kScGamma * kDeltaC];
    if (!SAVE) {
      const unsigned char* pf = a.pf + hc * (kDeltaTri * NS * kDeltaFrag);
      fp[0] = load_frag<NS>(pf, low_frag(w, 0), lane);
      if (w >= 2) fp[1] = load_frag<NS>(pf, low_frag(w, 1), lane);
      co = sc[kScO * kDeltaC + 16 * w + r];
    }
  };
  if (nch > 0) {
    load_rows(0);
    load_tri(0);
    load_update(0);
  }

  for (int c = 0; c < nch; ++c) {
    const size_t hc = hc0 + static_cast<size_t>(c) * a.h;
    const int next = min(c + 1, nch - 1);
    const long t0 = sq.t0 + static_cast<long>(c) * kDeltaC;
    const int n = min(kDeltaC, sq.len - c * kDeltaC);

    if (SAVE) {  // the state entering the chunk, (K, V) rows
#pragma unroll
      for (int i = 0; i < CT; ++i)
#pragma unroll
        for (int e = 0; e < NV; ++e) {
          const int v = v0 + 16 * e + r, d = 16 * (w * CT + i) + 4 * q;
          float* dst = a.s_chunk + (hc * KP + d) * vp + v;
#pragma unroll
          for (int x = 0; x < 4; ++x) dst[static_cast<long>(x) * vp] = S[i][e][x];
        }
    }

    lds_barrier();  // the state's parts
    f32x4 ot[NV];
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      f32x4 ks = {0.0f, 0.0f, 0.0f, 0.0f};
      ot[e] = ks;
#pragma unroll
      for (int s = 0; s < ND; ++s) {
        const Frag<NS> st = load_frag<NS>(Ssh + e * kState, s, lane);
        ks = mma(fk[s], st, ks);
        if (!SAVE) ot[e] = mma(st, fq[s], ot[e]);
      }
      f32x4 rr;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        rr[i] = fmaf(beta[i], 16 * w + 4 * q + i < n && v0 + 16 * e + r < a.V ? to_f32(vv[e][i]) : 0.0f, -cr[i] * ks[i]);
      put_tile<NS>(Rsh[e], r, 16 * w + 4 * q, rr);
    }
    load_rows(next);
    lds_barrier();  // R
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      f32x4 u = {0.0f, 0.0f, 0.0f, 0.0f}, u1 = u;
      u = mma(ft[0], get_tile<NS>(Rsh[e], r, q, 0), u);
      u1 = mma(ft[1], get_tile<NS>(Rsh[e], r, q, 1), u1);
      f32x4 us;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u[i] += u1[i];
        us[i] = cu[i] * u[i];
      }
      put_tile<NS>(Ush[e], r, 16 * w + 4 * q, us);
      if (!SAVE) {
        put_tile<NS>(Wsh[e], r, 16 * w + 4 * q, u);
      } else {
        const int v = v0 + 16 * e + r;
        float* dst = a.u_chunk + (hc * kDeltaC + 16 * w + 4 * q) * vp + v;
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[static_cast<long>(i) * vp] = u[i];
      }
    }
    load_tri(next);
    lds_barrier();  // u
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      const Frag<NS> u0 = get_tile<NS>(Ush[e], r, q, 0), u1 = get_tile<NS>(Ush[e], r, q, 1);
#pragma unroll
      for (int i = 0; i < CT; ++i) {
        f32x4 s = S[i][e];
#pragma unroll
        for (int x = 0; x < 4; ++x) s[x] *= gamma;
        s = mma(fkt[i][0], u0, s);
        s = mma(fkt[i][1], u1, s);
        S[i][e] = s;
      }
      put_states<NS, ND, CT, NV>(Ssh + e * kState, w, lane, e, S);
      if (!SAVE) {
        f32x4 o = ot[e];
#pragma unroll
        for (int x = 0; x < 4; ++x) o[x] *= co;
        o = mma(get_tile<NS>(Wsh[e], r, q, 0), fp[0], o);
        o = mma(get_tile<NS>(Wsh[e], r, q, 1), fp[1], o);
        const int t = 16 * w + r, v = v0 + 16 * e + 4 * q, left = a.V - v;
        if (t < n && left > 0)
          store4(a.o, (static_cast<size_t>(t0 + t) * a.h + head) * a.V + v, o_bf16, vec_o && left >= 4, left, o);
      }
    }
    load_update(next);
  }

  if (!SAVE && a.state_out)
#pragma unroll
    for (int i = 0; i < CT; ++i)
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        const int v = v0 + 16 * e + r, d = 16 * (w * CT + i) + 4 * q;
        store_state4(a.state_out, group * a.V + v, d, a.K, v < a.V, a.vec_state, S[i][e]);
      }
}

// The reverse walk: with D the gradient of the state leaving a chunk,
//   dU = P^T do + (e^{G_C-G} rk) (K D),  dR = T^T dU,
//   D <- e^{G_C} D + Q^T (scale e^G rq do) - K^T (beta e^G rk dR),
// the same three dependent products per chunk as the forward walk; D and dR are
// kept for the gradients' kernel.
template <typename IN, int KP, int NV>
__global__ __launch_bounds__(256) void delta_reverse_kernel(DeltaArgs a, int slices) {
  using Parts = DeltaParts<IN>;
  constexpr int NI = Parts::in, NS = Parts::state;
  constexpr int ND = KP / 32, CT = KP / 64;
  constexpr int kState = ND * NS * kDeltaFrag;
  __shared__ __align__(16) unsigned char Ssh[NV * kState];
  __shared__ __align__(16) uint16_t Rsh[NV][NS * kTile];
  __shared__ __align__(16) uint16_t Ush[NV][NS * kTile];
  __shared__ __align__(16) uint16_t Dsh[NV][NI * kTile];   // do
  __shared__ __align__(16) uint16_t Csh[NV][NS * kTile];   // scale e^G rq do

  long group;
  unsigned slice;
  xcd_group(blockIdx.x, slices, &group, &slice);
  if (group >= static_cast<long>(a.nseq) * a.h) return;
  const int seq = static_cast<int>(group / a.h), head = static_cast<int>(group - static_cast<long>(seq) * a.h);
  const int kh = head / (a.h / a.hk);
  const DeltaSeq sq = delta_seq(a, seq);
  const int nch = (sq.len + kDeltaC - 1) / kDeltaC;
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6), r = lane & 15, q = lane >> 4;
  const int v0 = static_cast<int>(slice) * 16 * NV;
  [[maybe_unused]] const int vp = delta_vp(a.V);

  f32x4 D[CT][NV];
#pragma unroll
  for (int i = 0; i < CT; ++i)
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      const int v = v0 + 16 * e + r, d = 16 * (w * CT + i) + 4 * q;
      D[i][e] = a.dstate_out ? load_state4(a.dstate_out, group * a.V + v, d, a.K, v < a.V, a.vec_state)
                             : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
  for (int e = 0; e < NV; ++e) put_states<NS, ND, CT, NV>(Ssh + e * kState, w, lane, e, D);

  // operands, asked for again right after their last use (as in the forward walk)
  Frag<NI> fk[ND], fkt[CT][2], fqt[CT][2];
  Frag<NS> ft[2], fp[2];
  zero_frag(ft[0]);  // (waves 2 and 3 have no first step; as above)
  zero_frag(fp[0]);
  f32x4 cr, cu, co;
  IN dv[NV][4];
  float gamma = 0.0f;
  const size_t kstep = static_cast<size_t>(a.hk) * (4 * ND * NI * kDeltaFrag);
  const size_t khead = (static_cast<size_t>(sq.slot0) * a.hk + kh) * (4 * ND * NI * kDeltaFrag);
  const size_t hc0 = static_cast<size_t>(sq.slot0) * a.h + head;
  auto load_rows = [&](int c) {  // do and the first product's operands
    const size_t hc = hc0 + static_cast<size_t>(c) * a.h;
    const float* sc = a.sc + hc * kDeltaSc;
    const unsigned char* ptf = a.ptf + hc * (kDeltaTri * NS * kDeltaFrag);
#pragma unroll
    for (int s = 0; s < ND; ++s) fk[s] = load_frag<NI>(a.kf + khead + c * kstep, w * ND + s, lane);
    fp[1] = load_frag<NS>(ptf, up_frag(w, 1), lane);
    if (w < 2) fp[0] = load_frag<NS>(ptf, up_frag(w, 0), lane);
    cu = *reinterpret_cast<const f32x4*>(sc + kScU * kDeltaC + 16 * w + 4 * q);
  };
  auto load_do = [&](int c) {
    const float* sc = a.sc + (hc0 + static_cast<size_t>(c) * a.h) * kDeltaSc;
    co = *reinterpret_cast<const f32x4*>(sc + kScO * kDeltaC + 16 * w + 4 * q);
    const long t0 = sq.t0 + static_cast<long>(c) * kDeltaC;
    const int n = min(kDeltaC, sq.len - c * kDeltaC);
#pragma unroll
    for (int e = 0; e < NV; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * w + 4 * q + i, v = v0 + 16 * e + r;
        const size_t row = static_cast<size_t>(t0 + (t < n ? t : 0));
        dv[e][i] = static_cast<const IN*>(a.dout)[(row * a.h + head) * a.V + min(v, a.V - 1)];
      }
  };
  auto load_tri = [&](int c) {
    const size_t hc = hc0 + static_cast<size_t>(c) * a.h;
    const unsigned char* ttf = a.ttf + hc * (kDeltaTri * NS * kDeltaFrag);
    ft[1] = load_frag<NS>(ttf, up_frag(w, 1), lane);
    if (w < 2) ft[0] = load_frag<NS>(ttf, up_frag(w, 0), lane);
    cr = *reinterpret_cast<const f32x4*>(a.sc + hc * kDeltaSc + kScR * kDeltaC + 16 * w + 4 * q);
  };
  auto load_update = [&](int c) {
#pragma unroll
    for (int i = 0; i < CT; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        fkt[i][s] = load_frag<NI>(a.ktf + khead + c * kstep, 2 * (w * CT + i) + s, lane);
        fqt[i][s] = load_frag<NI>(a.qtf + khead + c * kstep, 2 * (w * CT + i) + s, lane);
      }
    gamma = a.sc[(hc0 + static_cast<size_t>(c) * a.h) * kDeltaSc + kScGamma * kDeltaC];
  };
  if (nch > 0) {
    load_do(nch - 1);
    load_rows(nch - 1);
    load_tri(nch - 1);
    load_update(nch - 1);
  }

  for (int c = nch - 1; c >= 0; --c) {
    const size_t hc = hc0 + static_cast<size_t>(c) * a.h;
    const int next = max(c - 1, 0);
    const int n = min(kDeltaC, sq.len - c * kDeltaC);

#pragma unroll
    for (int i = 0; i < CT; ++i)
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        const int v = v0 + 16 * e + r, d = 16 * (w * CT + i) + 4 * q;
        float* dst = a.ds_chunk + (hc * KP + d) * vp + v;
#pragma unroll
        for (int x = 0; x < 4; ++x) dst[static_cast<long>(x) * vp] = D[i][e][x];
      }
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      f32x4 dd, cd;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dd[i] = 16 * w + 4 * q + i < n && v0 + 16 * e + r < a.V ? to_f32(dv[e][i]) : 0.0f;
        cd[i] = co[i] * dd[i];
      }
      put_tile<NI>(Dsh[e], r, 16 * w + 4 * q, dd);
      put_tile<NS>(Csh[e], r, 16 * w + 4 * q, cd);
    }
    load_do(next);

    lds_barrier();  // D's parts, do
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f}, y = x;
#pragma unroll
      for (int s = 0; s < ND; ++s) x = mma(fk[s], load_frag<NS>(Ssh + e * kState, s, lane), x);
      y = mma(fp[1], get_tile<NI>(Dsh[e], r, q, 1), y);
      y = mma(fp[0], get_tile<NI>(Dsh[e], r, q, 0), y);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = fmaf(cu[i], x[i], y[i]);
      put_tile<NS>(Rsh[e], r, 16 * w + 4 * q, x);
    }
    load_rows(next);
    lds_barrier();  // dU
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f}, y0 = y;
      y = mma(ft[1], get_tile<NS>(Rsh[e], r, q, 1), y);
      y0 = mma(ft[0], get_tile<NS>(Rsh[e], r, q, 0), y0);
      f32x4 ys;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] += y0[i];
        ys[i] = -cr[i] * y[i];
      }
      put_tile<NS>(Ush[e], r, 16 * w + 4 * q, ys);
      const int v = v0 + 16 * e + r;
      float* dst = a.dr_chunk + (hc * kDeltaC + 16 * w + 4 * q) * vp + v;
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[static_cast<long>(i) * vp] = y[i];
    }
    load_tri(next);
    lds_barrier();  // dR
#pragma unroll
    for (int e = 0; e < NV; ++e) {
#pragma unroll
      for (int i = 0; i < CT; ++i) {
        f32x4 s = D[i][e], s1 = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int x = 0; x < 4; ++x) s[x] *= gamma;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          s = mma(fkt[i][k], get_tile<NS>(Ush[e], r, q, k), s);
          s1 = mma(fqt[i][k], get_tile<NS>(Csh[e], r, q, k), s1);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) s[x] += s1[x];
        D[i][e] = s;
      }
      put_states<NS, ND, CT, NV>(Ssh + e * kState, w, lane, e, D);
    }
    load_update(next);
    lds_barrier();  // do's tiles may be written again
  }

  if (a.dstate_in)
#pragma unroll
    for (int i = 0; i < CT; ++i)
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        const int v = v0 + 16 * e + r, d = 16 * (w * CT + i) + 4 * q;
        store_state4(a.dstate_in, group * a.V + v, d, a.K, v < a.V, a.vec_state, D[i][e]);
      }
}

template <typename IN, int KP, int NV>
hipError_t go(const DeltaLaunch& l, int what, hipStream_t s) {
  const long groups = static_cast<long>(l.a.nseq) * l.a.h;
  const int slices = static_cast<int>(delta_slices(groups, l.a.V, what != 0));
  const dim3 grid(static_cast<unsigned>(delta_walk_blocks(groups, l.a.V, what != 0)));
  const int ob = l.o_dtype == kBF16;
  const int vec_o = l.a.V % 4 == 0 && (reinterpret_cast<uintptr_t>(l.a.o) & (ob ? 7 : 15)) == 0;
  if (what == 0)
    return timed_launch(s, [&] {
      hipLaunchKernelGGL((delta_pass_kernel<IN, KP, NV, false>), grid, dim3(256), 0, s, l.a, slices, ob, vec_o);
    });
  else if (what == 1)
    hipLaunchKernelGGL((delta_pass_kernel<IN, KP, NV, true>), grid, dim3(256), 0, s, l.a, slices, 0, 0);
  else
    hipLaunchKernelGGL((delta_reverse_kernel<IN, KP, NV>), grid, dim3(256), 0, s, l.a, slices);
  return hipGetLastError();
}

template <typename IN, int KP>
hipError_t pick_nv(const DeltaLaunch& l, int what, hipStream_t s) {
  return delta_nv(static_cast<long>(l.a.nseq) * l.a.h, l.a.V) == 2 ? go<IN, KP, 2>(l, what, s)
                                                                   : go<IN, KP, 1>(l, what, s);
}

template <typename IN>
hipError_t pick_k(const DeltaLaunch& l, int what, hipStream_t s) {
  return delta_kp(l.a.K) == 64 ? pick_nv<IN, 64>(l, what, s) : pick_nv<IN, 128>(l, what, s);
}

hipError_t pick(const DeltaLaunch& l, int what, hipStream_t s) {
  if (l.a.nseq == 0) return hipSuccess;
  return l.in_dtype == kBF16 ? pick_k<bf16s>(l, what, s) : pick_k<float>(l, what, s);
}

}  // namespace

hipError_t launch_delta_pass(const DeltaLaunch& l, bool save, hipStream_t s) { return pick(l, save ? 1 : 0, s); }
hipError_t launch_delta_reverse(const DeltaLaunch& l, hipStream_t s) { return pick(l, 2, s); }

}  // namespace ssm
