// One query of each sequence over its pages, for gfx950.
//
// The visible keys of a sequence, [0, sinks) and those of its window, are counted through as one range,
// which is cut into parts of a.chunk keys; a workgroup takes one part for the (up to 16) query heads of a
// key head, its four waves the part's tiles of 32 keys (16 in f32) in turn.  Per tile, as in the forward,
//   S^T = K Q^T,  P = 2^(S - m),  O^T += V^T P^T
// with K straight from memory as an operand (a lane holds 8 channels of a key), V through LDS, where it is
// read transposed.  The scale of a page of 8 bits goes to S and to P, so codes enter the products as they
// are (e4m3 is exact in bf16).  32-bit operands (q in f32, P) enter as three bf16 parts.
// Waves, then parts (a second kernel), are joined by their maxima and sums.
// The step reads the visible cache once and is bound by that.
#include "attn_device.h"

namespace ssm {
namespace {

struct e4m3s {
  uint8_t bits;
};

template <typename CT>
struct StepEl {  // f32 and bf16: operands as they are stored
  using Op = CT;
  using Raw = uint4;
  static __device__ __forceinline__ Raw zero() { return make_uint4(0u, 0u, 0u, 0u); }
  static __device__ __forceinline__ uint4 op(Raw r) { return r; }
  static __device__ __forceinline__ Raw load(const CT* row, int c, int D, int vec) { return attn_chunk<CT>(row, c, D, vec ? 2 : 0); }
};
template <>
struct StepEl<e4m3s> {  // 8 codes to 8 bf16
  using Op = bf16s;
  using Raw = uint2;
  static __device__ __forceinline__ Raw zero() { return make_uint2(0u, 0u); }
  static __device__ __forceinline__ uint4 op(Raw r) {
    return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.x, 1.0f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.x, 1.0f, true)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.y, 1.0f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.y, 1.0f, true)));
  }
  static __device__ __forceinline__ Raw load(const e4m3s* row, int c, int D, int vec) {
    Raw r = zero();
    if (vec) {
      if (c < D) r = *reinterpret_cast<const uint2*>(row + c);
      return r;
    }
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < D) w[i / 4] |= static_cast<uint32_t>(row[c + i].bits) << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
  }
};

// Visible keys of a sequence: x counts them through
struct StepKeys {
  int ns, lo, n;  // sinks ahead of the window, its first key, keys in all
  __device__ __forceinline__ int key(int x) const { return x < ns ? x : x - ns + lo; }
};
__device__ __forceinline__ StepKeys step_keys(const AttnStepArgs& a, int b) {
  const int len = min(max(a.lens[b], 0), a.table_rows * a.page);
  StepKeys k;
  k.lo = max(0, len - a.window);
  k.ns = min(a.sinks, k.lo);
  k.n = k.ns + len - k.lo;
  return k;
}

__device__ __forceinline__ void wave_sync() {  // LDS of this wave only
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// CT: the cache, QP: parts of q, DQ: channels (a multiple of 32)
template <typename CT, int QP, int DQ>
__global__ __launch_bounds__(256) void attn_step_kernel(const AttnStepArgs a, int q_bf16, int o_bf16) {
  using C = StepEl<CT>;
  using T = typename C::Op;
  using Raw = typename C::Raw;
  using E = AttnEl<T>;
  constexpr int NP = sizeof(T) == 2 ? 3 : 1;               // parts of P
  constexpr int TK = sizeof(T) == 2 ? 32 : 16;             // keys of a tile: one unit
  constexpr int KT = TK / 16, KS = DQ / E::kUnit, NT = DQ / 16;
  constexpr int CPR = DQ / E::kVec, NV = TK * CPR / 64;    // groups of a row, of a lane
  constexpr int VS = DQ * static_cast<int>(sizeof(T)) + 32;
  struct Info {  // of a tile's keys
    long base[TK];                                         // first element of the row, -1: left out
    float add[TK], ks[TK], vs[TK];                         // 0 or -infinity; scales
  };
  constexpr int kRed = 4 * 16 * (DQ + 2) * 4, kTiles = 4 * TK * VS;
  __shared__ __align__(16) unsigned char tiles[kTiles > kRed ? kTiles : kRed];
  __shared__ Info infos[4][2];

  const int g_heads = a.h / a.hk, ht = (g_heads + kAttnStepHeads - 1) / kAttnStepHeads;
  const unsigned split = blockIdx.x % a.nsplit;
  unsigned r = blockIdx.x / a.nsplit;
  const int h0 = static_cast<int>(r % ht) * kAttnStepHeads;
  r /= ht;
  const int kh = static_cast<int>(r % a.hk), b = static_cast<int>(r / a.hk);
  const int nh = min(kAttnStepHeads, g_heads - h0);        // query heads of this workgroup
  const int head0 = kh * g_heads + h0;
  const StepKeys keys = step_keys(a, b);
  const long begin = static_cast<long>(split) * a.chunk;
  if (begin >= keys.n && split > 0) return;
  const int end = static_cast<int>(min(static_cast<long>(keys.n), begin + a.chunk));
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64, g = lane / 16, c = lane % 16;
  unsigned char* const vl = tiles + wave * TK * VS;

  // q as columns, in parts
  Frag<QP> q[KS];
  {
    const long row = b * a.q_stride + static_cast<long>(head0 + c) * a.D;
#pragma unroll
    for (int u = 0; u < KS; ++u) {
      const int d = u * E::kUnit + g * E::kVec;
      if constexpr (QP == 1) {
        q[u].p[0] = make_uint4(0u, 0u, 0u, 0u);
        if (c < nh) q[u].p[0] = attn_chunk<T>(static_cast<const T*>(a.q) + row, d, a.D, a.vec ? 2 : 0);
      } else {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = c < nh && d + i < a.D ? static_cast<const float*>(a.q)[row + d + i] : 0.0f;
        q[u] = split8<QP>(x);
      }
    }
  }

  const float cs = a.scale * kLog2e;
  const int first = static_cast<int>(begin) + wave * TK;   // the wave's first tile
  // page entries of a tile, one key a lane
  struct Page {
    int pg, row;
  };
  const auto page_of = [&](int x0) {
    Page p{-1, 0};
    const int x = x0 + lane;
    if (lane < TK && x < end) {
      const int j = keys.key(x);
      p.row = j % a.page;
      p.pg = a.table[static_cast<long>(b) * a.table_rows + j / a.page];
    }
    return p;
  };
  const auto put_info = [&](Info& to, Page p) {
    if (lane < TK) {
      const bool in = p.pg >= 0 && p.pg < a.pages;
      const long ph = static_cast<long>(p.pg) * a.hk + kh;
      to.base[lane] = in ? (ph * a.page + p.row) * a.D : -1;
      to.add[lane] = in ? 0.0f : -INFINITY;
      if constexpr (sizeof(CT) == 1) {
        to.ks[lane] = in ? a.k_scale[ph] : 0.0f;
        to.vs[lane] = in ? a.v_scale[ph] : 0.0f;
      }
    }
  };
  const CT* const kc = static_cast<const CT*>(a.k_cache);
  const CT* const vc = static_cast<const CT*>(a.v_cache);
  Raw kn[KT][KS], vn[NV];
  const auto fetch = [&](const Info& in) {
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const long base = in.base[16 * k + c];
#pragma unroll
      for (int u = 0; u < KS; ++u) {
        kn[k][u] = C::zero();
        if (base >= 0) kn[k][u] = C::load(kc + base, u * E::kUnit + g * E::kVec, a.D, a.vec);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int x = lane + 64 * i;
      const long base = in.base[x / CPR];
      vn[i] = C::zero();
      if (base >= 0) vn[i] = C::load(vc + base, x % CPR * E::kVec, a.D, a.vec);
    }
  };

  float mx = -INFINITY, l = 0.0f;
  f32x4 o[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) o[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  Page next{-1, 0};
  if (first < end) {
    put_info(infos[wave][0], page_of(first));
    next = page_of(first + 4 * TK);
    wave_sync();
    fetch(infos[wave][0]);
  }
  int at = 0;
  for (int x0 = first; x0 < end; x0 += 4 * TK, at ^= 1) {
    const Info& in = infos[wave][at];
    put_info(infos[wave][at ^ 1], next);
    next = page_of(x0 + 8 * TK);
    wave_sync();
    f32x4 s[KT];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int x = lane + 64 * i;
      *reinterpret_cast<uint4*>(vl + x / CPR * VS + x % CPR * 16) = C::op(vn[i]);
    }
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      s[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < KS; ++u) {
        const uint4 kf = C::op(kn[k][u]);
#pragma unroll
        for (int p = QP - 1; p >= 0; --p) s[k] = attn_mma<T>(kf, q[u].p[p], s[k]);
      }
    }
    if (x0 + 4 * TK < end) fetch(infos[wave][at ^ 1]);
    wave_sync();
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const f32x4 add = *reinterpret_cast<const f32x4*>(&in.add[16 * k + 4 * g]);
      f32x4 ks = {1.0f, 1.0f, 1.0f, 1.0f};
      if constexpr (sizeof(CT) == 1) ks = *reinterpret_cast<const f32x4*>(&in.ks[16 * k + 4 * g]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[k][i] = fmaf(s[k][i], ks[i] * cs, add[i]);
        top = fmaxf(top, s[k][i]);
      }
    }
    top = group_max(top);
    const float to = fmaxf(mx, top), sub = to == -INFINITY ? 0.0f : to;
    const float f = exp2_fast(mx - sub);
    mx = to;
    l *= f;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      f32x4 vs = {1.0f, 1.0f, 1.0f, 1.0f};
      if constexpr (sizeof(CT) == 1) vs = *reinterpret_cast<const f32x4*>(&in.vs[16 * k + 4 * g]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = exp2_fast(s[k][i] - sub);
        l += p;
        s[k][i] = p * vs[i];
      }
    }
    const Frag<NP> p = attn_operand<T, NP>(s);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) o[t][i] *= f;
      const uint4 v = AttnTile<T, 64, DQ, 32>::cols(vl, 0, 16 * t, lane);
#pragma unroll
      for (int e = NP - 1; e >= 0; --e) o[t] = attn_mma<T>(v, p.p[e], o[t]);
    }
    wave_sync();
  }
  l = group_sum(l);

  // the four waves' parts
  __syncthreads();
  float* const red = reinterpret_cast<float*>(tiles);
  float* const mine = red + (wave * 16 + c) * (DQ + 2);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) mine[16 * t + 4 * g + i] = o[t][i];
  if (g == 0) {
    mine[DQ] = mx;
    mine[DQ + 1] = l;
  }
  __syncthreads();
  const int head = threadIdx.x / 16;
  if (head >= nh) return;
  float f[4], top = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) top = fmaxf(top, red[(w * 16 + head) * (DQ + 2) + DQ]);
  const float sub = top == -INFINITY ? 0.0f : top;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = exp2_fast(red[(w * 16 + head) * (DQ + 2) + DQ] - sub);
    sum += f[w] * red[(w * 16 + head) * (DQ + 2) + DQ + 1];
  }
  const long row = static_cast<long>(b) * a.h + head0 + head;
  float* const part = a.part + (row * a.nsplit + split) * (a.D + 2);
  const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
  for (int d = threadIdx.x % 16; d < a.D; d += 16) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) v += f[w] * red[(w * 16 + head) * (DQ + 2) + d];
    if (a.nsplit > 1) part[d] = v;
    else if (o_bf16) st<bf16s>(a.o, row * a.D + d, v * inv);
    else st<float>(a.o, row * a.D + d, v * inv);
  }
  if (a.nsplit > 1 && threadIdx.x % 16 == 0) {
    part[a.D] = top;
    part[a.D + 1] = sum;
  }
}

// Joins the parts of a (sequence, head): one wave each, two channels a lane
__global__ __launch_bounds__(64) void attn_join_kernel(const AttnStepArgs a, int o_bf16) {
  const long row = blockIdx.x;
  const int b = static_cast<int>(row / a.h), lane = threadIdx.x;
  const StepKeys keys = step_keys(a, b);
  const int n = max(1, static_cast<int>((static_cast<long>(keys.n) + a.chunk - 1) / a.chunk));
  const float* const part = a.part + row * a.nsplit * (a.D + 2);
  float top = -INFINITY;
  for (int s = lane; s < n; s += 64) top = fmaxf(top, part[static_cast<long>(s) * (a.D + 2) + a.D]);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
  const float sub = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f, v0 = 0.0f, v1 = 0.0f;
  for (int s = 0; s < n; ++s) {
    const float* const p = part + static_cast<long>(s) * (a.D + 2);
    const float f = exp2_fast(p[a.D] - sub);
    sum += f * p[a.D + 1];
    if (lane < a.D) v0 += f * p[lane];
    if (lane + 64 < a.D) v1 += f * p[lane + 64];
  }
  const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
  const long at = row * a.D + lane;
  if (o_bf16) {
    if (lane < a.D) st<bf16s>(a.o, at, v0 * inv);
    if (lane + 64 < a.D) st<bf16s>(a.o, at + 64, v1 * inv);
  } else {
    if (lane < a.D) st<float>(a.o, at, v0 * inv);
    if (lane + 64 < a.D) st<float>(a.o, at + 64, v1 * inv);
  }
}

template <typename CT, int QP, int DQ>
hipError_t go(const AttnStepLaunch& l, hipStream_t s) {
  const AttnStepArgs& a = l.a;
  const long blocks = static_cast<long>(a.batch) * a.hk * attn_head_tiles(a.h, a.hk) * a.nsplit;
  hipError_t e = timed_launch(s, [&] {
    hipLaunchKernelGGL((attn_step_kernel<CT, QP, DQ>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a,
                       l.in_dtype == kBF16, l.o_dtype == kBF16);
  });
  if (e == hipSuccess && a.nsplit > 1) {
    hipLaunchKernelGGL(attn_join_kernel, dim3(static_cast<unsigned>(a.batch) * a.h), dim3(64), 0, s, a, l.o_dtype == kBF16);
    e = hipGetLastError();
  }
  return e;
}

template <typename CT, int QP>
hipError_t pick(const AttnStepLaunch& l, hipStream_t s) {
  switch (attn_dq(l.a.D)) {
    case 32: return go<CT, QP, 32>(l, s);
    case 64: return go<CT, QP, 64>(l, s);
    case 96: return go<CT, QP, 96>(l, s);
    default: return go<CT, QP, 128>(l, s);
  }
}

}  // namespace

hipError_t launch_attn_step(const AttnStepLaunch& l, hipStream_t s) {
  if (l.a.batch == 0) return hipSuccess;
  if (l.cache_dtype == kF32) return pick<float, 1>(l, s);
  if (l.in_dtype == kBF16) return l.cache_dtype == kAttnE4M3 ? pick<e4m3s, 1>(l, s) : pick<bf16s, 1>(l, s);
  return l.cache_dtype == kAttnE4M3 ? pick<e4m3s, 3>(l, s) : pick<bf16s, 3>(l, s);
}

}  // namespace ssm
