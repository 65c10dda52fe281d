// One query of each sequence over its pages, for gfx950.
//
// The visible keys of a sequence, [0, sinks) and those of its window, are counted through as one range,
// which is cut into parts of a.chunk keys; a workgroup takes one part for the (up to 16) query heads of a
// key head, its four waves the part's tiles of 32 keys (16 in f32) in turn.  Per tile, as in the forward,
//   S^T = K Q^T,  P = 2^(S - m),  O^T += V^T P^T
// with K straight from memory as an operand (a lane holds channels of a key), V through LDS, where it is
// read transposed.  Codes are widened where they become operands (e4m3 is exact in bf16), the scale of a
// page goes to S and to P.  32-bit operands (q in f32, P) enter as three bf16 parts.
// Loads run ahead: the page entries two tiles, keys, values and scales one, and only a tile with keys that
// are left out takes branches.  Waves, then parts (a second kernel), are joined by their maxima and sums.
// The step reads the visible cache once and is bound by that.
#include "attn_device.h"

namespace ssm {
namespace {

struct e4m3s {
  uint8_t bits;
};

// Elements of the cache, CH of them in 16 bytes, and their operands
template <typename CT>
struct StepEl {  // f32 and bf16: as they are stored
  using Op = CT;
  static constexpr int kUnitBytes = 16;  // of an operand
  static __device__ __forceinline__ uint4 op(const uint32_t* w) { return make_uint4(w[0], w[1], w[2], w[3]); }
  static __device__ __forceinline__ uint4 chunk(const CT* row, int c, int D, int vec) { return attn_chunk<CT>(row, c, D, vec); }
};
template <>
struct StepEl<e4m3s> {  // 8 codes to 8 bf16
  using Op = bf16s;
  static constexpr int kUnitBytes = 8;
  static __device__ __forceinline__ uint4 op(const uint32_t* w) {
    return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], 1.0f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], 1.0f, true)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], 1.0f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], 1.0f, true)));
  }
  static __device__ __forceinline__ uint4 chunk(const e4m3s* row, int c, int D, int vec) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (vec > 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (c + 8 * h < D) {
          const uint2 x = *reinterpret_cast<const uint2*>(row + c + 8 * h);
          w[2 * h] = x.x;
          w[2 * h + 1] = x.y;
        }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (c + i < D) w[i / 4] |= static_cast<uint32_t>(row[c + i].bits) << (8 * (i & 3));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Visible keys of a sequence: x counts them through
struct StepKeys {
  int ns, lo, n;  // sinks ahead of the window, its first key, keys in all
  __device__ __forceinline__ int key(int x) const { return x < ns ? x : x - ns + lo; }
};
__device__ __forceinline__ StepKeys step_keys(const AttnStepArgs& a, int b) {
  const int len = a.pages > 0 ? min(max(a.lens[b], 0), a.table_rows * a.page) : 0;
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

// V in LDS as it is stored; transposed: row = channel c0 + lane % 16, along the tile's keys
template <typename CT, int kStride>
__device__ __forceinline__ uint4 step_cols(const unsigned char* lds, int c0, int lane) {
  const int g = lane / 16, j = lane % 16;
  if constexpr (sizeof(CT) == 1) {
    // lane j of a group of 16 reads 8 codes of its row; it gets the eight rows' codes of column j
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    typedef __attribute__((address_space(3))) i32x2* lds_ptr;
    const int row = 4 * g + j / 2 + (j < 8 ? 0 : 12);  // 4 g .., 16 + 4 g ..
    const i32x2 v = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_ptr)(lds + row * kStride + c0 + j % 2 * 8));
    const uint32_t w[2] = {static_cast<uint32_t>(v[0]), static_cast<uint32_t>(v[1])};
    return StepEl<CT>::op(w);
  } else if constexpr (sizeof(CT) == 2) {  // the same with 4 values of a row
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4* lds_ptr;
    const unsigned char* const p = lds + (4 * g + j / 4) * kStride + c0 * 2 + j % 4 * 8;
    const uint2 x = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p)));
    const uint2 y = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 16 * kStride)));
    return make_uint4(x.x, x.y, y.x, y.y);
  } else {
    const unsigned char* const p = lds + 4 * g * kStride + (c0 + j) * 4;
    return make_uint4(*reinterpret_cast<const uint32_t*>(p), *reinterpret_cast<const uint32_t*>(p + kStride),
                      *reinterpret_cast<const uint32_t*>(p + 2 * kStride), *reinterpret_cast<const uint32_t*>(p + 3 * kStride));
  }
}

// CT: the cache, QP: parts of q, DQ: channels (a multiple of 32), VEC: rows of aligned 16-byte groups
template <typename CT, int QP, int DQ, bool VEC>
__global__ __launch_bounds__(256, VEC && QP == 1 && sizeof(CT) < 4 ? 3 : 2) void attn_step_kernel(const AttnStepArgs a, int o_bf16) {
  using C = StepEl<CT>;
  using T = typename C::Op;
  using E = AttnEl<T>;
  constexpr int NP = sizeof(T) == 2 ? 3 : 1;               // parts of P
  constexpr int TK = sizeof(T) == 2 ? 32 : 16;             // keys of a tile: one unit
  constexpr int KT = TK / 16, KS = DQ / E::kUnit, NT = DQ / 16;
  constexpr int UW = C::kUnitBytes / 4;                    // words of K's units
  constexpr int kRagged = (DQ - 32) / E::kUnit;            // units from here on may hold channels past D
  constexpr int W8 = sizeof(CT) == 1 ? DQ / 64 * 2 : 0;    // units loaded two at a time, 16 codes a lane
  constexpr int CH = 16 / static_cast<int>(sizeof(CT));    // elements of 16 bytes
  constexpr int CPR = DQ / CH, NV = TK * CPR / 64;         // those of a row, of a lane
  constexpr int VS = DQ * static_cast<int>(sizeof(CT)) + 16;
  struct __align__(16) Info {                              // of a tile's keys, read 16 bytes at a time
    long base[TK];                                         // first element of the row
    float add[TK], ks[TK], vs[TK];                         // 0, or -infinity: left out; scales
  };
  static_assert(alignof(Info) == 16 && sizeof(long) * TK % 16 == 0 && sizeof(float) * TK % 16 == 0, "16-byte reads");
  constexpr int kRed = 4 * 16 * (DQ + 2) * 4, kTiles = 4 * TK * VS;
  __shared__ __align__(16) unsigned char tiles[kTiles > kRed ? kTiles : kRed];
  __shared__ Info infos[4][2];

  const int g_heads = a.h / a.hk, ht = (g_heads + kAttnStepHeads - 1) / kAttnStepHeads;
  // first every sequence's first part: the later ones, which shorter sequences do not have, would else all
  // lie on some of the 8 XCDs, round which workgroups are dealt (64 x 8 groups in two parts: 178 us)
  const unsigned groups = gridDim.x / a.nsplit, split = blockIdx.x / groups;
  unsigned r = blockIdx.x % groups;
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
  // channels of unit u in lane group g
  const auto chan = [&](int u) { return u < W8 ? 64 * (u / 2) + 16 * g + 8 * (u % 2) : u * E::kUnit + g * E::kVec; };

  // q as columns, in parts
  Frag<QP> q[KS];
  {
    const long row = b * a.q_stride + static_cast<long>(head0 + c) * a.D;
#pragma unroll
    for (int u = 0; u < KS; ++u) {
      const int d = chan(u);
      if constexpr (QP == 1) {
        q[u].p[0] = make_uint4(0u, 0u, 0u, 0u);
        if (c < nh) q[u].p[0] = attn_chunk<T>(static_cast<const T*>(a.q) + row, d, a.D, a.q_vec);
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
  struct Page {  // of one key a lane
    int pg, row;
  };
  const auto page_of = [&](int x0) {
    Page p{-1, 0};
    const int x = x0 + lane;
    if (lane < TK && x < end) {
      const int j = keys.key(x);
      int e;
      if (a.page_shift >= 0) {
        e = j >> a.page_shift;
        p.row = j & (a.page - 1);
      } else {
        e = j / a.page;
        p.row = j - e * a.page;
      }
      p.pg = a.table[static_cast<long>(b) * a.table_rows + e];
    }
    return p;
  };
  float ks_next = 0.0f, vs_next = 0.0f;
  bool there_next = false;
  // a tile's row addresses; its scales are loaded, and put there by the time they are used.  Whether every
  // key of it is there.
  const auto put_info = [&](Info& to, Page p) {
    const bool in = p.pg >= 0 && p.pg < a.pages;
    if (lane < TK) {
      const long ph = static_cast<long>(in ? p.pg : 0) * a.hk + kh;
      to.base[lane] = (ph * a.page + (in ? p.row : 0)) * a.D;
      to.add[lane] = in ? 0.0f : -INFINITY;
      if constexpr (sizeof(CT) == 1) {
        there_next = in;
        ks_next = a.k_scale[ph];
        vs_next = a.v_scale[ph];
      }
    }
    return __all(lane >= TK || in) != 0;
  };
  const CT* const kc = static_cast<const CT*>(a.k_cache);
  const CT* const vc = static_cast<const CT*>(a.v_cache);
  uint32_t kn[KT][KS * UW];
  uint4 vn[NV];
  const auto fetch = [&](const Info& in, bool whole) {
    // (channels past D: in the aligned form they read channel 0 on; V's are not stored, K's are put to zero where they
    // are used, as an infinite one beside the zeros of q would not vanish; a code is never infinite)
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const CT* const row = kc + in.base[16 * k + c];
      const bool there = whole || in.add[16 * k + c] == 0.0f;
#pragma unroll
      for (int u = 0; u < KS; u += u < W8 ? 2 : 1) {
        const int d = chan(u);
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (there) {
          if constexpr (VEC && (sizeof(CT) > 1 || W8 > 0)) {
            if (sizeof(CT) > 1 || u < W8) {
              const uint4 x = *reinterpret_cast<const uint4*>(row + (d < a.D ? d : 0));
              w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(row + (d < a.D ? d : 0));
              w[0] = x.x; w[1] = x.y;
            }
          } else if constexpr (VEC) {
            const uint2 x = *reinterpret_cast<const uint2*>(row + (d < a.D ? d : 0));
            w[0] = x.x; w[1] = x.y;
          } else {
            const uint4 x = C::chunk(row, d, a.D, a.vec);
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
          }
        }
#pragma unroll
        for (int i = 0; i < (u < W8 ? 2 * UW : UW); ++i) kn[k][u * UW + i] = w[i];
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int x = lane + 64 * i, d = x % CPR * CH;
      const CT* const row = vc + in.base[x / CPR];
      vn[i] = make_uint4(0u, 0u, 0u, 0u);
      if (whole || in.add[x / CPR] == 0.0f) {
        if constexpr (VEC) vn[i] = *reinterpret_cast<const uint4*>(row + (d < a.D ? d : 0));
        else vn[i] = C::chunk(row, d, a.D, a.vec);
      }
    }
  };

  float mx = -INFINITY, l = 0.0f;
  f32x4 o[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) o[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  Page next{-1, 0};
  bool whole = false;
  if (first < end) {
    const Page p = page_of(first);
    next = page_of(first + 4 * TK);
    whole = put_info(infos[wave][0], p);
    wave_sync();
    fetch(infos[wave][0], whole);
  }
  int at = 0;
  for (int x0 = first; x0 < end; x0 += 4 * TK, at ^= 1) {
    Info& in = infos[wave][at];
    if constexpr (sizeof(CT) == 1)
      if (lane < TK) {
        in.ks[lane] = ks_next * cs;
        in.vs[lane] = there_next ? vs_next : 0.0f;  // (P is zero there, but not its product with what is no number)
      }
    const bool whole_next = put_info(infos[wave][at ^ 1], next);
    next = page_of(x0 + 8 * TK);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int x = lane + 64 * i;
      *reinterpret_cast<uint4*>(vl + x / CPR * VS + x % CPR * 16) = vn[i];
    }
    f32x4 s[KT];
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      s[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < KS; ++u) {
        uint4 kf = C::op(&kn[k][u * UW]);
        if (VEC && sizeof(CT) > 1 && u >= kRagged && chan(u) >= a.D) kf = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int p = QP - 1; p >= 0; --p) s[k] = attn_mma<T>(kf, q[u].p[p], s[k]);
      }
    }
    wave_sync();
    if (x0 + 4 * TK < end) fetch(infos[wave][at ^ 1], whole_next);
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      f32x4 ks = {cs, cs, cs, cs};
      if constexpr (sizeof(CT) == 1) ks = *reinterpret_cast<const f32x4*>(&in.ks[16 * k + 4 * g]);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[k][i] *= ks[i];
    }
    if (!whole) {
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        const f32x4 add = *reinterpret_cast<const f32x4*>(&in.add[16 * k + 4 * g]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[k][i] = add[i] == 0.0f ? s[k][i] : -INFINITY;
      }
    }
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, s[k][i]);
    top = group_max(top);
    if (__any(top > mx + 8.0f)) {  // (a maximum that lies 2^8 behind at most serves as well)
      const float to = fmaxf(mx, top);
      const float f = mx == -INFINITY ? 0.0f : exp2_fast(mx - to);
      mx = to;
      l *= f;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][i] *= f;
    }
    const float sub = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      f32x4 vs = {1.0f, 1.0f, 1.0f, 1.0f};
      if constexpr (sizeof(CT) == 1) vs = *reinterpret_cast<const f32x4*>(&in.vs[16 * k + 4 * g]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = exp2_fast(s[k][i] - sub);
        l += p;
        s[k][i] = sizeof(CT) == 1 ? p * vs[i] : p;
      }
    }
    const Frag<NP> p = attn_operand<T, NP>(s);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint4 v = step_cols<CT, VS>(vl, 16 * t, lane);
#pragma unroll
      for (int e = NP - 1; e >= 0; --e) o[t] = attn_mma<T>(v, p.p[e], o[t]);
    }
    whole = whole_next;
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
  float* const part = a.part + (row * a.nsplit + split) * DQ;
  const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
  for (int d = threadIdx.x % 16; d < (a.nsplit > 1 ? DQ : a.D); d += 16) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) v += f[w] * red[(w * 16 + head) * (DQ + 2) + d];
    if (a.nsplit > 1) part[d] = v;
    else if (o_bf16) st<bf16s>(a.o, row * a.D + d, v * inv);
    else st<float>(a.o, row * a.D + d, v * inv);
  }
  if (a.nsplit > 1 && threadIdx.x % 16 == 0) {
    float* const stat = a.part_stat + (row * a.nsplit + split) * 2;
    stat[0] = top;
    stat[1] = sum;
  }
}

// Joins the parts of a (sequence, head).  DQ / 4 lanes hold four channels each, the 1024 / DQ groups of them
// take the parts in turn; the groups' sums meet in LDS.
template <int DQ>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnStepArgs a, int o_bf16) {
  constexpr int L = DQ / 4, G = 256 / L;  // (96 channels: 24 lanes, 10 groups)
  __shared__ __align__(16) float red[G][DQ];
  __shared__ float stat[4];
  const long row = blockIdx.x;
  const int b = static_cast<int>(row / a.h), lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const StepKeys keys = step_keys(a, b);
  const int n = max(1, static_cast<int>((static_cast<long>(keys.n) + a.chunk - 1) / a.chunk));
  const float* const stats = a.part_stat + row * a.nsplit * 2;
  float top = -INFINITY;
  for (int s = threadIdx.x; s < n; s += 256) top = fmaxf(top, stats[2 * s]);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
  if (lane == 0) stat[wave] = top;
  __syncthreads();
  top = fmaxf(fmaxf(stat[0], stat[1]), fmaxf(stat[2], stat[3]));
  const float sub = top == -INFINITY ? 0.0f : top;
  const int x = threadIdx.x % L, grp = threadIdx.x / L;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sum = 0.0f;
  if (grp < G) {
    const float4* const part = reinterpret_cast<const float4*>(a.part + row * a.nsplit * DQ) + x;
#pragma unroll 4
    for (int s = grp; s < n; s += G) {
      const float f = exp2_fast(stats[2 * s] - sub);
      const float4 p = part[static_cast<long>(s) * L];
      sum = fmaf(f, stats[2 * s + 1], sum);
      v[0] = fmaf(f, p.x, v[0]);
      v[1] = fmaf(f, p.y, v[1]);
      v[2] = fmaf(f, p.z, v[2]);
      v[3] = fmaf(f, p.w, v[3]);
    }
    *reinterpret_cast<float4*>(&red[grp][4 * x]) = make_float4(v[0], v[1], v[2], v[3]);
  }
  __shared__ float sums[G];
  if (grp < G && x == 0) sums[grp] = sum;
  __syncthreads();
  const int d = threadIdx.x;
  if (d >= a.D) return;
  float o = 0.0f, total = 0.0f;
#pragma unroll
  for (int i = 0; i < G; ++i) {
    o += red[i][d];
    total += sums[i];
  }
  const float inv = total > 0.0f || total != total ? 1.0f / total : 0.0f;
  if (o_bf16) st<bf16s>(a.o, row * a.D + d, o * inv);
  else st<float>(a.o, row * a.D + d, o * inv);
}

template <typename CT, int QP, int DQ, bool VEC>
hipError_t go(const AttnStepLaunch& l, hipStream_t s) {
  const AttnStepArgs& a = l.a;
  const long blocks = static_cast<long>(a.batch) * a.hk * attn_head_tiles(a.h, a.hk) * a.nsplit;
  hipError_t e = timed_launch(s, [&] {
    hipLaunchKernelGGL((attn_step_kernel<CT, QP, DQ, VEC>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a,
                       l.o_dtype == kBF16);
  });
  if (e == hipSuccess && a.nsplit > 1) {
    hipLaunchKernelGGL((attn_join_kernel<DQ>), dim3(static_cast<unsigned>(a.batch) * a.h), dim3(256), 0, s, a, l.o_dtype == kBF16);
    e = hipGetLastError();
  }
  return e;
}

template <typename CT, int QP, bool VEC>
hipError_t pick_d(const AttnStepLaunch& l, hipStream_t s) {
  switch (attn_dq(l.a.D)) {
    case 32: return go<CT, QP, 32, VEC>(l, s);
    case 64: return go<CT, QP, 64, VEC>(l, s);
    case 96: return go<CT, QP, 96, VEC>(l, s);
    default: return go<CT, QP, 128, VEC>(l, s);
  }
}
template <typename CT, int QP>
hipError_t pick(const AttnStepLaunch& l, hipStream_t s) {
  return l.a.vec == 2 ? pick_d<CT, QP, true>(l, s) : pick_d<CT, QP, false>(l, s);
}

}  // namespace

hipError_t launch_attn_step(const AttnStepLaunch& l, hipStream_t s) {
  if (l.a.batch == 0) return hipSuccess;
  if (l.cache_dtype == kF32) return pick<float, 1>(l, s);
  if (l.in_dtype == kBF16) return l.cache_dtype == kAttnE4M3 ? pick<e4m3s, 1>(l, s) : pick<bf16s, 1>(l, s);
  return l.cache_dtype == kAttnE4M3 ? pick<e4m3s, 3>(l, s) : pick<bf16s, 3>(l, s);
}

}  // namespace ssm
