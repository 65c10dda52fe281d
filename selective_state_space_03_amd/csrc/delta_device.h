// Device helpers of the gated delta rule's kernels: 16 x 16 x 32 bf16 matrix
// products on operands held as one to three bf16 parts, and the sequence and
// chunk bookkeeping.
//
// Operand fragment (A: row = lane % 16, B: column = lane % 16): 8 values along
// the contraction per lane, in slots (lane / 16, j).  Any assignment of
// contraction indices to slots gives the same product as long as A and B agree:
//   natural:  32 s + 8 (lane / 16) + j         (contraction over tokens)
//   tiled:    32 s + 16 (j / 4) + 4 (lane / 16) + j % 4   (contraction over key
//             channels: the order in which an accumulator tile holds its rows,
//             so a state tile is an operand without any exchange of lanes)
// Accumulator tile: column = lane % 16, row = 4 (lane / 16) + i.
#pragma once
#include "delta.h"
#include "ssm_device.h"

namespace ssm {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <int NP>
struct Frag {
  uint4 p[NP];
};

// Two floats' leading 16 bits, packed (the first in the low half).
__device__ __forceinline__ uint32_t pack_hi(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ uint32_t pack_rne(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float hi_part(float a) { return __uint_as_float(__float_as_uint(a) & 0xffff0000u); }

// Splits two floats into NP bf16 parts: leading bits by truncation (the
// remainder is exact), the last part rounded to nearest.  Three parts hold all
// 24 bits of the significand.
template <int NP>
__device__ __forceinline__ void split2(float a, float b, uint32_t (&out)[NP]) {
#pragma unroll
  for (int p = 0; p < NP - 1; ++p) {
    out[p] = pack_hi(a, b);
    a -= hi_part(a);
    b -= hi_part(b);
  }
  out[NP - 1] = pack_rne(a, b);
}

template <int NP>
__device__ __forceinline__ Frag<NP> split8(const float (&v)[8]) {
  Frag<NP> f;
  uint32_t w[4][NP];
#pragma unroll
  for (int i = 0; i < 4; ++i) split2<NP>(v[2 * i], v[2 * i + 1], w[i]);
#pragma unroll
  for (int p = 0; p < NP; ++p) f.p[p] = make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
  return f;
}

// acc += A B over the products of parts whose weight reaches the longer
// operand's last part.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mma(const Frag<NA>& a, const Frag<NB>& b, f32x4 acc) {
  constexpr int n = NA > NB ? NA : NB;
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
      if (i + j < n)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.p[i]),
                                                      __builtin_bit_cast(bf16x8, b.p[j]), acc, 0, 0, 0);
  return acc;
}

// Fragments in memory: [fragment][part][lane] of 16 bytes.
template <int NP>
__device__ __forceinline__ Frag<NP> load_frag(const unsigned char* base, int idx, int lane) {
  Frag<NP> f;
  const uint4* p = reinterpret_cast<const uint4*>(base) + (static_cast<size_t>(idx) * NP) * 64 + lane;
#pragma unroll
  for (int i = 0; i < NP; ++i) f.p[i] = p[i * 64];
  return f;
}
template <int NP>
__device__ __forceinline__ void store_frag(unsigned char* base, int idx, int lane, const Frag<NP>& f) {
  uint4* p = reinterpret_cast<uint4*>(base) + (static_cast<size_t>(idx) * NP) * 64 + lane;
#pragma unroll
  for (int i = 0; i < NP; ++i) p[i * 64] = f.p[i];
}

template <int NP>
__device__ __forceinline__ void zero_frag(Frag<NP>& f) {
#pragma unroll
  for (int i = 0; i < NP; ++i) f.p[i] = make_uint4(0u, 0u, 0u, 0u);
}

// Fragments kept of a lower (upper) triangular 64 x 64 operand: row tile i
// needs the token step s (32 columns) only where it meets the triangle.
__device__ __forceinline__ int low_frag(int i, int s) { return i < 2 ? i : 2 * i - 2 + s; }
__device__ __forceinline__ int up_frag(int i, int s) { return i < 2 ? 2 * i + s : i + 2; }

// 8 consecutive values of a row of `width`, as loaded, and widened.  vec: whole
// aligned groups (width a multiple of 8); columns past the end read the row's
// first ones and are dropped when widened.
template <typename IN>
struct Row8;
template <>
struct Row8<bf16s> {
  uint4 a;
  __device__ __forceinline__ void load(const bf16s* row, int c, int width, bool vec) {
    if (vec) {
      a = *reinterpret_cast<const uint4*>(row + (c < width ? c : 0));
    } else {
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = row[min(c + i, width - 1)].bits;
      a = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
  }
  __device__ __forceinline__ void get(int left, float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = 2 * i < left ? __uint_as_float(w[i] << 16) : 0.0f;
      v[2 * i + 1] = 2 * i + 1 < left ? __uint_as_float(w[i] & 0xffff0000u) : 0.0f;
    }
  }
};
template <>
struct Row8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* row, int c, int width, bool vec) {
    if (vec) {
      const float4* p = reinterpret_cast<const float4*>(row + (c < width ? c : 0));
      a = p[0];
      b = p[1];
    } else {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = row[min(c + i, width - 1)];
      a = make_float4(v[0], v[1], v[2], v[3]);
      b = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
  __device__ __forceinline__ void get(int left, float (&v)[8]) const {
    const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? x[i] : 0.0f;
  }
};

// 8 values into LDS in the inputs' type (they come from it)
__device__ __forceinline__ void put8(bf16s* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_hi(v[0], v[1]), pack_hi(v[2], v[3]), pack_hi(v[4], v[5]), pack_hi(v[6], v[7]));
}
__device__ __forceinline__ void put8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Waits for this wave's LDS accesses and joins the workgroup; global loads and
// stores stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

struct DeltaSeq {
  long t0;     // first token
  int len;
  long slot0;  // first chunk slot
};

// Offsets outside [0, tokens] or out of order are clamped, so no access leaves
// the tensors whatever cu holds.  Sequence s of a packed call owns the slots
// from cu[s] / 64 + s on, which leaves every sequence room for its chunks
// without a prefix sum over the sequences before it.
__device__ __forceinline__ DeltaSeq delta_seq(const DeltaArgs& a, int s) {
  DeltaSeq q;
  if (a.cu) {
    long b = a.cu[s], e = a.cu[s + 1];
    b = b < 0 ? 0 : (b > a.tokens ? a.tokens : b);
    e = e < b ? b : (e > a.tokens ? a.tokens : e);
    q.t0 = b;
    q.len = static_cast<int>(e - b);
    q.slot0 = b / kDeltaC + s;
  } else {
    q.t0 = static_cast<long>(s) * a.seqlen;
    q.len = a.seqlen;
    q.slot0 = static_cast<long>(s) * ((a.seqlen + kDeltaC - 1) / kDeltaC);
  }
  return q;
}

// The chunk in a slot: its first token and length (0: an unused slot).
__device__ __forceinline__ int delta_chunk(const DeltaArgs& a, long slot, long* t0) {
  int s;
  if (a.cu) {
    int lo = 0, hi = a.nseq - 1;
    while (lo < hi) {  // the last sequence whose slots begin at or before this one
      const int mid = (lo + hi + 1) >> 1;
      long b = a.cu[mid];
      b = b < 0 ? 0 : (b > a.tokens ? a.tokens : b);
      if (b / kDeltaC + mid <= slot) lo = mid;
      else hi = mid - 1;
    }
    s = lo;
  } else {
    s = static_cast<int>(slot / ((a.seqlen + kDeltaC - 1) / kDeltaC));
  }
  const DeltaSeq q = delta_seq(a, s);
  const long c = slot - q.slot0;
  const long left = q.len - c * kDeltaC;
  if (c < 0 || left <= 0) return 0;
  *t0 = q.t0 + c * kDeltaC;
  return left < kDeltaC ? static_cast<int>(left) : kDeltaC;
}

// Whether a token lies in one of the packed sequences.
__device__ __forceinline__ bool delta_inside(const DeltaArgs& a, long t) {
  int lo = 0, hi = a.nseq - 1;
  if (hi < 0) return false;
  while (lo < hi) {  // the last sequence that begins at or before it
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  const DeltaSeq q = delta_seq(a, lo);
  return t >= q.t0 && t < q.t0 + q.len;
}

// Workgroup b's (group, slice) for `slices` workgroups per group: the slices of
// a group go to one XCD (blocks are dealt round the 8 XCDs), whose L2 then
// serves the group's shared operands.  The grid holds 8 ceil(groups / 8) slices
// workgroups; group >= groups: nothing to do.
__device__ __forceinline__ void xcd_group(unsigned b, unsigned slices, long* group, unsigned* slice) {
  const unsigned x = b & 7u, rest = b >> 3;
  *slice = rest % slices;
  *group = static_cast<long>(rest / slices) * 8 + x;
}

}  // namespace ssm
