// New tokens into the attention's pages, for gfx950.
//
// A wave takes the keys (or values) of one head of one page that the call meets: the tokens that the page
// holds already, and the new ones.  8 bits: the page's scale is the least power of two s = 2^e with
// max |x| <= 448 s over the new ones, or the page's own where that is larger; products with 1 / s are exact.
// Aligned rows whose groups of 8 elements go evenly into the 64 lanes (heads of 8, 16, 32, 64 or 128) are read at once
// into registers, up to 16 groups a lane (8 in f32), from which the maximum and the codes are formed; others, heads of
// 40, 80 and 96 among them, pass twice over the new rows, for the maximum and (from L2) for the codes.  A page whose
// scale grows has its codes read and written again.  Bound by the reads and writes: 8192 tokens of 8 heads of 128 in
// 8 bits 14.7 us, 3.4 TB/s (in two passes 24).
#include "attn.h"
#include "delta_device.h"

namespace ssm {
namespace {

struct e4m3s {
  uint8_t bits;
};

// (the widest row of 8 elements: two 16-byte loads)
template <typename IN>
__device__ __forceinline__ void load_in8(const IN* row, int c, int D, int vec, float (&x)[8]) {
  Row8<IN> r;
  r.load(row, c, D, vec != 0);
  r.get(D - c, x);
}

__device__ __forceinline__ uint2 codes_of(const float (&x)[8]) {
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
  return make_uint2(lo, hi);
}
__device__ __forceinline__ void values_of(uint2 w, float (&x)[8]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w.x, true);
  const f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8(w.y, false), d = __builtin_amdgcn_cvt_pk_f32_fp8(w.y, true);
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  x[4] = c.x; x[5] = c.y; x[6] = d.x; x[7] = d.y;
}

// 8 elements of a row of the cache, from channel c on (a page's row is D elements)
__device__ __forceinline__ void put_row(bf16s* p, const float (&x)[8], int left, int vec) {
  if (vec) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_hi(x[0], x[1]), pack_hi(x[2], x[3]), pack_hi(x[4], x[5]), pack_hi(x[6], x[7]));
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < left) p[i].bits = static_cast<uint16_t>(__float_as_uint(x[i]) >> 16);  // (it came from bf16)
}
__device__ __forceinline__ void put_row(float* p, const float (&x)[8], int left, int vec) {
  if (vec) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < left) p[i] = x[i];
}
__device__ __forceinline__ void put_codes(e4m3s* p, uint2 w, int left, int vec) {
  if (vec) {
    *reinterpret_cast<uint2*>(p) = w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < left) p[i].bits = static_cast<uint8_t>((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
}
__device__ __forceinline__ uint2 get_codes(const e4m3s* p, int left, int vec) {
  if (vec) return *reinterpret_cast<const uint2*>(p);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < left) w[i / 4] |= static_cast<uint32_t>(p[i].bits) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}

// Exponent of the least power of two s with top <= 448 s (448 = 1.75 2^8), -100 at least
__device__ __forceinline__ int scale_exp(float top) {
  const uint32_t b = __float_as_uint(top);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, -100);
}

template <typename IN, typename CT>
__global__ __launch_bounds__(256) void attn_cache_kernel(const AttnCacheArgs a, long items) {
  const long item = static_cast<long>(blockIdx.x) * 4 + threadIdx.x / 64;  // (slot, head, keys or values)
  if (item >= items) return;  // whole waves leave together
  const int lane = threadIdx.x % 64;
  const bool values = item & 1;
  const int kh = static_cast<int>((item >> 1) % a.hk);
  const long slot = (item >> 1) / a.hk;
  long t0;
  int s, n, at;  // first token, sequence, its new tokens, the page's number among those it meets
  if (a.cu) {
    int lo = 0, hi = a.nseq - 1;
    const auto offset = [&](int i) { const long b = a.cu[i]; return b < 0 ? 0 : (b > a.tokens ? a.tokens : b); };
    while (lo < hi) {  // the last sequence whose slots begin at or before this one
      const int mid = (lo + hi + 1) >> 1;
      if (offset(mid) / a.page + 2L * mid <= slot) lo = mid;
      else hi = mid - 1;
    }
    s = lo;
    t0 = offset(s);
    n = static_cast<int>(max(0L, offset(s + 1) - t0));
    const long x = slot - (t0 / a.page + 2L * s);
    if (x < 0) return;
    at = static_cast<int>(x);
  } else {
    const int per = (a.seqlen - 1 + a.page - 1) / a.page + 1;
    s = static_cast<int>(slot / per);
    at = static_cast<int>(slot % per);
    t0 = static_cast<long>(s) * a.seqlen;
    n = a.seqlen;
  }
  const int held = max(0, a.lens[s]);
  const long entry = held / a.page + static_cast<long>(at);
  const long begin = entry * a.page;                                   // position of the page's first row
  const long end = min(begin + a.page, static_cast<long>(held) + n);   // .. past the last row written
  if (n == 0 || begin >= static_cast<long>(held) + n || entry >= a.table_rows) return;
  const int pg = a.table[static_cast<long>(s) * a.table_rows + entry];
  if (pg < 0 || pg >= a.pages) return;
  const int keep = static_cast<int>(max(0L, held - begin)), rows = static_cast<int>(end - begin);  // rows held, rows at the end
  const long stride = values ? a.v_stride : a.k_stride;
  const IN* const src = static_cast<const IN*>(values ? a.v : a.k) + static_cast<long>(kh) * a.D;
  const long first = t0 + begin - held;                                // token of row 0 (rows from keep on exist)
  const long ph = static_cast<long>(pg) * a.hk + kh;
  CT* const dst = static_cast<CT*>(values ? a.v_cache : a.k_cache) + ph * a.page * a.D;
  const int groups = (a.D + 7) / 8, count = (rows - keep) * groups;

  // the page's scale, of new rows with this largest value; codes held are put to it where it grows
  const auto scaled = [&](float top) {
    float* const scale = (values ? a.v_scale : a.k_scale) + ph;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
    float to = ldexpf(1.0f, scale_exp(top));
    if (keep > 0) {
      const float had = *scale;
      if (had >= to) return had;
      if constexpr (sizeof(CT) == 1) {
        const float f = had / to;
        for (int e = lane; e < keep * groups; e += 64) {
          const int row = e / groups, c = e % groups * 8, left = a.D - c;
          CT* const p = dst + static_cast<long>(row) * a.D + c;
          float x[8];
          values_of(get_codes(p, left, a.vec), x);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= f;
          put_codes(p, codes_of(x), left, a.vec);
        }
      }
    }
    if (lane == 0) *scale = to;
    return to;
  };
  const auto largest = [&](const float (&x)[8], float top) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float m = fabsf(x[i]);
      top = fmaxf(top, m < INFINITY ? m : 0.0f);
    }
    return top;
  };
  const auto put = [&](int row, int c, float (&x)[8], float inv) {
    CT* const p = dst + static_cast<long>(row) * a.D + c;
    if constexpr (sizeof(CT) == 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= inv;
      put_codes(p, codes_of(x), a.D - c, a.vec);
    } else {
      put_row(p, x, a.D - c, a.vec);
    }
  };

  constexpr int kHold = sizeof(IN) == 2 ? 16 : 8;
  const int per = 64 / groups;  // rows of the wave
  if (a.vec && per * groups == 64 && rows - keep <= kHold * per) {
    const int r0 = keep + lane / groups, c = lane % groups * 8;
    Row8<IN> held_rows[kHold];
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (keep + i * per < rows) held_rows[i].load(src + (first + min(r0 + i * per, rows - 1)) * stride, c, a.D, true);
    float inv = 1.0f;
    if constexpr (sizeof(CT) == 1) {
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < kHold; ++i) {
        if (keep + i * per >= rows) continue;
        float x[8];
        held_rows[i].get(8, x);
        top = largest(x, top);
      }
      inv = 1.0f / scaled(top);
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      if (r0 + i * per >= rows) continue;
      float x[8];
      held_rows[i].get(8, x);
      put(r0 + i * per, c, x, inv);
    }
    return;
  }

  float inv = 1.0f;
  if constexpr (sizeof(CT) == 1) {
    float top = 0.0f;
    for (int e = lane; e < count; e += 64) {
      float x[8];
      load_in8<IN>(src + (first + keep + e / groups) * stride, e % groups * 8, a.D, a.vec, x);
      top = largest(x, top);
    }
    inv = 1.0f / scaled(top);
  }
  for (int e = lane; e < count; e += 64) {
    float x[8];
    const int row = keep + e / groups, c = e % groups * 8;
    load_in8<IN>(src + (first + row) * stride, c, a.D, a.vec, x);
    put(row, c, x, inv);
  }
}

template <typename IN, typename CT>
hipError_t go(const AttnCacheArgs& a, hipStream_t s) {
  const long items = attn_cache_slots(a) * a.hk * 2;
  return timed_launch(s, [&] {
    hipLaunchKernelGGL((attn_cache_kernel<IN, CT>), dim3(static_cast<unsigned>((items + 3) / 4)), dim3(256), 0, s, a, items);
  });
}

}  // namespace

hipError_t launch_attn_cache(const AttnCacheArgs& a, int in_dtype, int cache_dtype, hipStream_t s) {
  if (a.tokens == 0 || a.nseq == 0) return hipSuccess;
  if (in_dtype == kBF16) return cache_dtype == kAttnE4M3 ? go<bf16s, e4m3s>(a, s) : go<bf16s, bf16s>(a, s);
  return cache_dtype == kAttnE4M3 ? go<float, e4m3s>(a, s) : go<float, float>(a, s);
}

}  // namespace ssm
