// Device helpers of the window attention's kernels: 16 x 16 matrix tiles of bf16 or
// f32 operands, tiles of rows in LDS, and the bookkeeping of sequences.
//
// Every operand is held as 16 bytes per lane (row or column = lane % 16, g = lane / 16):
//   along channels: unit u holds the channels kUnit u + kVec g + i
//   along tokens (transposed reads, and accumulator tiles handed on as operands):
//     bf16: token 16 (i / 4) + 4 g + i % 4 of 32,  f32: token 4 g + i of 16
// An accumulator tile has column = lane % 16, row = 4 g + i, so that tiles whose rows are
// tokens are operands of the next product over tokens without an exchange of lanes.
#pragma once
#include "attn.h"
#include "delta_device.h"

namespace ssm {

template <typename T>
struct AttnEl;
template <>
struct AttnEl<bf16s> {
  static constexpr int kVec = 8;     // elements in 16 bytes
  static constexpr int kUnit = 32;   // depth of a product of 16-byte operands
  static constexpr int kTile = 64;   // keys per step of the loops
};
template <>
struct AttnEl<float> {
  static constexpr int kVec = 4;
  static constexpr int kUnit = 16;
  static constexpr int kTile = 32;
};

// acc += A B over one unit
template <typename T>
__device__ __forceinline__ f32x4 attn_mma(uint4 a, uint4 b, f32x4 acc) {
  if constexpr (sizeof(T) == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  } else {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], y[i], acc, 0, 0, 0);
    return acc;
  }
}

// 16 bytes of a row of D channels from channel c on, zeros past the row's end
template <typename T>
__device__ __forceinline__ uint4 attn_chunk(const T* row, int c, int D, int vec) {
  constexpr int n = AttnEl<T>::kVec;
  if (vec == 2) return load16_if(row + c, c < D);
  uint4 r = make_uint4(0u, 0u, 0u, 0u);
  if (vec == 1) {
    const uint2* p = reinterpret_cast<const uint2*>(row + c);
    if (c < D) {
      const uint2 x = p[0];
      r.x = x.x;
      r.y = x.y;
    }
    if (c + n / 2 < D) {
      const uint2 x = p[1];
      r.z = x.x;
      r.w = x.y;
    }
    return r;
  }
  if constexpr (sizeof(T) == 2) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < D) w[i] = row[c + i].bits;
    return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < D) w[i] = __float_as_uint(row[c + i]);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Global loads in flight of this wave, those into LDS among them, are done
__device__ __forceinline__ void loads_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// A tile of kRows rows of kD channels (a multiple of 32) in LDS, in slots of 16 bytes: group c of row r lies
// in slot c ^ swap(r) of its row.  So neither 16 lanes that read one group of 16 rows, nor the transposed
// reads of two groups of four rows, meet in a bank.  96 channels take the room of 128.
// kVecRows: rows of aligned 16-byte groups go straight to LDS (a wave's load fills 64 slots in order, each
// lane fetches the group that belongs into its slot; the buffer's range check gives zeros for rows past
// the last and groups past D).  Other rows go through registers.
template <typename T, int kRows, int kD, bool kVecRows>
struct AttnTile {
  static constexpr int kSlots = (kD == 96 ? 128 : kD) * static_cast<int>(sizeof(T)) / 16;
  static constexpr int kStride = kSlots * 16;
  static constexpr int kBytes = kRows * kStride;
  static constexpr int kPer = kRows * kSlots / 256;  // slots per lane of 256
  static_assert(kRows * kSlots % 256 == 0, "whole accesses");

  static __device__ __forceinline__ int swap(int r) {
    if constexpr (kSlots == 4) return r >> 2 & 3;
    if constexpr (kSlots == 8) return sizeof(T) == 2 ? (r >> 1 & 3) * 2 + (r >> 3 & 1) : (r >> 2 & 1) * 4 + (r >> 3 & 1) * 2 + (r >> 1 & 1);
    return sizeof(T) == 2 ? (r & 7) * 2 + (r >> 3 & 1) : (r >> 2 & 3) * 4 + (r & 3);
  }
  // first channel of the group in slot x
  static __device__ __forceinline__ int channel(int x) { return (x % kSlots ^ swap(x / kSlots)) * AttnEl<T>::kVec; }

  // Where this lane's groups lie from the tile's first row on, in bytes
  struct Source {
    uint32_t at[kVecRows ? kPer : 1];
  };
  static __device__ __forceinline__ Source source(long stride, int D) {
    Source s;
    if constexpr (kVecRows) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int x = threadIdx.x + 256 * i, c = channel(x);
        s.at[i] = c < D ? static_cast<uint32_t>((x / kSlots * stride + c) * sizeof(T)) : 0x80000000u;
      }
    }
    return s;
  }
  // rows j0 .. of the n rows at `base` into LDS; done after loads_done() and a barrier
  static __device__ __forceinline__ void load(unsigned char* lds, const Source& s, const T* base, long stride, int j0, int n, int D) {
    static_assert(kVecRows, "16-byte groups");
    const int rows = min(kRows, n - j0);
    const uint32_t bytes = rows > 0 ? static_cast<uint32_t>(((rows - 1) * stride + D) * sizeof(T)) : 0u;
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(base + j0 * stride), 0, static_cast<int>(bytes), 0x00020000);
    unsigned char* const to = lds + uniform(threadIdx.x / 64) * 1024;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)(to + 4096 * i), 16, s.at[i], 0, 0, 0);
  }
  // the same through registers, rows from n on as zeros
  static __device__ __forceinline__ void fetch(const T* base, long stride, int j0, int n, int D, int vec, uint4 (&r)[kPer]) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int x = threadIdx.x + 256 * i, row = j0 + x / kSlots;
      r[i] = make_uint4(0u, 0u, 0u, 0u);
      if (row < n) r[i] = attn_chunk<T>(base + row * stride, channel(x), D, vec);
    }
  }
  static __device__ __forceinline__ void put(unsigned char* lds, const uint4 (&r)[kPer]) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) *reinterpret_cast<uint4*>(lds + (threadIdx.x + 256 * i) * 16) = r[i];
  }
  // rows row0 .. row0 + 15 (row0 a multiple of 16), channels of unit u
  static __device__ __forceinline__ uint4 rows(const unsigned char* lds, int row0, int u, int lane) {
    const int r = lane % 16, c = 4 * u + lane / 16;
    return *reinterpret_cast<const uint4*>(lds + row0 * kStride + r * kStride + (c ^ swap(r)) * 16);
  }
  // transposed: row = channel c0 + lane % 16, along the tokens from row0 on (32 in bf16, 16 in f32)
  static __device__ __forceinline__ uint4 cols(const unsigned char* lds, int row0, int c0, int lane) {
    const int g = lane / 16, j = lane % 16;
    if constexpr (sizeof(T) == 2) {
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s16x4* lds_ptr;
      // lane j of a group of 16 reads 8 bytes of row j / 4; it gets the four rows' values of column j
      const int r = 4 * g + j / 4, c = c0 / 8 + j % 4 / 2;
      const unsigned char* p = lds + row0 * kStride + r * kStride + (c ^ swap(r)) * 16 + j % 2 * 8;
      const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p));
      const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 16 * kStride));
      const uint2 a = __builtin_bit_cast(uint2, x), b = __builtin_bit_cast(uint2, y);
      return make_uint4(a.x, a.y, b.x, b.y);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * g + i, c = c0 / 4 + j / 4;
        w[i] = *reinterpret_cast<const uint32_t*>(lds + row0 * kStride + r * kStride + (c ^ swap(r)) * 16 + j % 4 * 4);
      }
      return make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
};

// Accumulator tiles over tokens as an operand of NP bf16 parts (f32: as they are).  x: the tiles of one
// unit, two of 16 tokens in bf16, one in f32.
template <typename T, int NP>
__device__ __forceinline__ Frag<NP> attn_operand(const f32x4* x) {
  Frag<NP> f;
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4][NP];
    split2<NP>(x[0][0], x[0][1], w[0]);
    split2<NP>(x[0][2], x[0][3], w[1]);
    split2<NP>(x[1][0], x[1][1], w[2]);
    split2<NP>(x[1][2], x[1][3], w[3]);
#pragma unroll
    for (int p = 0; p < NP; ++p) f.p[p] = make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
  } else {
    f.p[0] = __builtin_bit_cast(uint4, x[0]);
  }
  return f;
}

// Maximum and sum over the four groups of 16 lanes (the rows of accumulator tiles), in every lane
__device__ __forceinline__ float group_max(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float group_sum(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// One column (row of the output) of accumulator tiles over channels: D values at element `at` of a dense
// tensor in f32 or bf16; lane group g holds the channels 16 t + 4 g ..
template <int NT>
__device__ __forceinline__ void attn_store_row(void* out, size_t at, const f32x4 (&x)[NT], int D, int g, int bf16, int vec) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int d = 16 * t + 4 * g;
    if (D % 4 == 0 && vec > 0) {
      if (d < D) {
        if (bf16) *reinterpret_cast<uint2*>(static_cast<bf16s*>(out) + at + d) = make_uint2(pack_rne(x[t][0], x[t][1]), pack_rne(x[t][2], x[t][3]));
        else *reinterpret_cast<float4*>(static_cast<float*>(out) + at + d) = make_float4(x[t][0], x[t][1], x[t][2], x[t][3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (d + i < D) {
          if (bf16) st<bf16s>(out, at + d + i, x[t][i]);
          else st<float>(out, at + d + i, x[t][i]);
        }
    }
  }
}

struct AttnSeq {
  long q0, k0;  // first query and key
  int nq, nk;
};

// Offsets out of range or out of order are clamped: no access leaves the tensors whatever they hold.
__device__ __forceinline__ long attn_offset(const int32_t* cu, int i, long rows) {
  const long b = cu[i];
  return b < 0 ? 0 : (b > rows ? rows : b);
}
__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& a, int s) {
  AttnSeq q;
  if (a.cu_q) {
    q.q0 = attn_offset(a.cu_q, s, a.rows_q);
    q.nq = static_cast<int>(max(0L, attn_offset(a.cu_q, s + 1, a.rows_q) - q.q0));
    q.k0 = attn_offset(a.cu_k, s, a.rows_k);
    q.nk = static_cast<int>(max(0L, attn_offset(a.cu_k, s + 1, a.rows_k) - q.k0));
  } else {
    q.q0 = static_cast<long>(s) * a.lq;
    q.k0 = static_cast<long>(s) * a.lk;
    q.nq = a.lq;
    q.nk = a.lk;
  }
  return q;
}

// The tile of `rows` queries (keys) in slot x of a packed call: its sequence, and its number in it (-1: an
// unused slot).
__device__ __forceinline__ int attn_slot(const int32_t* cu, int nseq, long total, int rows, long x, AttnSeq* q, const AttnArgs& a,
                                         bool keys) {
  int lo = 0, hi = nseq - 1;
  while (lo < hi) {  // the last sequence whose slots begin at or before this one
    const int mid = (lo + hi + 1) >> 1;
    if (attn_offset(cu, mid, total) / rows + mid <= x) lo = mid;
    else hi = mid - 1;
  }
  *q = attn_seq(a, lo);
  const long t = x - ((keys ? q->k0 : q->q0) / rows + lo);
  return t < 0 || t * rows >= (keys ? q->nk : q->nq) ? -1 : static_cast<int>(t);
}

struct AttnWork {
  AttnSeq seq;
  int tile, head;  // tile < 0: nothing to do
};

// Workgroup b's tile and head.  The heads of a key head and their tiles share its keys: they are neighbours,
// and go to one XCD (workgroups are dealt round the 8 of them) where the (sequence, key head) pairs come out
// even on those.  Later tiles, which see more keys without a window, come first.
// heads: workgroups per key head and tile (h / hk, or 1).
__device__ __forceinline__ AttnWork attn_work(const AttnArgs& a, unsigned b, int rows, bool keys, int heads) {
  AttnWork w;
  const int n = keys ? a.lk : a.lq;
  const long slots = a.cu_q ? n / rows + a.nseq : (n + rows - 1) / rows;  // of a pair
  const unsigned pairs = a.cu_q ? a.hk : static_cast<unsigned>(a.nseq) * a.hk;
  const unsigned per = static_cast<unsigned>(slots) * heads;
  unsigned pair, r;
  if (pairs % 8 == 0) {
    pair = (b & 7u) + 8 * ((b >> 3) / per);
    r = (b >> 3) % per;
  } else {
    pair = b / per;
    r = b % per;
  }
  const unsigned kh = pair % a.hk;
  const long x = slots - 1 - r / heads;
  w.head = static_cast<int>(kh * heads + r % heads);
  if (a.cu_q) {
    w.tile = attn_slot(keys ? a.cu_k : a.cu_q, a.nseq, keys ? a.rows_k : a.rows_q, rows, x, &w.seq, a, keys);
  } else {
    w.seq = attn_seq(a, pair / a.hk);
    w.tile = static_cast<int>(x);
  }
  return w;
}

}  // namespace ssm
