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

// .. all but the last kLeft of them
template <int kLeft>
__device__ __forceinline__ void loads_left() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLeft) : "memory"); }

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint32_t lds_address(const unsigned char* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) unsigned char*)p));
}
// 16 bytes a lane from its offset in the buffer to `to` and on.  As an instruction of its own: behind the
// builtin the compiler waits for all such loads ahead of the next read of LDS, whatever that reads, so that
// none would be in flight during the products (prompt 221 us).  It counts outstanding loads from its own
// alone, and with others among them waits for more than it means to, not less.  The wait states are for
// M0, and for a descriptor that has just come back from a vector register.
__device__ __forceinline__ void load_to_lds(u32x4 rsrc, uint32_t offset, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(offset), "s"(rsrc)
               : "memory", "m0");
}

// A tile of kRows rows of kD channels (a multiple of 32) in LDS, in slots of 16 bytes: group c of row r lies
// in slot c ^ swap(r) of its row.  So neither 16 lanes that read one group of 16 rows, nor the transposed
// reads of two groups of four rows, meet in a bank.  96 channels take the room of 128.
// kVecRows: rows of aligned 16-byte groups go straight to LDS (a wave's load fills 64 slots in order, each
// lane fetches the group that belongs into its slot; the buffer's range check gives zeros for rows past
// the last and groups past D).  Other rows go through registers.
template <typename T, int kRows, int kD, bool kVecRows, int kThreads = 256>
struct AttnTile {
  static constexpr int kSlots = (kD == 96 ? 128 : kD) * static_cast<int>(sizeof(T)) / 16;
  static constexpr int kStride = kSlots * 16;
  static constexpr int kBytes = kRows * kStride;
  static constexpr int kAll = kRows * kSlots;
  static constexpr int kUse = kAll < kThreads ? kAll : kThreads;  // threads that load
  static constexpr int kPer = kAll / kUse;                        // slots of one of them
  static_assert(kAll % kUse == 0 && kUse % 64 == 0, "whole accesses");

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
    Source s{};
    if constexpr (kVecRows) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int x = threadIdx.x % kThreads + kUse * i, c = channel(x);
        s.at[i] = c < D ? static_cast<uint32_t>((x / kSlots * stride + c) * sizeof(T)) : 0x80000000u;
      }
    }
    return s;
  }
  // rows j0 .. of the n rows at `base` into LDS (at an address from lds_address); done after loads_done() and
  // a barrier
  static __device__ __forceinline__ void load(uint32_t lds, const Source& s, const T* base, long stride, int j0, int n, int D) {
    static_assert(kVecRows, "16-byte groups");
    const int wave = uniform(threadIdx.x % kThreads / 64);
    if (kUse < kThreads && wave >= kUse / 64) return;
    const int rows = min(kRows, n - j0);
    const uint32_t bytes = rows > 0 ? static_cast<uint32_t>(((rows - 1) * static_cast<int>(stride) + D) * static_cast<int>(sizeof(T))) : 0u;
    const uint64_t from = reinterpret_cast<uint64_t>(base + j0 * stride);
    const u32x4 rsrc = {static_cast<uint32_t>(from), static_cast<uint32_t>(from >> 32) & 0xffffu, bytes, 0x00020000u};
    const uint32_t to = lds + static_cast<uint32_t>(wave) * 1024u;
#pragma unroll
    for (int i = 0; i < kPer; ++i) load_to_lds(rsrc, s.at[i], to + 16u * kUse * i);
  }
  // the same through registers, rows from n on as zeros
  static __device__ __forceinline__ void fetch(const T* base, long stride, int j0, int n, int D, int vec, uint4 (&r)[kPer]) {
    if (kUse < kThreads && threadIdx.x % kThreads >= kUse) return;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int x = threadIdx.x % kThreads + kUse * i, row = j0 + x / kSlots;
      r[i] = make_uint4(0u, 0u, 0u, 0u);
      if (row < n) r[i] = attn_chunk<T>(base + row * stride, channel(x), D, vec);
    }
  }
  static __device__ __forceinline__ void put(unsigned char* lds, const uint4 (&r)[kPer]) {
    if (kUse < kThreads && threadIdx.x % kThreads >= kUse) return;
#pragma unroll
    for (int i = 0; i < kPer; ++i) *reinterpret_cast<uint4*>(lds + (threadIdx.x % kThreads + kUse * i) * 16) = r[i];
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

// 32 x 32 tiles of bf16 (a unit is 16 deep; h = lane / 32): operands hold rows or columns lane % 32 and the
// depths 8 h + i; an accumulator has column = lane % 32, row = 8 (i / 4) + 4 h + i % 4, so that its values
// 8 s .. 8 s + 7 are an operand of unit s over the tokens 16 s + 8 (i / 4) + 4 h + i % 4.  A vector
// instruction of another wave goes beside a 32 x 32 x 16 product without loss (32 FMA beside 8 products
// 131 ns, the products alone 130), beside 16 x 16 x 32 only in part (106 ns for 64 and 63).
typedef float f32x16 __attribute__((ext_vector_type(16)));
__device__ __forceinline__ f32x16 mma32(uint4 a, uint4 b, f32x16 acc) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
}
template <typename Tile>  // of bf16
struct Wide {
  // Addresses in LDS: of this lane's part of the first unit, which the others differ from in bits of their own
  static __device__ __forceinline__ uint32_t rows_at(const unsigned char* lds, int lane) {
    const int r = lane % 32;
    return lds_address(lds) + r * Tile::kStride + (lane / 32 ^ Tile::swap(r)) * 16;
  }
  static __device__ __forceinline__ uint32_t cols_at(const unsigned char* lds, int lane) {
    const int j = lane % 16, r = 4 * (lane / 32) + j / 4, c = 2 * (lane / 16 % 2) + j % 4 / 2;
    return lds_address(lds) + r * Tile::kStride + (c ^ Tile::swap(r)) * 16 + j % 2 * 8;
  }
  // rows row0 .. row0 + 31, channels 16 u ..
  static __device__ __forceinline__ uint4 rows(uint32_t at, int row0, int u) {
    typedef const __attribute__((address_space(3))) u32x4* lds_ptr;
    const u32x4 v = *(lds_ptr)((at ^ (u << 5)) + row0 * Tile::kStride);
    return make_uint4(v.x, v.y, v.z, v.w);
  }
  // transposed: row = channel 32 d + lane % 32, along the tokens of the unit from row0 (a multiple of 16) on
  static __device__ __forceinline__ uint4 cols(uint32_t at, int row0, int d) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4* lds_ptr;
    constexpr uint32_t kEight = Tile::kSlots == 4 ? 32 : 16;  // what eight rows on change in the slot
    const uint32_t p = at ^ (d << 6);
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + row0 * Tile::kStride));
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)((p ^ kEight) + (row0 + 8) * Tile::kStride));
    const uint2 a = __builtin_bit_cast(uint2, x), b = __builtin_bit_cast(uint2, y);
    return make_uint4(a.x, a.y, b.x, b.y);
  }
};
// values 8 s .. of an accumulator over tokens as an operand of NP bf16 parts
template <int NP>
__device__ __forceinline__ Frag<NP> wide_operand(const f32x16& x, int s) {
  Frag<NP> f;
  uint32_t w[4][NP];
#pragma unroll
  for (int i = 0; i < 4; ++i) split2<NP>(x[8 * s + 2 * i], x[8 * s + 2 * i + 1], w[i]);
#pragma unroll
  for (int p = 0; p < NP; ++p) f.p[p] = make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
  return f;
}
// Of a lane in half h with the query at pos, and a tile of keys from j0 on: key j0 + 4 h + j is seen if j <= d
// and (j > w or j < f).
struct WideMask {
  int d, w, f;
};
__host__ __device__ constexpr WideMask wide_mask(int pos, int j0, int h, int window, int sinks) {
  return {pos - j0 - 4 * h, pos - j0 - 4 * h - window, sinks - j0 - 4 * h};
}
// A key that none of the 32 queries from position p0 on sees: where a tile that is not there lies
__host__ __device__ constexpr int wide_none(int p0) { return p0 + 32; }
// Scores of a tile from key j0 on, of queries from position p0 on (32 of them, the lane's at pos), of keys that
// are not seen.  Tiles in which every query sees every key pass by; others mostly meet one border.
template <int KT>
__device__ __forceinline__ void wide_hide(f32x16 (&s)[KT], int j0, int p0, int pos, int h, int window, int sinks) {
  const auto [d, w, f] = wide_mask(pos, j0, h, window, sinks);
  if (j0 + 32 * KT - 1 > p0) {
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[k][e] = 32 * k + 8 * (e / 4) + e % 4 <= d ? s[k][e] : -INFINITY;
  }
  if (j0 > p0 + 31 - window || j0 + 32 * KT <= sinks) return;
  if (j0 >= sinks) {
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[k][e] = 32 * k + 8 * (e / 4) + e % 4 > w ? s[k][e] : -INFINITY;
  } else {
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int j = 32 * k + 8 * (e / 4) + e % 4;
        s[k][e] = j > w || j < f ? s[k][e] : -INFINITY;
      }
  }
}
__device__ __forceinline__ float half_max(float x) {  // over the two halves of the wave
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

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

// Four channels from d on of a row of D at element `at` of a dense tensor in f32 or bf16
__device__ __forceinline__ void attn_store4(void* out, size_t at, float x0, float x1, float x2, float x3, int d, int D, int bf16, int vec) {
  if (D % 4 == 0 && vec > 0) {
    if (d < D) {
      if (bf16) *reinterpret_cast<uint2*>(static_cast<bf16s*>(out) + at + d) = make_uint2(pack_rne(x0, x1), pack_rne(x2, x3));
      else *reinterpret_cast<float4*>(static_cast<float*>(out) + at + d) = make_float4(x0, x1, x2, x3);
    }
  } else {
    const float x[4] = {x0, x1, x2, x3};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (d + i < D) {
        if (bf16) st<bf16s>(out, at + d + i, x[i]);
        else st<float>(out, at + d + i, x[i]);
      }
  }
}
// One column (row of the output) of accumulator tiles over channels: lane group g holds 16 t + 4 g ..
template <int NT>
__device__ __forceinline__ void attn_store_row(void* out, size_t at, const f32x4 (&x)[NT], int D, int g, int bf16, int vec) {
#pragma unroll
  for (int t = 0; t < NT; ++t) attn_store4(out, at, x[t][0], x[t][1], x[t][2], x[t][3], 16 * t + 4 * g, D, bf16, vec);
}
// What rounding to bf16 takes from x
__device__ __forceinline__ float rest_of(float x) { return x - __uint_as_float(pack_rne(x, 0.0f) << 16); }

// .. of 32 x 32 tiles: half h of the wave holds 32 t + 8 i + 4 h ..
template <int NT>
__device__ __forceinline__ void wide_store_row(void* out, size_t at, const f32x16 (&x)[NT], int D, int h, int bf16, int vec) {
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      attn_store4(out, at, x[t][4 * i], x[t][4 * i + 1], x[t][4 * i + 2], x[t][4 * i + 3], 32 * t + 8 * i + 4 * h, D, bf16, vec);
}

template <int NT>
__device__ __forceinline__ void wide_store_o(const AttnArgs& a, size_t at, f32x16 (&o)[NT], int h, int bf16) {
  wide_store_row<NT>(a.o, at, o, a.D, h, bf16, a.vec);
  if (!a.o_rest) return;
#pragma unroll
  for (int d = 0; d < NT; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = rest_of(o[d][e]);
  wide_store_row<NT>(a.o_rest, at, o, a.D, h, 1, a.vec);
}

// Factor of the scores in powers of two.  Not zero: a score of -infinity (a key that is not seen) has to stay that.
__device__ __forceinline__ float attn_log2_scale(float scale) { return fmaxf(scale * kLog2e, 1e-30f); }

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

// The keys that some query at the positions p .. last sees, as tiles of BN: the sinks, then those from the window's
// begin on.  A tile ends where its range does and the rows behind are zeros: a row that none of these queries sees is
// not in any product, where a NaN would not vanish beside P = 0.
template <int BN>
struct AttnKeys {
  int sinks, end;    // sinks ahead of the window, past the last key
  int ns, n, shift;  // tiles of sinks, of all; from where tiles of the window would lie to where they do
  __device__ __forceinline__ AttnKeys(const AttnArgs& a, int p, int last) {
    const int lo = max(0, p - a.window + 1);
    const bool apart = lo > a.sinks;
    sinks = apart ? a.sinks : 0;
    end = last + 1;
    ns = (sinks + BN - 1) / BN;
    shift = (apart ? lo : 0) - ns * BN;
    n = last < 0 ? 0 : (end - shift + BN - 1) / BN;
  }
  __device__ __forceinline__ int key(int t) const { return t * BN + (t < ns ? 0 : shift); }  // first of tile t
  __device__ __forceinline__ int upto(int t) const { return t < ns ? sinks : end; }           // its rows end
  __device__ __forceinline__ int window(int t, int w) const { return t < ns ? 0 : w; }        // of its mask
};

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
// even on those.  The longest come first: later queries, earlier keys (tile by tile over the pairs).
// heads: workgroups per key head and tile (h / hk, or 1).
__device__ __forceinline__ AttnWork attn_work(const AttnArgs& a, unsigned b, int rows, bool keys, int heads) {
  AttnWork w;
  const int n = keys ? a.lk : a.lq;
  const long slots = a.cu_q ? n / rows + a.nseq : (n + rows - 1) / rows;  // of a pair
  const unsigned pairs = a.cu_q ? a.hk : static_cast<unsigned>(a.nseq) * a.hk;
  const unsigned per = static_cast<unsigned>(slots) * heads;
  unsigned pair, r;
  if (keys && pairs % 8 == 0) {
    pair = (b & 7u) + 8 * ((b >> 3) % (pairs / 8));
    r = (b >> 3) / (pairs / 8);
  } else if (keys) {
    pair = b % pairs;
    r = b / pairs;
  } else if (pairs % 8 == 0) {
    pair = (b & 7u) + 8 * ((b >> 3) / per);
    r = (b >> 3) % per;
  } else {
    pair = b / per;
    r = b % per;
  }
  const unsigned kh = pair % a.hk;
  const long x = keys ? r : slots - 1 - r / heads;
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
