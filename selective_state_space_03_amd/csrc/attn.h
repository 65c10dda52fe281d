// Internal interface of the window attention's and its cache's kernels
// (attn_*.hip) and their host side (attn_api.cpp).
//
// The query at position p of a sequence sees the keys
//   j <= p  with  j > p - window  or  j < sinks,
// P_pj = e^{scale q_p.k_j - lse_p} over them, o_p = sum_j P_pj v_j.
#pragma once
#include "ssm_internal.h"

namespace ssm {

constexpr int kAttnMaxD = 128;        // channels of a head that the kernels hold
constexpr int kAttnAll = 1 << 30;     // a window that no sequence reaches; the longest sequence

struct AttnArgs {
  const void *q, *k, *v;              // rows of a token: (h, D), (hk, D), (hk, D); strides in elements
  long q_stride, k_stride, v_stride;
  const int32_t *cu_q, *cu_k;         // (nseq + 1) offsets, or null: nseq sequences of lq queries and lk keys
  int nseq, lq, lk, h, hk, D;
  long rows_q, rows_k;                // all queries, all keys
  int window, sinks;                  // window: 1 .. kAttnAll
  float scale;
  int vec;                            // rows of 16-byte groups (2), of 8-byte groups (1), of any elements (0)
  void* o;                            // (rows_q, h, D)
  void* o_rest;                       // bf16: what rounding took from an o in bf16, or null
  float* lse;                         // (rows_q, h) or null
  int nsplit;                         // parts of the visible keys (forward of few queries), 1: whole
  float* part;                        // (rows_q, h, nsplit, attn_dq(D)) sums, then (rows_q, h, nsplit) of (maximum, sum)
  // backward
  const void* dout;
  void *dq, *dk, *dv;                 // dense, or null
  int grad_bf16;
  float* delta;                       // (rows_q, h): sum_d do o
  int sink_tiles, span;               // tiles of 64 keys with sinks whose queries are cut into pieces of span
  float *dk_part, *dv_part;           // (pieces, hk, sink_tiles, 64, D): their partial sums
};

struct AttnLaunch {
  AttnArgs a;
  int in_dtype, o_dtype, grad_dtype;
};

inline int attn_dq(int D) { return (D + 31) / 32 * 32; }
// Query tiles over all sequences (packed: sequence i owns the tiles from cu[i] / rows + i on)
inline long attn_tiles(const AttnArgs& a, int rows, bool keys) {
  const long n = keys ? a.lk : a.lq;
  return a.cu_q ? n / rows + a.nseq : static_cast<long>(a.nseq) * ((n + rows - 1) / rows);
}
// Pieces of queries over all sequences
inline long attn_pieces(const AttnArgs& a) {
  return a.cu_q ? a.lq / a.span + a.nseq : static_cast<long>(a.nseq) * ((a.lq + a.span - 1) / a.span);
}
// Parts of the keys of a forward in bf16 whose workgroups of 128 queries leave half of the CUs idle: as many as fill
// them, of 512 keys or more (8 heads of 128 and 8192 keys: one query 123 -> 25 us, 128 queries 29)
inline int attn_fwd_splits(const AttnArgs& a) {
  const long blocks = attn_tiles(a, 128, false) * a.h;
  const long seen = a.window == kAttnAll ? a.lk : (a.lk < a.window + 128L + a.sinks ? a.lk : a.window + 128L + a.sinks);
  if (a.cu_q || blocks == 0 || blocks > 128 || seen < 2048 || a.window < 1024) return 1;
  const long fill = 256 / blocks, most = seen / 512;
  return static_cast<int>(fill < most ? fill : most);
}
constexpr int kSinkRows = 64;  // keys of a tile of the backward pass
// Workgroups of its queries, each two heads of `rows` queries or one of twice as many
inline long attn_query_blocks(const AttnArgs& a, int rows) {
  return a.h / a.hk % 2 == 0 ? attn_tiles(a, rows, false) * a.h / 2 : attn_tiles(a, 2 * rows, false) * a.h;
}
hipError_t launch_attn_fwd(const AttnLaunch& l, hipStream_t s);
hipError_t launch_attn_bwd(const AttnLaunch& l, hipStream_t s);
hipError_t launch_attn_sinks(const AttnArgs& a, hipStream_t s);

// ---- the paged cache
struct AttnCacheArgs {
  const void *k, *v;                  // tokens (hk, D); strides in elements
  long k_stride, v_stride;
  const int32_t *cu, *lens, *table;   // cu or null: nseq sequences of seqlen tokens
  int nseq, seqlen, hk, D, table_rows, pages, page;
  long tokens;
  void *k_cache, *v_cache;            // (pages, hk, page, D)
  float *k_scale, *v_scale;           // (pages, hk), 8 bits only
  int vec;                            // rows of groups of 8 elements, aligned
};
// Pages met over all sequences: sequence i owns the slots from cu[i] / page + 2 i on
inline long attn_cache_slots(const AttnCacheArgs& a) {
  if (a.cu) return a.tokens / a.page + 2L * a.nseq;
  return a.seqlen == 0 ? 0 : static_cast<long>(a.nseq) * ((a.seqlen - 1L + a.page - 1) / a.page + 1);
}
hipError_t launch_attn_cache(const AttnCacheArgs& a, int in_dtype, int cache_dtype, hipStream_t s);

struct AttnStepArgs {
  const void* q;                      // (batch, h, D)
  long q_stride;
  const void *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int32_t *table, *lens;
  int batch, h, hk, D, table_rows, pages, page;
  int window, sinks;
  float scale;
  int q_vec, vec;                     // rows of q and of the cache: 16-byte groups (2), 8-byte groups (1), any (0)
  int page_shift;                     // log2(page), or -1
  int nsplit, chunk;                  // parts of a sequence's visible keys, keys in one
  void* o;                            // (batch, h, D)
  float* part;                        // (batch, h, nsplit, attn_dq(D)): the parts' sums of P v
  float* part_stat;                   // (batch, h, nsplit, 2): maximum and sum of their softmax
};
struct AttnStepLaunch {
  AttnStepArgs a;
  int in_dtype, cache_dtype, o_dtype;
};
constexpr int kAttnE4M3 = 2;          // SSM_E4M3
constexpr int kAttnStepHeads = 16;    // query heads of a key head that share a workgroup
inline int attn_head_tiles(int h, int hk) { return (h / hk + kAttnStepHeads - 1) / kAttnStepHeads; }
hipError_t launch_attn_step(const AttnStepLaunch& l, hipStream_t s);

}  // namespace ssm
