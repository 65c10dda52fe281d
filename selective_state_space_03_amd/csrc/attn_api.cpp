// Host side of the window attention's entry points and of its paged cache's
// (include/ssm_mi355x.h): argument validation without a GPU, workspace layout,
// launches on the caller's stream.
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "../../include/ssm_mi355x.h"
#include "attn.h"

namespace {

ssm_status_t fail(ssm_status_t s, const char* what) { return static_cast<ssm_status_t>(ssm::set_error(s, what)); }
ssm_status_t ok() { return static_cast<ssm_status_t>(ssm::set_error(SSM_OK, "")); }
ssm_status_t done(ssm_status_t s) { return s == SSM_OK ? ok() : s; }
ssm_status_t hip_status(hipError_t e) {
  return e == hipSuccess ? ok() : fail(SSM_ERR_HIP, hipGetErrorString(e));
}

bool valid_dtype(int32_t d) { return d == SSM_F32 || d == SSM_BF16; }
size_t esize(int32_t d) { return d == SSM_E4M3 ? 1 : d == SSM_BF16 ? 2 : 4; }
size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
bool aligned(std::initializer_list<const void*> ps, uintptr_t to) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & (to - 1)) return false;
  return true;
}

struct Range {
  const void* p;
  size_t bytes;
};
bool overlaps(Range a, Range b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
  const auto a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}
ssm_status_t check_overlap(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  for (const Range& o : outs) {
    for (const Range& i : ins)
      if (overlaps(o, i)) return fail(SSM_ERR_INVALID_ARG, "an output overlaps an input");
    for (const Range& p : outs)
      if (&p != &o && overlaps(o, p)) return fail(SSM_ERR_INVALID_ARG, "two outputs overlap");
  }
  return SSM_OK;
}

// A row stride of tokens of `width` elements: 0 (dense), or at least a row, and no offset past 2^58.
ssm_status_t stride_check(int64_t stride, int64_t width, int64_t rows) {
  if (stride && (stride < width || stride > (static_cast<int64_t>(1) << 40)))
    return fail(SSM_ERR_INVALID_ARG, "q_stride, k_stride or v_stride is shorter than a token's row (or beyond 2^40)");
  if (rows > 0 && stride > (static_cast<int64_t>(1) << 58) / rows)
    return fail(SSM_ERR_INVALID_ARG, "q_stride, k_stride or v_stride times the tokens is beyond 2^58");
  return SSM_OK;
}
Range rows_of(const void* p, int64_t stride, int64_t width, int64_t rows, int32_t dtype) {
  const int64_t st = stride ? stride : width;
  return {p, rows > 0 ? static_cast<size_t>((rows - 1) * st + width) * esize(dtype) : 0};
}

ssm_status_t heads_check(int32_t hk, int32_t h, int32_t d) {
  if (hk <= 0 || h <= 0 || d <= 0) return fail(SSM_ERR_INVALID_ARG, "nkheads, nheads and d_head must be positive");
  if (h % hk != 0) return fail(SSM_ERR_INVALID_ARG, "nheads must be a multiple of nkheads");
  if (d > ssm::kAttnMaxD) return fail(SSM_ERR_UNSUPPORTED, "d_head must be at most 128");
  if (h > 65536) return fail(SSM_ERR_UNSUPPORTED, "nheads must be at most 65536");
  return SSM_OK;
}

template <typename P>
ssm_status_t mask_check(const P* p) {
  if (!(p->scale >= 0.0f && p->scale < INFINITY)) return fail(SSM_ERR_INVALID_ARG, "scale must be finite and not negative");
  if (p->window < 0 || p->sinks < 0) return fail(SSM_ERR_INVALID_ARG, "window or sinks is negative");
  return SSM_OK;
}

// 16-byte groups in every row (2), 8-byte groups (1), any elements (0)
int vec_of(int32_t d, int32_t dtype, std::initializer_list<int64_t> strides, std::initializer_list<const void*> ps) {
  for (int v = 2; v > 0; --v) {
    const int64_t b = v == 2 ? 16 : 8, e = static_cast<int64_t>(esize(dtype));
    bool fits = d * e % b == 0 && aligned(ps, 16);
    // (a tile's rows are addressed in 31 bits)
    for (int64_t s : strides) fits = fits && s * e % b == 0 && (v == 1 || s <= 1 << 22);
    if (fits) return v;
  }
  return 0;
}

// ---------------------------------------------------------------- whole sequences

template <typename P>
int64_t rows_q(const P* p) { return static_cast<int64_t>(p->batch) * p->seqlen; }
template <typename P>
int64_t rows_k(const P* p) { return static_cast<int64_t>(p->batch) * p->seqlen_k; }

template <typename P>
void attn_plan(const P* p, ssm::AttnLaunch& l) {
  ssm::AttnArgs& a = l.a;
  const int64_t qw = static_cast<int64_t>(p->nheads) * p->d_head, kw = static_cast<int64_t>(p->nkheads) * p->d_head;
  a.q = p->q;
  a.k = p->k;
  a.v = p->v;
  a.q_stride = p->q_stride ? p->q_stride : qw;
  a.k_stride = p->k_stride ? p->k_stride : kw;
  a.v_stride = p->v_stride ? p->v_stride : kw;
  a.cu_q = p->cu_seqlens;
  a.cu_k = p->cu_seqlens_k ? p->cu_seqlens_k : p->cu_seqlens;
  a.nseq = p->num_seqs;
  a.lq = p->seqlen;
  a.lk = p->seqlen_k;
  a.h = p->nheads;
  a.hk = p->nkheads;
  a.D = p->d_head;
  a.rows_q = rows_q(p);
  a.rows_k = rows_k(p);
  // a window that reaches over every sequence is none, and sinks only matter behind a window
  a.window = p->window == 0 || p->window >= p->seqlen_k ? ssm::kAttnAll : p->window;
  a.sinks = a.window == ssm::kAttnAll ? 0 : std::min(p->sinks, p->seqlen_k);
  a.scale = p->scale;
  l.in_dtype = p->x_dtype;
}

// Sizes that the workspace and the grids go by are usable.
template <typename P>
bool attn_fields(const P* p) {
  if (!(p->batch >= 0 && p->seqlen >= 0 && p->seqlen_k >= 0 && p->num_seqs >= 0 && p->nkheads > 0 && p->nheads > 0 &&
        p->nheads <= 65536 && p->nheads % p->nkheads == 0 && p->d_head > 0 && p->d_head <= ssm::kAttnMaxD &&
        p->seqlen <= ssm::kAttnAll && p->seqlen_k <= ssm::kAttnAll && p->window >= 0 && p->sinks >= 0))
    return false;
  ssm::AttnLaunch l{};
  attn_plan(p, l);
  const long most = (1L << 24) - 1;
  return ssm::attn_tiles(l.a, 64, false) <= most / p->nheads && ssm::attn_tiles(l.a, 64, true) <= most / p->nkheads;
}

template <typename P>
ssm_status_t attn_common(const P* p) {
  if (p->batch < 0 || p->seqlen < 0 || p->seqlen_k < 0 || p->num_seqs < 0)
    return fail(SSM_ERR_INVALID_ARG, "batch, seqlen, seqlen_k or num_seqs is negative");
  ssm_status_t s = heads_check(p->nkheads, p->nheads, p->d_head);
  if (s == SSM_OK) s = mask_check(p);
  if (s != SSM_OK) return s;
  if (!valid_dtype(p->x_dtype)) return fail(SSM_ERR_INVALID_ARG, "x_dtype: unknown dtype");
  if (p->seqlen > ssm::kAttnAll || p->seqlen_k > ssm::kAttnAll)
    return fail(SSM_ERR_UNSUPPORTED, "seqlen and seqlen_k must be at most 2^30");
  if (p->cu_seqlens ? p->batch != 1 : p->num_seqs != p->batch)
    return fail(SSM_ERR_INVALID_ARG, "packed sequences need batch 1; without cu_seqlens num_seqs must equal batch");
  if (p->cu_seqlens_k && !p->cu_seqlens) return fail(SSM_ERR_INVALID_ARG, "cu_seqlens_k without cu_seqlens");
  if (p->cu_seqlens && !p->cu_seqlens_k && p->seqlen != p->seqlen_k)
    return fail(SSM_ERR_INVALID_ARG, "without cu_seqlens_k seqlen_k must equal seqlen");
  if (!aligned({p->cu_seqlens, p->cu_seqlens_k, p->lse}, 4))
    return fail(SSM_ERR_INVALID_ARG, "cu_seqlens, cu_seqlens_k or lse is not 4-byte aligned");
  const int64_t qw = static_cast<int64_t>(p->nheads) * p->d_head, kw = static_cast<int64_t>(p->nkheads) * p->d_head;
  s = stride_check(p->q_stride, qw, rows_q(p));
  if (s == SSM_OK) s = stride_check(p->k_stride, kw, rows_k(p));
  if (s == SSM_OK) s = stride_check(p->v_stride, kw, rows_k(p));
  if (s != SSM_OK) return s;
  if ((rows_q(p) > 0 && !p->q) || (rows_k(p) > 0 && (!p->k || !p->v))) return fail(SSM_ERR_INVALID_ARG, "q, k or v is NULL");
  if (!aligned({p->q, p->k, p->v}, esize(p->x_dtype))) return fail(SSM_ERR_INVALID_ARG, "q, k or v is not aligned to its element size");
  if (!valid_dtype(p->o_dtype)) return fail(SSM_ERR_INVALID_ARG, "o_dtype: unknown dtype");
  if (rows_q(p) > 0 && !p->o) return fail(SSM_ERR_INVALID_ARG, "o is NULL");
  if (!aligned({p->o}, esize(p->o_dtype))) return fail(SSM_ERR_INVALID_ARG, "o is not aligned to its element size");
  if (p->o_rest && p->o_dtype != SSM_BF16) return fail(SSM_ERR_INVALID_ARG, "o_rest goes with an o in bf16");
  if (!aligned({p->o_rest}, 2)) return fail(SSM_ERR_INVALID_ARG, "o_rest is not aligned to its element size");
  if (!attn_fields(p)) return fail(SSM_ERR_UNSUPPORTED, "too many tiles and heads for one launch");
  return SSM_OK;
}

template <typename P>
Range q_range(const P* p) {
  return rows_of(p->q, p->q_stride, static_cast<int64_t>(p->nheads) * p->d_head, rows_q(p), p->x_dtype);
}
template <typename P>
Range k_range(const P* p, const void* ptr, int64_t stride) {
  return rows_of(ptr, stride, static_cast<int64_t>(p->nkheads) * p->d_head, rows_k(p), p->x_dtype);
}
template <typename P>
size_t q_elems(const P* p) { return static_cast<size_t>(rows_q(p)) * p->nheads * p->d_head; }
template <typename P>
size_t k_elems(const P* p) { return static_cast<size_t>(rows_k(p)) * p->nkheads * p->d_head; }
template <typename P>
size_t cu_bytes(const P* p) { return (static_cast<size_t>(p->num_seqs) + 1) * 4; }

// The workspace holds the parts of a call whose keys are split, which goes by sizes and types, not by alignment.
int fwd_splits(const ssm_attn_params_t* p) {
  if (p->x_dtype != SSM_BF16 || p->o_dtype != SSM_BF16) return 1;
  ssm::AttnLaunch l{};
  attn_plan(p, l);
  return ssm::attn_fwd_splits(l.a);
}
size_t fwd_ws(const ssm_attn_params_t* p) {
  const int n = fwd_splits(p);
  return n > 1 ? static_cast<size_t>(rows_q(p)) * p->nheads * n * (ssm::attn_dq(p->d_head) + 2) * 4 : 0;
}

ssm_status_t attn_check(const ssm_attn_params_t* p) {
  if (!p) return fail(SSM_ERR_INVALID_ARG, "params is NULL");
  if (p->struct_size != sizeof(*p)) return fail(SSM_ERR_INVALID_ARG, "struct_size does not match this library");
  const ssm_status_t s = attn_common(p);
  if (s != SSM_OK) return s;
  const size_t need = fwd_ws(p);
  if (need > 0 && (!p->workspace || p->workspace_bytes < need)) return fail(SSM_ERR_WORKSPACE, "workspace is missing or too small");
  if (need > 0 && !aligned({p->workspace}, 256)) return fail(SSM_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return check_overlap({{p->o, q_elems(p) * esize(p->o_dtype)}, {p->lse, static_cast<size_t>(rows_q(p)) * p->nheads * 4}, {p->o_rest, q_elems(p) * 2},
                        {p->workspace, need}},
                       {q_range(p), k_range(p, p->k, p->k_stride), k_range(p, p->v, p->v_stride), {p->cu_seqlens, cu_bytes(p)},
                        {p->cu_seqlens_k, cu_bytes(p)}});
}

// ---------------------------------------------------------------- backward

// The tiles of keys that hold sinks are seen by all later queries: where they are few, these are cut into
// pieces, each about the queries that a window shows to another tile.
template <typename P>
void sink_plan(const P* p, ssm::AttnArgs& a) {
  a.sink_tiles = 0;
  a.span = 64;
  const int tiles = (a.sinks + 63) / 64;
  if (tiles == 0 || tiles > 4) return;
  const int64_t span = std::max<int64_t>((static_cast<int64_t>(a.window) + 64 + 63) / 64 * 64, 128);
  if (span >= a.lq) return;
  a.sink_tiles = tiles;
  a.span = static_cast<int>(span);
}

struct BwdWs {
  size_t delta, dk_part, dv_part, total;
};
template <typename P>
BwdWs bwd_ws(const P* p) {
  ssm::AttnLaunch l{};
  attn_plan(p, l);
  sink_plan(p, l.a);
  BwdWs w{};
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t o = at;
    at = align256(at + bytes);
    return o;
  };
  w.delta = take(static_cast<size_t>(rows_q(p)) * p->nheads * 4);
  if (l.a.sink_tiles > 0) {
    const size_t part = static_cast<size_t>(ssm::attn_pieces(l.a)) * p->nkheads * l.a.sink_tiles * 64 * p->d_head * 4;
    w.dk_part = take(part);
    w.dv_part = take(part);
  }
  w.total = at;
  return w;
}
// Workgroups of keys, pieces and queries stand in one launch, of 512 threads each.
bool bwd_fields(const ssm_attn_bwd_params_t* p) {
  if (!attn_fields(p)) return false;
  ssm::AttnLaunch l{};
  attn_plan(p, l);
  sink_plan(p, l.a);
  const long most = (1L << 23) - 1, sinks = l.a.sink_tiles > 0 ? std::max<long>(ssm::attn_pieces(l.a), l.a.nseq) * l.a.sink_tiles : 0;
  return sinks + ssm::attn_tiles(l.a, ssm::kSinkRows, true) <= (most - ssm::attn_query_blocks(l.a, 64)) / p->nkheads;
}

ssm_status_t attn_bwd_check(const ssm_attn_bwd_params_t* p) {
  if (!p) return fail(SSM_ERR_INVALID_ARG, "params is NULL");
  if (p->struct_size != sizeof(*p)) return fail(SSM_ERR_INVALID_ARG, "struct_size does not match this library");
  const ssm_status_t s = attn_common(p);
  if (s != SSM_OK) return s;
  if (!bwd_fields(p)) return fail(SSM_ERR_UNSUPPORTED, "too many tiles and heads for one launch");
  if (!valid_dtype(p->grad_dtype)) return fail(SSM_ERR_INVALID_ARG, "grad_dtype: unknown dtype");
  if (rows_q(p) > 0 && (!p->lse || !p->dout)) return fail(SSM_ERR_INVALID_ARG, "lse or dout is NULL");
  if (!aligned({p->dout}, esize(p->x_dtype)) || !aligned({p->dq, p->dk, p->dv}, esize(p->grad_dtype)))
    return fail(SSM_ERR_INVALID_ARG, "dout or a gradient is not aligned to its element size");
  const size_t need = bwd_ws(p).total;
  if (need > 0 && (!p->workspace || p->workspace_bytes < need)) return fail(SSM_ERR_WORKSPACE, "workspace is missing or too small");
  if (!aligned({p->workspace}, 256)) return fail(SSM_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  const size_t eg = esize(p->grad_dtype);
  return check_overlap({{p->dq, q_elems(p) * eg}, {p->dk, k_elems(p) * eg}, {p->dv, k_elems(p) * eg}, {p->workspace, need}},
                       {q_range(p), k_range(p, p->k, p->k_stride), k_range(p, p->v, p->v_stride), {p->cu_seqlens, cu_bytes(p)},
                        {p->cu_seqlens_k, cu_bytes(p)}, {p->o, q_elems(p) * esize(p->o_dtype)}, {p->o_rest, q_elems(p) * 2},
                        {p->lse, static_cast<size_t>(rows_q(p)) * p->nheads * 4}, {p->dout, q_elems(p) * esize(p->x_dtype)}});
}

// ---------------------------------------------------------------- cache

// The pool, the table and the lengths, common to the write and the step.
template <typename P>
ssm_status_t pages_check(const P* p, int32_t seqs) {
  if (p->table_rows < 0 || p->pages < 0 || p->page_size <= 0)
    return fail(SSM_ERR_INVALID_ARG, "table_rows or pages is negative, or page_size not positive");
  if (p->page_size > 65536) return fail(SSM_ERR_UNSUPPORTED, "page_size must be at most 65536");
  if (static_cast<int64_t>(p->table_rows) * p->page_size > (1L << 30))
    return fail(SSM_ERR_UNSUPPORTED, "table_rows * page_size must be at most 2^30");
  if (static_cast<int64_t>(p->pages) * p->nkheads > (1LL << 58) / (static_cast<int64_t>(p->page_size) * p->d_head * 4))
    return fail(SSM_ERR_INVALID_ARG, "pages hold more than 2^58 bytes");
  if (p->cache_dtype != SSM_F32 && p->cache_dtype != SSM_BF16 && p->cache_dtype != SSM_E4M3)
    return fail(SSM_ERR_INVALID_ARG, "cache_dtype: unknown dtype");
  const bool scaled = p->cache_dtype == SSM_E4M3;
  if (!scaled && (p->k_scale || p->v_scale)) return fail(SSM_ERR_INVALID_ARG, "k_scale and v_scale belong to a cache in SSM_E4M3");
  if (p->pages > 0 && (!p->k_cache || !p->v_cache || (scaled && (!p->k_scale || !p->v_scale))))
    return fail(SSM_ERR_INVALID_ARG, "k_cache, v_cache, k_scale or v_scale is NULL");
  if (seqs > 0 && (!p->lens || (p->table_rows > 0 && !p->page_table))) return fail(SSM_ERR_INVALID_ARG, "lens or page_table is NULL");
  if (!aligned({p->k_cache, p->v_cache}, esize(p->cache_dtype)) || !aligned({p->k_scale, p->v_scale, p->lens, p->page_table}, 4))
    return fail(SSM_ERR_INVALID_ARG, "a cache, a scale, lens or page_table is not aligned to its element size");
  return SSM_OK;
}
template <typename P>
size_t pool_bytes(const P* p) { return static_cast<size_t>(p->pages) * p->nkheads * p->page_size * p->d_head * esize(p->cache_dtype); }
template <typename P>
size_t scale_bytes(const P* p) { return static_cast<size_t>(p->pages) * p->nkheads * 4; }
// rows of 8 elements in 16-byte groups (codes: 8-byte groups)
bool cache_vec(int32_t d, std::initializer_list<int64_t> strides, std::initializer_list<const void*> ps) {
  bool fits = d % 8 == 0 && aligned(ps, 16);
  for (int64_t s : strides) fits = fits && s % 8 == 0;
  return fits;
}

void cache_plan(const ssm_attn_cache_params_t* p, ssm::AttnCacheArgs& a) {
  const int64_t kw = static_cast<int64_t>(p->nkheads) * p->d_head;
  a.k = p->k;
  a.v = p->v;
  a.k_stride = p->k_stride ? p->k_stride : kw;
  a.v_stride = p->v_stride ? p->v_stride : kw;
  a.cu = p->cu_seqlens;
  a.lens = p->lens;
  a.table = p->page_table;
  a.nseq = p->num_seqs;
  a.seqlen = p->seqlen;
  a.hk = p->nkheads;
  a.D = p->d_head;
  a.table_rows = p->table_rows;
  a.pages = p->pages;
  a.page = p->page_size;
  a.tokens = static_cast<int64_t>(p->batch) * p->seqlen;
  a.k_cache = p->k_cache;
  a.v_cache = p->v_cache;
  a.k_scale = p->k_scale;
  a.v_scale = p->v_scale;
  a.vec = cache_vec(p->d_head, {a.k_stride, a.v_stride}, {p->k, p->v, p->k_cache, p->v_cache});
}

ssm_status_t attn_cache_check(const ssm_attn_cache_params_t* p) {
  if (!p) return fail(SSM_ERR_INVALID_ARG, "params is NULL");
  if (p->struct_size != sizeof(*p)) return fail(SSM_ERR_INVALID_ARG, "struct_size does not match this library");
  if (p->batch < 0 || p->seqlen < 0 || p->num_seqs < 0) return fail(SSM_ERR_INVALID_ARG, "batch, seqlen or num_seqs is negative");
  ssm_status_t s = heads_check(p->nkheads, p->nkheads, p->d_head);
  if (s != SSM_OK) return s;
  if (!valid_dtype(p->x_dtype)) return fail(SSM_ERR_INVALID_ARG, "x_dtype: unknown dtype");
  if (p->seqlen > ssm::kAttnAll) return fail(SSM_ERR_UNSUPPORTED, "seqlen must be at most 2^30");
  if (p->cu_seqlens ? p->batch != 1 : p->num_seqs != p->batch)
    return fail(SSM_ERR_INVALID_ARG, "packed sequences need batch 1; without cu_seqlens num_seqs must equal batch");
  s = pages_check(p, p->num_seqs);
  if (s != SSM_OK) return s;
  if (p->cache_dtype != p->x_dtype && p->cache_dtype != SSM_E4M3)
    return fail(SSM_ERR_UNSUPPORTED, "cache_dtype must be x_dtype or SSM_E4M3");
  const int64_t kw = static_cast<int64_t>(p->nkheads) * p->d_head, tokens = static_cast<int64_t>(p->batch) * p->seqlen;
  s = stride_check(p->k_stride, kw, tokens);
  if (s == SSM_OK) s = stride_check(p->v_stride, kw, tokens);
  if (s != SSM_OK) return s;
  if (tokens > 0 && (!p->k || !p->v)) return fail(SSM_ERR_INVALID_ARG, "k or v is NULL");
  if (!aligned({p->k, p->v}, esize(p->x_dtype)) || !aligned({p->cu_seqlens}, 4))
    return fail(SSM_ERR_INVALID_ARG, "k, v or cu_seqlens is not aligned to its element size");
  ssm::AttnCacheArgs a{};
  cache_plan(p, a);
  if (ssm::attn_cache_slots(a) > ((1L << 24) - 1) / p->nkheads)
    return fail(SSM_ERR_UNSUPPORTED, "too many pages and heads for one launch");
  const size_t table = static_cast<size_t>(p->num_seqs) * p->table_rows * 4;
  return check_overlap({{p->k_cache, pool_bytes(p)}, {p->v_cache, pool_bytes(p)}, {p->k_scale, scale_bytes(p)}, {p->v_scale, scale_bytes(p)}},
                       {rows_of(p->k, p->k_stride, kw, tokens, p->x_dtype), rows_of(p->v, p->v_stride, kw, tokens, p->x_dtype),
                        {p->cu_seqlens, cu_bytes(p)}, {p->lens, static_cast<size_t>(p->num_seqs) * 4}, {p->page_table, table}});
}

// ---------------------------------------------------------------- one token

// Parts of a sequence: up to 2048 workgroups (eight for every CU: sequences are of unlike lengths), a part 512
// keys at least, or 2048 where every CU has a workgroup without them, as the join is a launch of its own.
// 64 sequences of up to 8192 tokens, 8 key heads, in 8 bits: one part 145 us, two 135, four 128, eight 133;
// with a window of 1024: one part 41, two 52; one sequence of 32768: parts of 256 24.5 us, of 512 19.8.
void step_plan(const ssm_attn_decode_params_t* p, ssm::AttnStepArgs& a) {
  const int64_t qw = static_cast<int64_t>(p->nheads) * p->d_head, cap = static_cast<int64_t>(p->table_rows) * p->page_size;
  a.q = p->q;
  a.q_stride = p->q_stride ? p->q_stride : qw;
  a.k_cache = p->k_cache;
  a.v_cache = p->v_cache;
  a.k_scale = p->k_scale;
  a.v_scale = p->v_scale;
  a.table = p->page_table;
  a.lens = p->lens;
  a.batch = p->batch;
  a.h = p->nheads;
  a.hk = p->nkheads;
  a.D = p->d_head;
  a.table_rows = p->table_rows;
  a.pages = p->pages;
  a.page = p->page_size;
  a.page_shift = -1;
  for (int i = 0; i <= 16; ++i)
    if (p->page_size == 1 << i) a.page_shift = i;
  a.window = p->window == 0 || p->window >= cap ? ssm::kAttnAll : p->window;
  a.sinks = a.window == ssm::kAttnAll ? 0 : static_cast<int>(std::min<int64_t>(p->sinks, cap));
  a.scale = p->scale;
  const int64_t most = std::min<int64_t>(cap, a.window == ssm::kAttnAll ? cap : static_cast<int64_t>(a.window) + a.sinks);
  const int64_t groups = static_cast<int64_t>(p->batch) * p->nkheads * ssm::attn_head_tiles(p->nheads, p->nkheads);
  const int64_t want = std::max<int64_t>(1, 2048 / std::max<int64_t>(1, groups));
  const int64_t chunk = std::max<int64_t>(groups >= 256 ? 2048 : 512, ((most + want - 1) / want + 127) / 128 * 128);
  a.chunk = static_cast<int>(chunk);
  a.nsplit = static_cast<int>(std::max<int64_t>(1, (most + chunk - 1) / chunk));
}

size_t step_ws(const ssm_attn_decode_params_t* p) {
  ssm::AttnStepArgs a{};
  step_plan(p, a);
  return a.nsplit > 1 ? static_cast<size_t>(p->batch) * p->nheads * a.nsplit * (ssm::attn_dq(p->d_head) + 2) * 4 : 0;
}

ssm_status_t attn_step_common(const ssm_attn_decode_params_t* p) {
  if (p->batch < 0) return fail(SSM_ERR_INVALID_ARG, "batch is negative");
  ssm_status_t s = heads_check(p->nkheads, p->nheads, p->d_head);
  if (s == SSM_OK) s = mask_check(p);
  if (s != SSM_OK) return s;
  if (!valid_dtype(p->x_dtype) || !valid_dtype(p->o_dtype)) return fail(SSM_ERR_INVALID_ARG, "x_dtype or o_dtype: unknown dtype");
  s = pages_check(p, p->batch);
  if (s != SSM_OK) return s;
  if (p->cache_dtype != p->x_dtype && p->cache_dtype == SSM_F32)
    return fail(SSM_ERR_UNSUPPORTED, "a cache in f32 needs q in f32");
  if (static_cast<int64_t>(p->batch) * p->nheads >= (1L << 24)) return fail(SSM_ERR_UNSUPPORTED, "batch * nheads must be below 2^24");
  return SSM_OK;
}

ssm_status_t attn_step_check(const ssm_attn_decode_params_t* p) {
  if (!p) return fail(SSM_ERR_INVALID_ARG, "params is NULL");
  if (p->struct_size != sizeof(*p)) return fail(SSM_ERR_INVALID_ARG, "struct_size does not match this library");
  ssm_status_t s = attn_step_common(p);
  if (s != SSM_OK) return s;
  const int64_t qw = static_cast<int64_t>(p->nheads) * p->d_head;
  s = stride_check(p->q_stride, qw, p->batch);
  if (s != SSM_OK) return s;
  if (p->batch > 0 && (!p->q || !p->o)) return fail(SSM_ERR_INVALID_ARG, "q or o is NULL");
  if (!aligned({p->q}, esize(p->x_dtype)) || !aligned({p->o}, esize(p->o_dtype)))
    return fail(SSM_ERR_INVALID_ARG, "q or o is not aligned to its element size");
  const size_t need = step_ws(p);
  if (need > 0 && (!p->workspace || p->workspace_bytes < need)) return fail(SSM_ERR_WORKSPACE, "workspace is missing or too small");
  if (!aligned({p->workspace}, 256)) return fail(SSM_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  const size_t table = static_cast<size_t>(p->batch) * p->table_rows * 4;
  return check_overlap({{p->o, static_cast<size_t>(p->batch * qw) * esize(p->o_dtype)}, {p->workspace, need}},
                       {rows_of(p->q, p->q_stride, qw, p->batch, p->x_dtype), {p->k_cache, pool_bytes(p)}, {p->v_cache, pool_bytes(p)},
                        {p->k_scale, scale_bytes(p)}, {p->v_scale, scale_bytes(p)}, {p->lens, static_cast<size_t>(p->batch) * 4},
                        {p->page_table, table}});
}

}  // namespace

extern "C" {

ssm_status_t ssm_attn_check(const ssm_attn_params_t* p) { return done(attn_check(p)); }

size_t ssm_attn_workspace_size(const ssm_attn_params_t* p) {
  if (!p || p->struct_size != sizeof(*p) || !attn_fields(p)) return 0;
  return fwd_ws(p);
}

ssm_status_t ssm_attn_fwd(const ssm_attn_params_t* p, void* stream) {
  const ssm_status_t s = attn_check(p);
  if (s != SSM_OK) return s;
  ssm::AttnLaunch l{};
  attn_plan(p, l);
  l.a.o = p->o;
  l.a.lse = p->lse;
  l.a.o_rest = p->o_rest;
  l.a.nsplit = fwd_splits(p);
  l.a.part = static_cast<float*>(p->workspace);
  l.o_dtype = p->o_dtype;
  l.a.vec = vec_of(p->d_head, p->x_dtype, {l.a.q_stride, l.a.k_stride, l.a.v_stride}, {p->q, p->k, p->v, p->o, p->o_rest});
  return hip_status(ssm::launch_attn_fwd(l, static_cast<hipStream_t>(stream)));
}

ssm_status_t ssm_attn_bwd_check(const ssm_attn_bwd_params_t* p) { return done(attn_bwd_check(p)); }

size_t ssm_attn_bwd_workspace_size(const ssm_attn_bwd_params_t* p) {
  if (!p || p->struct_size != sizeof(*p) || !bwd_fields(p)) return 0;
  return bwd_ws(p).total;
}

ssm_status_t ssm_attn_bwd(const ssm_attn_bwd_params_t* p, void* stream) {
  const ssm_status_t s = attn_bwd_check(p);
  if (s != SSM_OK) return s;
  ssm::AttnLaunch l{};
  attn_plan(p, l);
  sink_plan(p, l.a);
  l.a.o = const_cast<void*>(p->o);
  l.a.lse = const_cast<float*>(p->lse);
  l.a.o_rest = const_cast<void*>(p->o_rest);
  l.a.dout = p->dout;
  l.a.dq = p->dq;
  l.a.dk = p->dk;
  l.a.dv = p->dv;
  l.a.grad_bf16 = p->grad_dtype == SSM_BF16;
  l.o_dtype = p->o_dtype;
  l.grad_dtype = p->grad_dtype;
  const BwdWs w = bwd_ws(p);
  unsigned char* const ws = static_cast<unsigned char*>(p->workspace);
  l.a.delta = reinterpret_cast<float*>(ws + w.delta);
  l.a.dk_part = reinterpret_cast<float*>(ws + w.dk_part);
  l.a.dv_part = reinterpret_cast<float*>(ws + w.dv_part);
  l.a.vec = vec_of(p->d_head, p->x_dtype, {l.a.q_stride, l.a.k_stride, l.a.v_stride},
                   {p->q, p->k, p->v, p->o, p->o_rest, p->dout, p->dq, p->dk, p->dv});
  return hip_status(ssm::launch_attn_bwd(l, static_cast<hipStream_t>(stream)));
}

ssm_status_t ssm_attn_cache_check(const ssm_attn_cache_params_t* p) { return done(attn_cache_check(p)); }

ssm_status_t ssm_attn_cache_write(const ssm_attn_cache_params_t* p, void* stream) {
  const ssm_status_t s = attn_cache_check(p);
  if (s != SSM_OK) return s;
  ssm::AttnCacheArgs a{};
  cache_plan(p, a);
  return hip_status(ssm::launch_attn_cache(a, p->x_dtype, p->cache_dtype, static_cast<hipStream_t>(stream)));
}

ssm_status_t ssm_attn_decode_check(const ssm_attn_decode_params_t* p) { return done(attn_step_check(p)); }

size_t ssm_attn_decode_workspace_size(const ssm_attn_decode_params_t* p) {
  if (!p || p->struct_size != sizeof(*p)) return 0;
  const ssm_status_t s = attn_step_common(p);
  ssm::set_error(SSM_OK, "");
  return s == SSM_OK ? step_ws(p) : 0;
}

ssm_status_t ssm_attn_decode_step(const ssm_attn_decode_params_t* p, void* stream) {
  const ssm_status_t s = attn_step_check(p);
  if (s != SSM_OK) return s;
  ssm::AttnStepLaunch l{};
  step_plan(p, l.a);
  l.a.o = p->o;
  l.a.part = static_cast<float*>(p->workspace);
  if (l.a.nsplit > 1) l.a.part_stat = l.a.part + static_cast<size_t>(p->batch) * p->nheads * l.a.nsplit * ssm::attn_dq(p->d_head);
  l.a.q_vec = vec_of(p->d_head, p->x_dtype, {l.a.q_stride}, {p->q});
  l.a.vec = vec_of(p->d_head, p->cache_dtype, {}, {p->k_cache, p->v_cache});
  l.in_dtype = p->x_dtype;
  l.cache_dtype = p->cache_dtype;
  l.o_dtype = p->o_dtype;
  return hip_status(ssm::launch_attn_step(l, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
