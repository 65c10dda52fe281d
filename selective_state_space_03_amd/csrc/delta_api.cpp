// Host side of the gated delta rule's and the block norm's entry points
// (include/ssm_mi355x.h): argument validation without a GPU, workspace layout,
// launches on the caller's stream.
#include <cmath>
#include <cstdio>
#include <initializer_list>

#include "../../include/ssm_mi355x.h"
#include "delta.h"

namespace {

ssm_status_t fail(ssm_status_t s, const char* what) { return static_cast<ssm_status_t>(ssm::set_error(s, what)); }
ssm_status_t ok() { return static_cast<ssm_status_t>(ssm::set_error(SSM_OK, "")); }

bool valid_dtype(int32_t d) { return d == SSM_F32 || d == SSM_BF16; }
size_t esize(int32_t d) { return d == SSM_BF16 ? 2 : 4; }
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
// No output may overlap an input or another output; `same` pairs may coincide exactly.
ssm_status_t check_overlap(std::initializer_list<Range> outs, std::initializer_list<Range> ins, const void* same_out,
                           const void* same_in) {
  for (const Range& o : outs) {
    for (const Range& i : ins) {
      if (o.p == same_out && i.p == same_in && o.p == i.p) continue;
      if (overlaps(o, i)) return fail(SSM_ERR_INVALID_ARG, "an output overlaps an input");
    }
    for (const Range& p : outs)
      if (&p != &o && overlaps(o, p)) return fail(SSM_ERR_INVALID_ARG, "two outputs overlap");
  }
  return SSM_OK;
}

// Whether the last of `rows` rows lies past every address: no range is formed of such a
// call, as its offsets would leave 63 bits.
bool far_rows(int64_t rows, std::initializer_list<int64_t> strides) {
  for (int64_t s : strides)
    if (rows > 0 && s > (static_cast<int64_t>(1) << 58) / rows) return true;
  return false;
}

// ---------------------------------------------------------------- gated delta rule

// Sizes and strides shared by the three entry points; tokens: rows of q, k, v.
template <typename P>
ssm_status_t delta_sizes(const P* p, long tokens) {
  if (p->nkheads <= 0 || p->nheads <= 0 || p->d_key <= 0 || p->d_value <= 0)
    return fail(SSM_ERR_INVALID_ARG, "nkheads, nheads, d_key and d_value must be positive");
  if (p->nheads % p->nkheads != 0) return fail(SSM_ERR_INVALID_ARG, "nheads must be a multiple of nkheads");
  if (p->d_key > ssm::kDeltaMaxK) return fail(SSM_ERR_UNSUPPORTED, "d_key must be at most 128");
  if (p->d_value > 65536 || p->nheads > 65536) return fail(SSM_ERR_UNSUPPORTED, "d_value and nheads must be at most 65536");
  if (!valid_dtype(p->x_dtype)) return fail(SSM_ERR_INVALID_ARG, "x_dtype: unknown dtype");
  if (!std::isfinite(p->scale)) return fail(SSM_ERR_INVALID_ARG, "scale must be finite");
  if (p->qk_norm && !(p->eps >= 0.0f && p->eps < INFINITY)) return fail(SSM_ERR_INVALID_ARG, "eps must be finite and not negative");
  const int64_t kw = static_cast<int64_t>(p->nkheads) * p->d_key, vw = static_cast<int64_t>(p->nheads) * p->d_value;
  const int64_t most = static_cast<int64_t>(1) << 40;
  if ((p->q_stride && (p->q_stride < kw || p->q_stride > most)) || (p->k_stride && (p->k_stride < kw || p->k_stride > most)) ||
      (p->v_stride && (p->v_stride < vw || p->v_stride > most)))
    return fail(SSM_ERR_INVALID_ARG, "q_stride, k_stride or v_stride is shorter than a token's row (or beyond 2^40)");
  if (far_rows(tokens, {p->q_stride, p->k_stride, p->v_stride}))
    return fail(SSM_ERR_INVALID_ARG, "q_stride, k_stride or v_stride times the tokens is beyond 2^58");
  if (tokens > 0 && (!p->q || !p->k || !p->v || !p->g || !p->beta))
    return fail(SSM_ERR_INVALID_ARG, "q, k, v, g or beta is NULL");
  if (!aligned({p->q, p->k, p->v}, esize(p->x_dtype)) || !aligned({p->g, p->beta}, 4))
    return fail(SSM_ERR_INVALID_ARG, "q, k, v, g or beta is not aligned to its element size");
  return SSM_OK;
}

template <typename P>
Range rows_of(const P* p, const void* ptr, int64_t stride, int64_t width, long tokens) {
  const int64_t st = stride ? stride : width;
  return {ptr, tokens > 0 ? static_cast<size_t>((tokens - 1) * st + width) * esize(p->x_dtype) : 0};
}

struct DeltaWs {
  size_t kf, qf, ktf, qtf, tf, pf, ttf, ptf, sc, s_chunk, ds_chunk, u_chunk, dr_chunk, dq_part, dk_part, total;
};

template <typename P>
long delta_slots(const P* p) {
  if (p->cu_seqlens) return static_cast<long>(p->seqlen) / ssm::kDeltaC + p->num_seqs;
  return static_cast<long>(p->batch) * ((static_cast<long>(p->seqlen) + ssm::kDeltaC - 1) / ssm::kDeltaC);
}

template <typename P>
DeltaWs delta_ws(const P* p, bool bwd) {
  const size_t slots = delta_slots(p), kc = slots * p->nkheads, hc = slots * p->nheads;
  const size_t nd = ssm::delta_kp(p->d_key) / 32;
  const size_t ni = p->x_dtype == SSM_BF16 ? 1 : 3, ns = 3;
  DeltaWs w{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at = align256(at + bytes);
    return o;
  };
  const size_t rows = kc * 4 * nd * ni * ssm::kDeltaFrag;
  w.kf = take(rows);
  w.qf = take(rows);
  w.ktf = take(rows);
  w.tf = take(hc * ssm::kDeltaTri * ns * ssm::kDeltaFrag);
  w.sc = take(hc * ssm::kDeltaSc * sizeof(float));
  if (!bwd) {
    w.pf = take(hc * ssm::kDeltaTri * ns * ssm::kDeltaFrag);
  } else {
    w.qtf = take(rows);
    w.ttf = take(hc * ssm::kDeltaTri * ns * ssm::kDeltaFrag);
    w.ptf = take(hc * ssm::kDeltaTri * ns * ssm::kDeltaFrag);
    const size_t vp = ssm::delta_vp(p->d_value);
    const size_t state = hc * ssm::delta_kp(p->d_key) * vp * sizeof(float), rows64 = hc * ssm::kDeltaC * vp * sizeof(float);
    w.s_chunk = take(state);
    w.ds_chunk = take(state);
    w.u_chunk = take(rows64);
    w.dr_chunk = take(rows64);
    if (p->nheads != p->nkheads) {
      const size_t part = static_cast<size_t>(p->batch) * p->seqlen * p->nheads * ssm::delta_kp(p->d_key) * sizeof(float);
      w.dq_part = take(part);
      w.dk_part = take(part);
    }
  }
  w.total = at;
  return w;
}

// A launch holds fewer than 2^32 threads: workgroups of 256, of 512 in the gradients of K > 64.
template <typename P>
bool delta_too_many(const P* p, bool bwd) {
  const long most = bwd && p->d_key > 64 ? 1L << 23 : 1L << 24;
  const long groups = static_cast<long>(p->num_seqs) * p->nheads;
  return delta_slots(p) > (most - 1) / p->nheads || ssm::delta_walk_blocks(groups, p->d_value, bwd) >= 1L << 24;
}

template <typename P>
bool delta_ws_fields(const P* p, bool bwd) {  // the fields the workspace size depends on are usable
  return p->batch >= 0 && p->seqlen >= 0 && p->num_seqs >= 0 && p->nkheads > 0 && p->nheads > 0 && p->nheads <= 65536 &&
         p->d_key > 0 && p->d_key <= ssm::kDeltaMaxK && p->d_value > 0 && p->d_value <= 65536 && valid_dtype(p->x_dtype) &&
         !delta_too_many(p, bwd);
}

// Everything but the outputs, common to forward and backward.
template <typename P>
ssm_status_t delta_seq_check(const P* p, bool bwd) {
  if (p->batch < 0 || p->seqlen < 0 || p->num_seqs < 0) return fail(SSM_ERR_INVALID_ARG, "batch, seqlen or num_seqs is negative");
  const long tokens = static_cast<long>(p->batch) * p->seqlen;
  const ssm_status_t s = delta_sizes(p, tokens);
  if (s != SSM_OK) return s;
  if (p->cu_seqlens ? p->batch != 1 : p->num_seqs != p->batch)
    return fail(SSM_ERR_INVALID_ARG, "packed sequences need batch 1; without cu_seqlens num_seqs must equal batch");
  if (!aligned({p->cu_seqlens, p->state_in}, 4)) return fail(SSM_ERR_INVALID_ARG, "cu_seqlens or state_in is not 4-byte aligned");
  if (delta_too_many(p, bwd))
    return fail(SSM_ERR_UNSUPPORTED, "too many chunks, sequences and heads for one launch");
  const size_t need = delta_ws(p, bwd).total;
  if (need > 0 && (!p->workspace || p->workspace_bytes < need)) return fail(SSM_ERR_WORKSPACE, "workspace is missing or too small");
  if (!aligned({p->workspace}, 256)) return fail(SSM_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return SSM_OK;
}

ssm_status_t delta_check(const ssm_delta_chunk_params_t* p) {
  if (!p) return fail(SSM_ERR_INVALID_ARG, "params is NULL");
  if (p->struct_size != sizeof(*p)) return fail(SSM_ERR_INVALID_ARG, "struct_size does not match this library");
  if (!valid_dtype(p->o_dtype)) return fail(SSM_ERR_INVALID_ARG, "o_dtype: unknown dtype");
  const ssm_status_t s = delta_seq_check(p, false);
  if (s != SSM_OK) return s;
  const long tokens = static_cast<long>(p->batch) * p->seqlen;
  if (tokens > 0 && !p->o) return fail(SSM_ERR_INVALID_ARG, "o is NULL");
  if (!aligned({p->o}, esize(p->o_dtype)) || !aligned({p->state_out}, 4))
    return fail(SSM_ERR_INVALID_ARG, "o or state_out is not aligned to its element size");
  const int64_t kw = static_cast<int64_t>(p->nkheads) * p->d_key, vw = static_cast<int64_t>(p->nheads) * p->d_value;
  const size_t state = static_cast<size_t>(p->num_seqs) * vw * p->d_key * 4, gb = static_cast<size_t>(tokens) * p->nheads * 4;
  return check_overlap({{p->o, static_cast<size_t>(tokens) * vw * esize(p->o_dtype)}, {p->state_out, state},
                        {p->workspace, delta_ws(p, false).total}},
                       {rows_of(p, p->q, p->q_stride, kw, tokens), rows_of(p, p->k, p->k_stride, kw, tokens),
                        rows_of(p, p->v, p->v_stride, vw, tokens), {p->g, gb}, {p->beta, gb}, {p->state_in, state},
                        {p->cu_seqlens, (static_cast<size_t>(p->num_seqs) + 1) * 4}},
                       p->state_out, p->state_in);
}

ssm_status_t delta_bwd_check(const ssm_delta_chunk_bwd_params_t* p) {
  if (!p) return fail(SSM_ERR_INVALID_ARG, "params is NULL");
  if (p->struct_size != sizeof(*p)) return fail(SSM_ERR_INVALID_ARG, "struct_size does not match this library");
  if (!valid_dtype(p->grad_dtype)) return fail(SSM_ERR_INVALID_ARG, "grad_dtype: unknown dtype");
  const ssm_status_t s = delta_seq_check(p, true);
  if (s != SSM_OK) return s;
  const long tokens = static_cast<long>(p->batch) * p->seqlen;
  if (tokens > 0 && !p->dout) return fail(SSM_ERR_INVALID_ARG, "dout is NULL");
  if (!aligned({p->dout}, esize(p->x_dtype)) || !aligned({p->dq, p->dk, p->dv}, esize(p->grad_dtype)) ||
      !aligned({p->dg, p->dbeta, p->dstate_in, p->dstate_out}, 4))
    return fail(SSM_ERR_INVALID_ARG, "dout or a gradient is not aligned to its element size");
  const int64_t kw = static_cast<int64_t>(p->nkheads) * p->d_key, vw = static_cast<int64_t>(p->nheads) * p->d_value;
  const size_t T = tokens, state = static_cast<size_t>(p->num_seqs) * vw * p->d_key * 4, gb = T * p->nheads * 4;
  const size_t eg = esize(p->grad_dtype);
  return check_overlap({{p->dq, T * kw * eg}, {p->dk, T * kw * eg}, {p->dv, T * vw * eg}, {p->dg, gb}, {p->dbeta, gb},
                        {p->dstate_in, state}, {p->workspace, delta_ws(p, true).total}},
                       {rows_of(p, p->q, p->q_stride, kw, tokens), rows_of(p, p->k, p->k_stride, kw, tokens),
                        rows_of(p, p->v, p->v_stride, vw, tokens), {p->g, gb}, {p->beta, gb}, {p->state_in, state},
                        {p->dout, T * vw * esize(p->x_dtype)}, {p->dstate_out, state},
                        {p->cu_seqlens, (static_cast<size_t>(p->num_seqs) + 1) * 4}},
                       p->dstate_in, p->dstate_out);
}

template <typename P>
void delta_plan(const P* p, bool bwd, ssm::DeltaLaunch& l) {
  ssm::DeltaArgs& a = l.a;
  const int64_t kw = static_cast<int64_t>(p->nkheads) * p->d_key, vw = static_cast<int64_t>(p->nheads) * p->d_value;
  a.q = p->q;
  a.k = p->k;
  a.v = p->v;
  a.q_stride = p->q_stride ? p->q_stride : kw;
  a.k_stride = p->k_stride ? p->k_stride : kw;
  a.v_stride = p->v_stride ? p->v_stride : vw;
  a.g = p->g;
  a.beta = p->beta;
  a.cu = p->cu_seqlens;
  a.state_in = p->state_in;
  a.nseq = p->num_seqs;
  a.seqlen = p->seqlen;
  a.hk = p->nkheads;
  a.h = p->nheads;
  a.K = p->d_key;
  a.V = p->d_value;
  a.tokens = static_cast<long>(p->batch) * p->seqlen;
  a.slots = a.tokens > 0 && p->num_seqs > 0 ? delta_slots(p) : 0;  // (no sequence: no chunk, and cu[1] is not there)
  a.scale = p->scale;
  a.eps = p->eps;
  a.qk_norm = p->qk_norm != 0;
  a.vec_qk = p->d_key % 8 == 0 && a.q_stride % 8 == 0 && a.k_stride % 8 == 0 && aligned({p->q, p->k}, 16);
  const DeltaWs w = delta_ws(p, bwd);
  unsigned char* ws = static_cast<unsigned char*>(p->workspace);
  a.kf = ws + w.kf;
  a.qf = ws + w.qf;
  a.ktf = ws + w.ktf;
  a.tf = ws + w.tf;
  a.sc = reinterpret_cast<float*>(ws + w.sc);
  if (!bwd) {
    a.pf = ws + w.pf;
  } else {
    a.qtf = ws + w.qtf;
    a.ttf = ws + w.ttf;
    a.ptf = ws + w.ptf;
    a.s_chunk = reinterpret_cast<float*>(ws + w.s_chunk);
    a.ds_chunk = reinterpret_cast<float*>(ws + w.ds_chunk);
    a.u_chunk = reinterpret_cast<float*>(ws + w.u_chunk);
    a.dr_chunk = reinterpret_cast<float*>(ws + w.dr_chunk);
    a.dq_part = reinterpret_cast<float*>(ws + w.dq_part);
    a.dk_part = reinterpret_cast<float*>(ws + w.dk_part);
  }
  l.in_dtype = p->x_dtype;
}

ssm_status_t delta_step_check(const ssm_delta_decode_params_t* p) {
  if (!p) return fail(SSM_ERR_INVALID_ARG, "params is NULL");
  if (p->struct_size != sizeof(*p)) return fail(SSM_ERR_INVALID_ARG, "struct_size does not match this library");
  if (p->batch < 0) return fail(SSM_ERR_INVALID_ARG, "batch is negative");
  if (!valid_dtype(p->o_dtype)) return fail(SSM_ERR_INVALID_ARG, "o_dtype: unknown dtype");
  const ssm_status_t s = delta_sizes(p, p->batch);
  if (s != SSM_OK) return s;
  const int64_t kw = static_cast<int64_t>(p->nkheads) * p->d_key, vw = static_cast<int64_t>(p->nheads) * p->d_value;
  if (p->batch * vw >= (1L << 27)) return fail(SSM_ERR_UNSUPPORTED, "batch * nheads * d_value must be below 2^27");
  if (p->batch == 0) return SSM_OK;
  if (!p->state || !p->o) return fail(SSM_ERR_INVALID_ARG, "state or o is NULL");
  if (!aligned({p->state}, 4) || !aligned({p->o}, esize(p->o_dtype)))
    return fail(SSM_ERR_INVALID_ARG, "state or o is not aligned to its element size");
  const size_t gb = static_cast<size_t>(p->batch) * p->nheads * 4;
  return check_overlap({{p->o, static_cast<size_t>(p->batch) * vw * esize(p->o_dtype)},
                        {p->state, static_cast<size_t>(p->batch) * vw * p->d_key * 4}},
                       {rows_of(p, p->q, p->q_stride, kw, p->batch), rows_of(p, p->k, p->k_stride, kw, p->batch),
                        rows_of(p, p->v, p->v_stride, vw, p->batch), {p->g, gb}, {p->beta, gb}},
                       nullptr, nullptr);
}

// ---------------------------------------------------------------- block norm

template <typename P>
bool norm_too_many(const P* p) {  // rows of all groups
  return p->rows > 0x7fffffffLL / (p->width / p->group_size);
}

template <typename P>
ssm_status_t norm_check_common(const P* p) {
  if (p->rows < 0 || p->width <= 0 || p->group_size <= 0) return fail(SSM_ERR_INVALID_ARG, "rows is negative, or width or group_size not positive");
  if (p->width % p->group_size != 0) return fail(SSM_ERR_INVALID_ARG, "group_size must divide width");
  if (p->group_size > ssm::kNormMax) return fail(SSM_ERR_UNSUPPORTED, "group_size must be at most 16384");
  if (p->group_size != p->width && (p->residual || p->scale || p->out_norm_w))
    return fail(SSM_ERR_UNSUPPORTED, "group_size must equal width where residual, scale or out_norm_w is given");
  if (!valid_dtype(p->x_dtype) || !valid_dtype(p->res_dtype)) return fail(SSM_ERR_INVALID_ARG, "x_dtype or res_dtype: unknown dtype");
  if (p->norm_w && p->norm_w_len != p->group_size && p->norm_w_len != p->width)
    return fail(SSM_ERR_INVALID_ARG, "norm_w_len must be group_size or width");
  if (p->gate_first && !p->z) return fail(SSM_ERR_INVALID_ARG, "gate_first without z");
  if (!(p->eps >= 0.0f && p->eps < INFINITY)) return fail(SSM_ERR_INVALID_ARG, "eps must be finite and not negative");
  const int64_t most = static_cast<int64_t>(1) << 40;
  if ((p->x_stride && (p->x_stride < p->width || p->x_stride > most)) || (p->z_stride && (p->z_stride < p->width || p->z_stride > most)))
    return fail(SSM_ERR_INVALID_ARG, "x_stride or z_stride is shorter than a row (or beyond 2^40)");
  if (far_rows(p->rows, {p->x_stride, p->z_stride}))
    return fail(SSM_ERR_INVALID_ARG, "x_stride or z_stride times the rows is beyond 2^58");
  if (norm_too_many(p))
    return fail(SSM_ERR_UNSUPPORTED, "rows * (width / group_size) must be below 2^31");
  if (p->rows > 0 && !p->x) return fail(SSM_ERR_INVALID_ARG, "x is NULL");
  if (!aligned({p->x, p->z}, esize(p->x_dtype)) || !aligned({p->residual}, esize(p->res_dtype)) ||
      !aligned({p->norm_w, p->scale, p->out_norm_w}, 4))
    return fail(SSM_ERR_INVALID_ARG, "an input is not aligned to its element size");
  return SSM_OK;
}

template <typename P>
Range norm_rows(const P* p, const void* ptr, int64_t stride) {
  const int64_t st = stride ? stride : p->width;
  return {ptr, p->rows > 0 ? static_cast<size_t>((p->rows - 1) * st + p->width) * esize(p->x_dtype) : 0};
}

ssm_status_t norm_check(const ssm_block_norm_params_t* p) {
  if (!p) return fail(SSM_ERR_INVALID_ARG, "params is NULL");
  if (p->struct_size != sizeof(*p)) return fail(SSM_ERR_INVALID_ARG, "struct_size does not match this library");
  const ssm_status_t s = norm_check_common(p);
  if (s != SSM_OK) return s;
  if (!valid_dtype(p->out_dtype)) return fail(SSM_ERR_INVALID_ARG, "out_dtype: unknown dtype");
  if (p->rows > 0 && !p->out && !p->residual_out) return fail(SSM_ERR_INVALID_ARG, "out and residual_out are both NULL");
  if (!aligned({p->out}, esize(p->out_dtype)) || !aligned({p->residual_out}, esize(p->res_dtype)))
    return fail(SSM_ERR_INVALID_ARG, "out or residual_out is not aligned to its element size");
  const size_t n = static_cast<size_t>(p->rows) * p->width, w = static_cast<size_t>(p->width) * 4;
  return check_overlap({{p->out, n * esize(p->out_dtype)}, {p->residual_out, n * esize(p->res_dtype)}},
                       {norm_rows(p, p->x, p->x_stride), norm_rows(p, p->z, p->z_stride), {p->residual, n * esize(p->res_dtype)},
                        {p->norm_w, static_cast<size_t>(p->norm_w ? p->norm_w_len : 0) * 4}, {p->scale, w}, {p->out_norm_w, w}},
                       p->residual_out, p->residual);
}

template <typename P>
int norm_period(const P* p) {
  return p->norm_w && p->norm_w_len != p->group_size ? p->width / p->group_size : 1;
}

size_t norm_bwd_ws(const ssm_block_norm_bwd_params_t* p) {
  const long rows = static_cast<long>(p->rows) * (p->width / p->group_size);
  return align256(static_cast<size_t>(ssm::norm_bwd_parts(rows, p->group_size, norm_period(p))) * 3 * p->group_size * sizeof(float));
}

ssm_status_t norm_bwd_check(const ssm_block_norm_bwd_params_t* p) {
  if (!p) return fail(SSM_ERR_INVALID_ARG, "params is NULL");
  if (p->struct_size != sizeof(*p)) return fail(SSM_ERR_INVALID_ARG, "struct_size does not match this library");
  const ssm_status_t s = norm_check_common(p);
  if (s != SSM_OK) return s;
  if (!valid_dtype(p->grad_dtype) || !valid_dtype(p->dout_dtype) || !valid_dtype(p->dres_dtype))
    return fail(SSM_ERR_INVALID_ARG, "grad_dtype, dout_dtype or dres_dtype: unknown dtype");
  if (p->rows > 0 && !p->dout && !p->dresidual_out) return fail(SSM_ERR_INVALID_ARG, "dout and dresidual_out are both NULL");
  if ((p->dz && !p->z) || (p->dresidual && !p->residual) || (p->dnorm_w && !p->norm_w) || (p->dscale && !p->scale) ||
      (p->dout_norm_w && !p->out_norm_w))
    return fail(SSM_ERR_INVALID_ARG, "a gradient is asked for whose input was not given");
  if (!aligned({p->dx, p->dz}, esize(p->grad_dtype)) || !aligned({p->dresidual}, esize(p->res_dtype)) ||
      !aligned({p->dout}, esize(p->dout_dtype)) || !aligned({p->dresidual_out}, esize(p->dres_dtype)) ||
      !aligned({p->dnorm_w, p->dscale, p->dout_norm_w}, 4))
    return fail(SSM_ERR_INVALID_ARG, "a gradient is not aligned to its element size");
  if (norm_period(p) > ssm::kNormMaxPeriod)
    return fail(SSM_ERR_UNSUPPORTED, "norm_w of the whole width must hold at most 2^22 groups");
  const size_t need = norm_bwd_ws(p);
  if (!p->workspace || p->workspace_bytes < need) return fail(SSM_ERR_WORKSPACE, "workspace is missing or too small");
  if (!aligned({p->workspace}, 256)) return fail(SSM_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  const size_t n = static_cast<size_t>(p->rows) * p->width, w = static_cast<size_t>(p->width) * 4;
  const size_t nw = static_cast<size_t>(p->norm_w ? p->norm_w_len : 0) * 4;
  return check_overlap({{p->dx, n * esize(p->grad_dtype)}, {p->dz, n * esize(p->grad_dtype)}, {p->dresidual, n * esize(p->res_dtype)},
                        {p->dnorm_w, nw}, {p->dscale, w}, {p->dout_norm_w, w}, {p->workspace, need}},
                       {norm_rows(p, p->x, p->x_stride), norm_rows(p, p->z, p->z_stride), {p->residual, n * esize(p->res_dtype)},
                        {p->norm_w, nw}, {p->scale, w}, {p->out_norm_w, w}, {p->dout, n * esize(p->dout_dtype)},
                        {p->dresidual_out, n * esize(p->dres_dtype)}},
                       nullptr, nullptr);
}

template <typename P>
void norm_plan(const P* p, ssm::NormArgs& a) {
  a.x = p->x;
  a.z = p->z;
  a.res = p->residual;
  a.norm_w = p->norm_w;
  a.scale = p->scale;
  a.out_w = p->out_norm_w;
  a.groups = p->width / p->group_size;
  a.rows = static_cast<long>(p->rows) * a.groups;
  a.n = p->group_size;
  a.w_period = norm_period(p);
  a.x_stride = p->x_stride ? p->x_stride : p->width;
  a.z_stride = p->z_stride ? p->z_stride : p->width;
  a.x_dtype = p->x_dtype;
  a.res_dtype = p->res_dtype;
  a.eps = p->eps;
  a.gate_first = p->gate_first != 0;
}
// Elements per access: rows, strides and every pointer must be multiples of them.
int norm_vec(const ssm::NormArgs& a, std::initializer_list<const void*> ps) {
  for (int v : {8, 4})
    if (a.n % v == 0 && a.x_stride % v == 0 && a.z_stride % v == 0 && aligned(ps, 16)) return v;
  return 1;
}

ssm_status_t hip_status(hipError_t e) {
  if (e == hipSuccess) return ok();
  char buf[200];
  std::snprintf(buf, sizeof(buf), "HIP launch failed: %s", hipGetErrorString(e));
  return fail(SSM_ERR_HIP, buf);
}

}  // namespace

extern "C" {

ssm_status_t ssm_delta_chunk_check(const ssm_delta_chunk_params_t* p) {
  const ssm_status_t s = delta_check(p);
  return s == SSM_OK ? ok() : s;
}

size_t ssm_delta_chunk_workspace_size(const ssm_delta_chunk_params_t* p) {
  if (!p || p->struct_size != sizeof(*p) || !delta_ws_fields(p, false)) return 0;
  return delta_ws(p, false).total;
}

ssm_status_t ssm_delta_chunk_fwd(const ssm_delta_chunk_params_t* p, void* stream) {
  const ssm_status_t s = delta_check(p);
  if (s != SSM_OK) return s;
  ssm::DeltaLaunch l{};
  delta_plan(p, false, l);
  l.a.state_out = p->state_out;
  l.a.o = p->o;
  l.o_dtype = p->o_dtype;
  l.a.vec_state = p->d_key % 4 == 0 && aligned({p->state_in, p->state_out}, 16);
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = ssm::launch_delta_prep(l, false, st);
  if (e == hipSuccess) e = ssm::launch_delta_pass(l, false, st);
  return hip_status(e);
}

ssm_status_t ssm_delta_chunk_bwd_check(const ssm_delta_chunk_bwd_params_t* p) {
  const ssm_status_t s = delta_bwd_check(p);
  return s == SSM_OK ? ok() : s;
}

size_t ssm_delta_chunk_bwd_workspace_size(const ssm_delta_chunk_bwd_params_t* p) {
  if (!p || p->struct_size != sizeof(*p) || !delta_ws_fields(p, true)) return 0;
  return delta_ws(p, true).total;
}

ssm_status_t ssm_delta_chunk_bwd(const ssm_delta_chunk_bwd_params_t* p, void* stream) {
  const ssm_status_t s = delta_bwd_check(p);
  if (s != SSM_OK) return s;
  ssm::DeltaLaunch l{};
  delta_plan(p, true, l);
  ssm::DeltaArgs& a = l.a;
  a.dout = p->dout;
  a.dstate_out = p->dstate_out;
  a.dq = p->dq;
  a.dk = p->dk;
  a.dv = p->dv;
  a.dg = p->dg;
  a.dbeta = p->dbeta;
  a.dstate_in = p->dstate_in;
  l.grad_dtype = p->grad_dtype;
  a.vec_state = p->d_key % 4 == 0 && aligned({p->state_in, p->dstate_out, p->dstate_in}, 16);
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = ssm::launch_delta_prep(l, true, st);
  if (e == hipSuccess && a.slots > 0) e = ssm::launch_delta_pass(l, true, st);
  if (e == hipSuccess) e = ssm::launch_delta_reverse(l, st);
  if (e == hipSuccess) e = ssm::launch_delta_grads(l, st);
  return hip_status(e);
}

ssm_status_t ssm_delta_decode_check(const ssm_delta_decode_params_t* p) {
  const ssm_status_t s = delta_step_check(p);
  return s == SSM_OK ? ok() : s;
}

ssm_status_t ssm_delta_decode_step(const ssm_delta_decode_params_t* p, void* stream) {
  const ssm_status_t s = delta_step_check(p);
  if (s != SSM_OK) return s;
  ssm::DeltaStepArgs a{};
  const int64_t kw = static_cast<int64_t>(p->nkheads) * p->d_key, vw = static_cast<int64_t>(p->nheads) * p->d_value;
  a.q = p->q;
  a.k = p->k;
  a.v = p->v;
  a.q_stride = p->q_stride ? p->q_stride : kw;
  a.k_stride = p->k_stride ? p->k_stride : kw;
  a.v_stride = p->v_stride ? p->v_stride : vw;
  a.g = p->g;
  a.beta = p->beta;
  a.state = p->state;
  a.o = p->o;
  a.batch = p->batch;
  a.hk = p->nkheads;
  a.h = p->nheads;
  a.K = p->d_key;
  a.V = p->d_value;
  a.o_bf16 = p->o_dtype == SSM_BF16;
  a.scale = p->scale;
  a.eps = p->eps;
  a.qk_norm = p->qk_norm != 0;
  a.vec = p->d_key % 8 == 0 && a.q_stride % 8 == 0 && a.k_stride % 8 == 0 && aligned({p->q, p->k, p->state}, 16);
  return hip_status(ssm::launch_delta_step(a, p->x_dtype, static_cast<hipStream_t>(stream)));
}

ssm_status_t ssm_block_norm_check(const ssm_block_norm_params_t* p) {
  const ssm_status_t s = norm_check(p);
  return s == SSM_OK ? ok() : s;
}

ssm_status_t ssm_block_norm_fwd(const ssm_block_norm_params_t* p, void* stream) {
  const ssm_status_t s = norm_check(p);
  if (s != SSM_OK) return s;
  ssm::NormArgs a{};
  norm_plan(p, a);
  a.out = p->out;
  a.res_out = p->residual_out;
  a.out_dtype = p->out_dtype;
  a.vec = norm_vec(a, {p->x, p->z, p->norm_w, p->residual, p->scale, p->residual_out, p->out_norm_w, p->out});
  return hip_status(ssm::launch_norm_fwd(a, static_cast<hipStream_t>(stream)));
}

ssm_status_t ssm_block_norm_bwd_check(const ssm_block_norm_bwd_params_t* p) {
  const ssm_status_t s = norm_bwd_check(p);
  return s == SSM_OK ? ok() : s;
}

size_t ssm_block_norm_bwd_workspace_size(const ssm_block_norm_bwd_params_t* p) {
  if (!p || p->struct_size != sizeof(*p) || p->rows < 0 || p->width <= 0 || p->group_size <= 0 ||
      p->width % p->group_size != 0 || p->group_size > ssm::kNormMax || norm_too_many(p) ||
      norm_period(p) > ssm::kNormMaxPeriod)
    return 0;
  return norm_bwd_ws(p);
}

ssm_status_t ssm_block_norm_bwd(const ssm_block_norm_bwd_params_t* p, void* stream) {
  const ssm_status_t s = norm_bwd_check(p);
  if (s != SSM_OK) return s;
  ssm::NormArgs a{};
  norm_plan(p, a);
  a.dout = p->dout;
  a.dres = p->dresidual_out;
  a.dout_dtype = p->dout_dtype;
  a.dres_dtype = p->dres_dtype;
  a.grad_dtype = p->grad_dtype;
  a.dx = p->dx;
  a.dz = p->dz;
  a.dresidual = p->dresidual;
  a.dnorm_w = p->dnorm_w;
  a.dscale = p->dscale;
  a.dout_w = p->dout_norm_w;
  a.part = static_cast<float*>(p->workspace);
  a.parts = ssm::norm_bwd_parts(a.rows, a.n, a.w_period);
  a.vec = norm_vec(a, {p->x, p->z, p->norm_w, p->residual, p->scale, p->out_norm_w, p->dout, p->dresidual_out, p->dx, p->dz,
                       p->dresidual});
  return hip_status(ssm::launch_norm_bwd(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
