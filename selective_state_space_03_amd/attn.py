"""Binding of attention with a sliding window and sinks (ssm_attn_*) and its paged cache:
argument marshalling as in binding.py, no fallback."""
from __future__ import annotations

import ctypes
import math

import torch

from .binding import (
    _DT,
    SSM_E4M3,
    AttnBwdParams,
    AttnCacheParams,
    AttnDecodeParams,
    AttnParams,
    Call,
    _clear,
    _code,
    _empty,
    lib,
)
from .delta import _arg, _dtype, _fits, _gpu, _on, _rows, _workspace

_F32, _I32 = torch.float32, torch.int32
_byref = ctypes.byref
# the cache's element types; scales only beside the 8-bit one
_CACHE = {**_DT, torch.float8_e4m3fn: SSM_E4M3}


class _PackedGrads(Call):
    """A backward call of packed sequences: rows outside every one of them are not written by the library, so each
    run clears the gradients first, on the call's stream (the offsets may have changed since the last)."""

    def run(self):
        _clear(list(self.out.values()), self._stream.value)
        return super().run()


def _mask(p, window, sinks, scale, d):
    if window is not None and window < 1:
        raise ValueError("window must be at least 1 (None: no window)")
    if sinks < 0:
        raise ValueError("sinks must not be negative")
    _fits(max(window or 0, sinks), "window or sinks", "tokens")
    p.window, p.sinks = window or 0, sinks
    p.scale = 1.0 / math.sqrt(d) if scale is None else scale


def _offsets(cu, name, device):
    if cu.dim() != 1 or cu.numel() < 1:
        raise ValueError(f"{name} must hold the offsets of every sequence and the end of the last")
    return _arg(cu, name, cu.shape, _I32, device)


def _inputs(p, q, k, v, window, sinks, scale, cu_seqlens, cu_seqlens_k):
    batch, lq, h, d = q.shape
    lk, hk = k.shape[1], k.shape[2]
    _fits(max(batch, lq, lk, h, hk, d), "q or k", "sequences, tokens, heads or channels")
    dev = q.device
    p.struct_size = ctypes.sizeof(type(p))
    p.batch, p.seqlen, p.seqlen_k, p.nkheads, p.nheads, p.d_head = batch, lq, lk, hk, h, d
    p.q, p.q_stride = _rows(q, "q", (batch, lq, h, d), q.dtype, dev)
    p.x_dtype = _code(q, "q")
    p.k, p.k_stride = _rows(k, "k", (batch, lk, hk, d), q.dtype, dev)
    p.v, p.v_stride = _rows(v, "v", (batch, lk, hk, d), q.dtype, dev)
    _mask(p, window, sinks, scale, d)
    p.num_seqs = batch
    if cu_seqlens is not None:
        p.cu_seqlens = _offsets(cu_seqlens, "cu_seqlens", dev)
        p.num_seqs = cu_seqlens.numel() - 1
    if cu_seqlens_k is not None:
        if cu_seqlens is None or cu_seqlens_k.shape != cu_seqlens.shape:
            raise ValueError("cu_seqlens_k needs a cu_seqlens of as many sequences")
        p.cu_seqlens_k = _offsets(cu_seqlens_k, "cu_seqlens_k", dev)


def _rest(p, o, o_rest, dev):
    if o_rest is not None and o.dtype != torch.bfloat16:
        raise TypeError("o_rest goes with an o in bfloat16")
    p.o_rest = _arg(o_rest, "o_rest", o.shape, torch.bfloat16, dev)


def attn_fwd(q, k, v, *, window=None, sinks=0, scale=None, cu_seqlens=None, cu_seqlens_k=None, lse=None, o=None,
             o_dtype=None, o_rest=None, workspace=None, stream=None, prepare=False):
    """Causal attention with a sliding window and sinks over whole sequences (ssm_attn_fwd): q (batch, L, H, D),
    k and v (batch, Lk, Hk, D); head h reads key head h // (H // Hk).  The query at position p sees the keys
    j <= p with j > p - window (all without a window) or j < sinks; with more keys than queries the queries
    are the last positions.  cu_seqlens: int32 offsets on the GPU of sequences packed into one batch row
    (queries of no sequence are not written), cu_seqlens_k those of the keys where they differ.  scale
    defaults to 1 / sqrt(D).  q, k and v may be slices of a wider tensor along the token's row.  lse: a
    (batch, L, H) fp32 tensor that receives the log of the softmax's sum (attn_bwd needs it).  o_rest: a bfloat16
    tensor like o that receives what rounding took from an o in bfloat16, for attn_bwd.
    Returns o (batch, L, H, D), or with prepare=True a Call that enqueues this same call again."""
    L_ = lib()
    dev = _gpu(q, "q")
    p = AttnParams()
    _inputs(p, q, k, v, window, sinks, scale, cu_seqlens, cu_seqlens_k)
    if o is None:
        o = _empty(tuple(q.shape), o_dtype or q.dtype, dev, stream)
    p.lse = _arg(lse, "lse", q.shape[:3], _F32, dev)
    p.o = _arg(o, "o", q.shape, o.dtype, dev)
    p.o_dtype = _code(o, "o")
    _rest(p, o, o_rest, dev)
    workspace = _workspace(p, L_.ssm_attn_workspace_size(_byref(p)), workspace, dev, stream)
    call = Call(L_.ssm_attn_fwd, p, _on(dev, stream), o, (q, k, v, cu_seqlens, cu_seqlens_k, lse, o_rest, workspace))
    return call if prepare else call.run()


def attn_bwd(q, k, v, o, lse, dout, *, window=None, sinks=0, scale=None, cu_seqlens=None, cu_seqlens_k=None,
             grad_dtype=None, o_rest=None, workspace=None, stream=None, prepare=False):
    """Backward of attn_fwd (ssm_attn_bwd): the forward's inputs, its results o and lse, and dout (batch, L, H, D) in
    q's dtype.  Returns a dict of the gradients q, k and v in grad_dtype (fp32 unless given; zeros for rows of
    no sequence), or with prepare=True a Call whose run() enqueues it again (its .out is that dict).
    The rounding of an o in bfloat16 enters the gradients of q and k (as much as theirs to bfloat16, or several
    times that); with its o_rest from attn_fwd, or an o in fp32, it does not."""
    L_ = lib()
    dev = _gpu(q, "q")
    p = AttnBwdParams()
    _inputs(p, q, k, v, window, sinks, scale, cu_seqlens, cu_seqlens_k)
    if not isinstance(o, torch.Tensor) or not isinstance(lse, torch.Tensor):
        raise TypeError("o and lse must be the forward's results")
    p.o = _arg(o, "o", q.shape, o.dtype, dev)
    p.o_dtype = _code(o, "o")
    _rest(p, o, o_rest, dev)
    p.lse = _arg(lse, "lse", q.shape[:3], _F32, dev)
    p.dout = _arg(dout, "dout", q.shape, q.dtype, dev)
    gd = grad_dtype or _F32
    p.grad_dtype = _dtype(gd, "grad_dtype")
    out = {"q": _empty(tuple(q.shape), gd, dev, stream), "k": _empty(tuple(k.shape), gd, dev, stream),
           "v": _empty(tuple(v.shape), gd, dev, stream)}
    for name, field in (("q", "dq"), ("k", "dk"), ("v", "dv")):
        if out[name].numel() > 0:
            setattr(p, field, out[name].data_ptr())
    workspace = _workspace(p, L_.ssm_attn_bwd_workspace_size(_byref(p)), workspace, dev, stream)
    kind = Call if cu_seqlens is None else _PackedGrads
    call = kind(L_.ssm_attn_bwd, p, _on(dev, stream), out, (q, k, v, o, o_rest, lse, dout, cu_seqlens, cu_seqlens_k, workspace))
    return call if prepare else call.run()


def _pages(p, k_cache, v_cache, page_table, lens, k_scale, v_scale, seqs, hk, d, dev):
    if k_cache.dtype not in _CACHE:
        raise TypeError(f"k_cache: dtype {k_cache.dtype} not supported (float32, bfloat16 or float8_e4m3fn)")
    if k_cache.dim() != 4 or page_table.dim() != 2:
        raise ValueError("k_cache must be (pages, Hk, page_size, D) and page_table (sequences, rows)")
    pages, page = k_cache.shape[0], k_cache.shape[2]
    _fits(max(pages, page, page_table.shape[1]), "k_cache or page_table", "pages or rows")
    shape = (pages, hk, page, d)
    p.k_cache = _arg(k_cache, "k_cache", shape, k_cache.dtype, dev)
    p.v_cache = _arg(v_cache, "v_cache", shape, k_cache.dtype, dev)
    p.cache_dtype = _CACHE[k_cache.dtype]
    p.k_scale = _arg(k_scale, "k_scale", (pages, hk), _F32, dev)
    p.v_scale = _arg(v_scale, "v_scale", (pages, hk), _F32, dev)
    p.page_table = _arg(page_table, "page_table", (seqs, page_table.shape[1]), _I32, dev)
    p.lens = _arg(lens, "lens", (seqs,), _I32, dev)
    p.pages, p.page_size, p.table_rows = pages, page, page_table.shape[1]


def attn_cache_write(k, v, k_cache, v_cache, page_table, lens, *, cu_seqlens=None, k_scale=None, v_scale=None,
                     stream=None, prepare=False):
    """New tokens into the attention's paged cache (ssm_attn_cache_write): k and v (batch, L, Hk, D) go behind the
    lens (sequences,) int32 tokens that each sequence holds; with cu_seqlens sequences packed into one batch
    row.  k_cache, v_cache (pages, Hk, page_size, D) in k's dtype, or float8_e4m3fn with k_scale and v_scale
    (pages, Hk) fp32 (powers of two that the call chooses; a page's codes follow a scale that grows);
    page_table (sequences, rows) int32, entries out of range (-1) for pages that are not kept.  lens is not
    changed.  Returns (k_cache, v_cache), or with prepare=True a Call that enqueues this same write again."""
    L_ = lib()
    dev = _gpu(k, "k")
    batch, seqlen, hk, d = k.shape
    _fits(max(batch, seqlen, hk, d), "k", "sequences, tokens, heads or channels")
    p = AttnCacheParams()
    p.struct_size = ctypes.sizeof(AttnCacheParams)
    p.batch, p.seqlen, p.num_seqs, p.nkheads, p.d_head = batch, seqlen, batch, hk, d
    p.k, p.k_stride = _rows(k, "k", (batch, seqlen, hk, d), k.dtype, dev)
    p.x_dtype = _code(k, "k")
    p.v, p.v_stride = _rows(v, "v", (batch, seqlen, hk, d), k.dtype, dev)
    if cu_seqlens is not None:
        p.cu_seqlens = _offsets(cu_seqlens, "cu_seqlens", dev)
        p.num_seqs = cu_seqlens.numel() - 1
    _pages(p, k_cache, v_cache, page_table, lens, k_scale, v_scale, p.num_seqs, hk, d, dev)
    call = Call(L_.ssm_attn_cache_write, p, _on(dev, stream), (k_cache, v_cache),
                (k, v, page_table, lens, cu_seqlens, k_scale, v_scale))
    return call if prepare else call.run()


def attn_decode_step(q, k_cache, v_cache, page_table, lens, *, k_scale=None, v_scale=None, window=None, sinks=0, scale=None,
                     o=None, o_dtype=None, workspace=None, stream=None, prepare=False):
    """One query of each sequence over its pages (ssm_attn_decode_step): q (batch, H, D); the cache, its scales and
    page_table as in attn_cache_write; lens (batch,) int32 counts the query's own token, which has been written.
    window, sinks and scale as in attn_fwd; what pages hold in which no visible key lies does not matter.  Returns o
    (batch, H, D), or with prepare=True a Call that enqueues this same step again on each run()."""
    L_ = lib()
    dev = _gpu(q, "q")
    batch, h, d = q.shape
    _fits(max(batch, h, d), "q", "sequences, heads or channels")
    hk = k_cache.shape[1] if k_cache.dim() == 4 else 0
    p = AttnDecodeParams()
    p.struct_size = ctypes.sizeof(AttnDecodeParams)
    p.batch, p.nkheads, p.nheads, p.d_head = batch, hk, h, d
    p.q, p.q_stride = _rows(q, "q", (batch, h, d), q.dtype, dev)
    p.x_dtype = _code(q, "q")
    _pages(p, k_cache, v_cache, page_table, lens, k_scale, v_scale, batch, hk, d, dev)
    _mask(p, window, sinks, scale, d)
    if o is None:
        o = _empty((batch, h, d), o_dtype or q.dtype, dev, stream)
    p.o = _arg(o, "o", (batch, h, d), o.dtype, dev)
    p.o_dtype = _code(o, "o")
    workspace = _workspace(p, L_.ssm_attn_decode_workspace_size(_byref(p)), workspace, dev, stream)
    call = Call(L_.ssm_attn_decode_step, p, _on(dev, stream), o,
                (q, k_cache, v_cache, page_table, lens, k_scale, v_scale, workspace))
    return call if prepare else call.run()
