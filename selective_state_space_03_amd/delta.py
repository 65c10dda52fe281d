"""Binding of the gated delta rule (ssm_delta_*) and the block norm
(ssm_block_norm_*): argument marshalling as in binding.py, no fallback."""
from __future__ import annotations

import ctypes
import math

import torch

from .binding import (
    _DT,
    BlockNormBwdParams,
    BlockNormParams,
    Call,
    DeltaChunkBwdParams,
    DeltaChunkParams,
    DeltaDecodeParams,
    _Handle,
    _clear,
    _code,
    _empty,
    _ptr,
    _stream,
    lib,
)

_F32 = torch.float32
_byref = ctypes.byref
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(device, stream):
    """The stream's handle, without building a Stream object for the current one."""
    if stream is None and _raw_stream is not None and device.index is not None:
        return _Handle(_raw_stream(device.index), device.index)
    return _stream(device, stream)


def _arg(t, name, shape, dtype, device):
    """_ptr, with its checks in the fewest calls for a tensor that passes them (a decode step's
    launch is bound by the host)."""
    if t is None:
        return None
    if type(t) is torch.Tensor and t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.device == device:
        return t.data_ptr() or None
    return _ptr(t, name, shape, dtype, device)


def _gpu(t, name):
    """The device that every other argument is compared with, which has to be a GPU."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    return t.device


def _fits(n, name, what):
    """Sizes that the library holds in 31 bits: ctypes would cut a longer one without a word."""
    if n > 0x7fffffff:
        raise ValueError(f"{name} has {n} {what}, more than 2^31 - 1")


def _dtype(d, name):
    if d not in _DT:
        raise TypeError(f"{name}: dtype {d} not supported (float32 or bfloat16)")
    return _DT[d]


def _rows(t, name, shape, dtype, device):
    """Pointer and row stride of a tensor whose rows (its last two dimensions) are dense and whose
    leading dimensions step evenly from row to row, as a slice of a wider projection does."""
    if t.is_contiguous():
        return _arg(t, name, shape, dtype, device), 0
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.numel() == 0:
        return None, 0
    lead = t.dim() - 2
    width, want = t.shape[-1] * t.shape[-2], (t.shape[-1], 1)
    dense = all(n == 1 or s == w for n, s, w in zip(t.shape[-2:], t.stride()[-2:], want))
    row = None
    for i in range(lead - 1, -1, -1):  # from the innermost leading dimension out
        if t.shape[i] == 1:
            continue
        if row is None:
            row, span = t.stride(i), t.stride(i) * t.shape[i]
        elif t.stride(i) == span:
            span *= t.shape[i]
        else:
            dense = False
    if row is None:
        row = width
    if not dense or row < width:
        raise ValueError(f"{name} must have dense rows at an even stride (strides {t.stride()} of shape {tuple(t.shape)})")
    return t.data_ptr(), row


class _PackedGrads(Call):
    """A backward call of packed sequences: tokens outside every one of them are not written by the library, so
    each run clears their gradients first, on the call's stream (the offsets may have changed since the last)."""

    def run(self):
        _clear([self.out[name] for name in ("q", "k", "v", "g", "beta")], self._stream.value)
        return super().run()


def _workspace(p, need, workspace, dev, stream):
    if workspace is None and need > 0:
        workspace = _empty(need, torch.uint8, dev, stream)
    if workspace is not None:
        p.workspace = _ptr(workspace, "workspace", device=dev)
        p.workspace_bytes = workspace.numel() * workspace.element_size()
    return workspace


def _delta_inputs(p, q, k, v, g, beta, scale, qk_norm, eps, cu_seqlens, state_in):
    batch, seqlen, hk, dk = q.shape
    _fits(max(batch, seqlen), "q", "sequences or tokens")
    h, dv = v.shape[2], v.shape[3]
    dev = q.device
    p.struct_size = ctypes.sizeof(type(p))
    p.batch, p.seqlen, p.nkheads, p.nheads, p.d_key, p.d_value = batch, seqlen, hk, h, dk, dv
    p.q, p.q_stride = _rows(q, "q", (batch, seqlen, hk, dk), q.dtype, dev)
    p.x_dtype = _code(q, "q")
    p.k, p.k_stride = _rows(k, "k", (batch, seqlen, hk, dk), q.dtype, dev)
    p.v, p.v_stride = _rows(v, "v", (batch, seqlen, h, dv), q.dtype, dev)
    p.g = _arg(g, "g", (batch, seqlen, h), _F32, dev)
    p.beta = _arg(beta, "beta", (batch, seqlen, h), _F32, dev)
    p.scale = 1.0 / math.sqrt(dk) if scale is None else scale
    p.qk_norm = 1 if qk_norm else 0
    p.eps = eps
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must hold the offsets of every sequence and the end of the last")
        p.num_seqs = cu_seqlens.numel() - 1
        p.cu_seqlens = _ptr(cu_seqlens, "cu_seqlens", None, torch.int32, dev)
    else:
        p.num_seqs = batch
    shape = (p.num_seqs, h, dv, dk)
    p.state_in = _arg(state_in, "state_in", shape, _F32, dev)
    return shape


def delta_chunk_fwd(q, k, v, g, beta, *, scale=None, qk_norm=False, eps=1e-6, cu_seqlens=None, state_in=None,
                    state_out=None, o=None, o_dtype=None, workspace=None, stream=None, prepare=False):
    """The gated delta rule over whole sequences (ssm_delta_chunk_fwd): q, k (batch, L, Hk, K),
    v (batch, L, H, V), g and beta (batch, L, H) fp32; head h reads key head h // (H // Hk).
    cu_seqlens: int32 offsets on the GPU of sequences packed into one batch row (tokens of no sequence
    are not written).  scale defaults to
    1 / sqrt(K); qk_norm scales q and k to unit length first.  state_in / state_out
    (sequences, H, V, K) fp32.  q, k and v may be slices of a wider tensor along the token's row.
    Returns o (batch, L, H, V), or with prepare=True a Call that enqueues this same call again."""
    L_ = lib()
    dev = _gpu(q, "q")
    p = DeltaChunkParams()
    shape = _delta_inputs(p, q, k, v, g, beta, scale, qk_norm, eps, cu_seqlens, state_in)
    if o is None:
        o = _empty(v.shape, o_dtype or q.dtype, dev, stream)
    p.state_out = _arg(state_out, "state_out", shape, _F32, dev)
    p.o = _arg(o, "o", v.shape, o.dtype, dev)
    p.o_dtype = _code(o, "o")
    workspace = _workspace(p, L_.ssm_delta_chunk_workspace_size(_byref(p)), workspace, dev, stream)
    call = Call(L_.ssm_delta_chunk_fwd, p, _on(dev, stream), o, (q, k, v, g, beta, cu_seqlens, state_in, state_out,
                                                                    workspace))
    return call if prepare else call.run()


def delta_chunk_bwd(q, k, v, g, beta, dout, *, scale=None, qk_norm=False, eps=1e-6, cu_seqlens=None, state_in=None,
                    dstate_out=None, grad_dtype=None, workspace=None, stream=None, prepare=False):
    """Backward of delta_chunk_fwd (ssm_delta_chunk_bwd): the forward's inputs, dout (batch, L, H, V) in
    q's dtype and optionally the final state's gradient.  Returns a dict of gradients: q, k, v in
    grad_dtype (fp32 unless given), g, beta and, where a state was given, state_in in fp32 (zeros for
    tokens of no sequence); or with
    prepare=True a Call whose run() enqueues it again (its .out is that dict)."""
    L_ = lib()
    dev = _gpu(q, "q")
    p = DeltaChunkBwdParams()
    shape = _delta_inputs(p, q, k, v, g, beta, scale, qk_norm, eps, cu_seqlens, state_in)
    p.dout = _arg(dout, "dout", v.shape, q.dtype, dev)
    p.dstate_out = _arg(dstate_out, "dstate_out", shape, _F32, dev)
    gd = grad_dtype or _F32
    p.grad_dtype = _dtype(gd, "grad_dtype")
    out = {"q": _empty(tuple(q.shape), gd, dev, stream), "k": _empty(tuple(k.shape), gd, dev, stream),
           "v": _empty(tuple(v.shape), gd, dev, stream), "g": _empty(tuple(g.shape), _F32, dev, stream),
           "beta": _empty(tuple(g.shape), _F32, dev, stream)}
    if state_in is not None:
        out["state_in"] = _empty(shape, _F32, dev, stream)
    for name, field in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("state_in", "dstate_in")):
        if name in out and out[name].numel() > 0:
            setattr(p, field, out[name].data_ptr())
    workspace = _workspace(p, L_.ssm_delta_chunk_bwd_workspace_size(_byref(p)), workspace, dev, stream)
    kind = Call if cu_seqlens is None else _PackedGrads
    call = kind(L_.ssm_delta_chunk_bwd, p, _on(dev, stream), out, (q, k, v, g, beta, dout, cu_seqlens, state_in,
                                                                   dstate_out, workspace))
    return call if prepare else call.run()


def delta_decode_step(q, k, v, g, beta, state, *, scale=None, qk_norm=False, eps=1e-6, o=None, o_dtype=None, stream=None,
                      prepare=False):
    """One token of the gated delta rule (ssm_delta_decode_step): q, k (batch, Hk, K), v (batch, H, V),
    g and beta (batch, H) fp32, state (batch, H, V, K) fp32 updated in place.  Returns o (batch, H, V),
    or with prepare=True a Call that enqueues this same step again on each run()."""
    L_ = lib()
    dev = _gpu(q, "q")
    batch, hk, dk = q.shape
    _fits(batch, "q", "sequences")
    h, dv = v.shape[1], v.shape[2]
    p = DeltaDecodeParams()
    p.struct_size = ctypes.sizeof(DeltaDecodeParams)
    p.batch, p.nkheads, p.nheads, p.d_key, p.d_value = batch, hk, h, dk, dv
    p.q, p.q_stride = _rows(q, "q", (batch, hk, dk), q.dtype, dev)
    p.x_dtype = _code(q, "q")
    p.k, p.k_stride = _rows(k, "k", (batch, hk, dk), q.dtype, dev)
    p.v, p.v_stride = _rows(v, "v", (batch, h, dv), q.dtype, dev)
    p.g = _arg(g, "g", (batch, h), _F32, dev)
    p.beta = _arg(beta, "beta", (batch, h), _F32, dev)
    p.scale = 1.0 / math.sqrt(dk) if scale is None else scale
    p.qk_norm = 1 if qk_norm else 0
    p.eps = eps
    p.state = _arg(state, "state", (batch, h, dv, dk), _F32, dev)
    if o is None:
        o = _empty((batch, h, dv), o_dtype or q.dtype, dev, stream)
    p.o = _arg(o, "o", (batch, h, dv), o.dtype, dev)
    p.o_dtype = _code(o, "o")
    call = Call(L_.ssm_delta_decode_step, p, _on(dev, stream), o, (q, k, v, g, beta, state))
    return call if prepare else call.run()


def _norm_inputs(p, x, norm_w, z, gate_first, residual, scale, out_norm_w, group_size, eps):
    dev, width = x.device, x.shape[-1]
    _fits(width, "x", "values a row")
    shape = tuple(x.shape)
    rows = shape[0] if len(shape) == 2 else math.prod(shape[:-1])
    p.struct_size = ctypes.sizeof(type(p))
    p.rows, p.width = rows, width
    if group_size is None:
        n = norm_w.numel() if norm_w is not None else width
        group_size = n if 0 < n < width and width % n == 0 else width
    p.group_size = int(group_size)

    def lines(t, name):  # rows of the last dimension at an even stride
        if t is None or t.is_contiguous():
            return _arg(t, name, shape, x.dtype, dev), 0
        return _rows(t.unsqueeze(-2), name, shape[:-1] + (1, width), x.dtype, dev)

    p.x, p.x_stride = lines(x, "x")
    p.x_dtype = _code(x, "x")
    p.z, p.z_stride = lines(z, "z")
    p.gate_first = 1 if gate_first else 0
    if norm_w is not None:
        p.norm_w = _arg(norm_w, "norm_w", (norm_w.numel(),), _F32, dev)
        p.norm_w_len = norm_w.numel()
    p.residual = _arg(residual, "residual", shape, residual.dtype, dev) if residual is not None else None
    p.res_dtype = _code(residual, "residual") if residual is not None else 0
    p.scale = _arg(scale, "scale", (width,), _F32, dev)
    p.out_norm_w = _arg(out_norm_w, "out_norm_w", (width,), _F32, dev)
    p.eps = eps
    return shape


def block_norm_fwd(x, *, norm_w=None, z=None, gate_first=False, residual=None, scale=None, out_norm_w=None,
                   group_size=None, eps=1e-6, out=None, out_dtype=None, residual_out=None, stream=None, prepare=False):
    """The norms before and after a block with its gate and residual scale (ssm_block_norm_fwd), on the last
    dimension of x: a = norm(x) norm_w SiLU(z) (the gate inside the norm with gate_first; in groups of
    group_size, by default len(norm_w)), t = residual + scale a, out = norm(t) out_norm_w.  Returns
    (out, residual_out): out is None where a residual but no out_norm_w is given (t is residual_out
    then), residual_out is None without a residual; with prepare=True a Call whose .out is that pair."""
    L_ = lib()
    dev = _gpu(x, "x")
    p = BlockNormParams()
    shape = _norm_inputs(p, x, norm_w, z, gate_first, residual, scale, out_norm_w, group_size, eps)
    if residual is not None and residual_out is None:
        residual_out = _empty(shape, residual.dtype, dev, stream)
    if out is None and (residual is None or out_norm_w is not None):
        out = _empty(shape, out_dtype or x.dtype, dev, stream)
    if residual_out is not None:
        p.residual_out = _arg(residual_out, "residual_out", shape, (residual if residual is not None else residual_out).dtype, dev)
        p.res_dtype = _code(residual_out, "residual_out")
    if out is not None:
        p.out = _arg(out, "out", shape, out.dtype, dev)
    p.out_dtype = _code(out, "out") if out is not None else 0
    call = Call(L_.ssm_block_norm_fwd, p, _on(dev, stream), (out, residual_out),
                (x, norm_w, z, residual, scale, out_norm_w))
    return call if prepare else call.run()


def block_norm_bwd(x, *, norm_w=None, z=None, gate_first=False, residual=None, scale=None, out_norm_w=None,
                   group_size=None, eps=1e-6, dout=None, dresidual=None, grad_dtype=None, workspace=None, stream=None,
                   prepare=False):
    """Backward of block_norm_fwd (ssm_block_norm_bwd): the forward's inputs and the gradients of its two
    results.  Returns a dict of gradients for the inputs that were given: x and z in grad_dtype (fp32
    unless given), residual in the residual's dtype, norm_w, scale and out_norm_w in fp32."""
    L_ = lib()
    dev = _gpu(x, "x")
    p = BlockNormBwdParams()
    shape = _norm_inputs(p, x, norm_w, z, gate_first, residual, scale, out_norm_w, group_size, eps)
    if dout is not None:
        p.dout, p.dout_dtype = _arg(dout, "dout", shape, dout.dtype, dev), _code(dout, "dout")
    if dresidual is not None:
        p.dresidual_out = _arg(dresidual, "dresidual", shape, dresidual.dtype, dev)
        p.dres_dtype = _code(dresidual, "dresidual")
    gd = grad_dtype or _F32
    p.grad_dtype = _dtype(gd, "grad_dtype")
    out = {"x": _empty(shape, gd, dev, stream)}
    if z is not None:
        out["z"] = _empty(shape, gd, dev, stream)
    if norm_w is not None:
        out["norm_w"] = _empty((norm_w.numel(),), _F32, dev, stream)
    if residual is not None:
        out["residual"] = _empty(shape, residual.dtype, dev, stream)
    if scale is not None:
        out["scale"] = _empty((shape[-1],), _F32, dev, stream)
    if out_norm_w is not None:
        out["out_norm_w"] = _empty((shape[-1],), _F32, dev, stream)
    for name, field in (("x", "dx"), ("z", "dz"), ("norm_w", "dnorm_w"), ("residual", "dresidual"), ("scale", "dscale"),
                        ("out_norm_w", "dout_norm_w")):
        if name in out and out[name].numel() > 0:
            setattr(p, field, out[name].data_ptr())
    workspace = _workspace(p, L_.ssm_block_norm_bwd_workspace_size(_byref(p)), workspace, dev, stream)
    call = Call(L_.ssm_block_norm_bwd, p, _on(dev, stream), out,
                (x, norm_w, z, residual, scale, out_norm_w, dout, dresidual, workspace))
    return call if prepare else call.run()
