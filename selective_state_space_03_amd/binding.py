"""Thin Python binding of libssm_mi355x.so (the C ABI in include/ssm_mi355x.h).

Argument marshalling only: torch tensors are checked for device, dtype, shape
and contiguity, outputs and workspace are allocated with torch, and raw device
pointers plus the current HIP stream go through ctypes.  Every step of the
computation runs in the library's HIP kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# SSM_MI355X_LIB names another build of the same library (the host-sanitized
# one of build_sanitized.py, for the CPU-side checks)
LIB_PATH = os.environ.get("SSM_MI355X_LIB") or os.path.join(_HERE, "libssm_mi355x.so")

SSM_F32, SSM_BF16 = 0, 1
# time_split value of the blocked single-pass scan (SSM_SCAN_BLOCKED in the header)
SCAN_BLOCKED = -1
STATUS = {0: "SSM_OK", 1: "SSM_ERR_INVALID_ARG", 2: "SSM_ERR_UNSUPPORTED", 3: "SSM_ERR_WORKSPACE", 4: "SSM_ERR_HIP",
          5: "SSM_ERR_INTERNAL"}

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_f32 = ctypes.c_float


class ScanParams(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32), ("batch", _i32), ("seqlen", _i32), ("dim", _i32), ("d_state", _i32),
        ("conv_k", _i32), ("x", _vp), ("x_dtype", _i32), ("conv_w", _vp), ("conv_b", _vp),
        ("conv_cache_in", _vp), ("conv_cache_out", _vp), ("dt", _vp), ("dt_dtype", _i32), ("dt_rank1", _i32),
        ("dt_w", _vp), ("dt_bias", _vp), ("dt_softplus", _i32), ("dt_min", _f32), ("dt_max", _f32),
        ("A", _vp), ("B", _vp), ("C", _vp), ("bc_dtype", _i32), ("D", _vp), ("z", _vp), ("z_dtype", _i32),
        ("ssm_state_in", _vp), ("ssm_state_out", _vp), ("y", _vp), ("y_dtype", _i32), ("time_split", _i32),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
        ("discretization", _i32),
    ]


class DecodeParams(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32), ("batch", _i32), ("dim", _i32), ("d_state", _i32), ("conv_k", _i32),
        ("x", _vp), ("x_dtype", _i32), ("conv_w", _vp), ("conv_b", _vp), ("conv_cache", _vp),
        ("dt", _vp), ("dt_dtype", _i32), ("dt_rank1", _i32), ("dt_w", _vp), ("dt_bias", _vp),
        ("dt_softplus", _i32), ("dt_min", _f32), ("dt_max", _f32), ("A", _vp), ("B", _vp), ("C", _vp),
        ("bc_dtype", _i32), ("D", _vp), ("z", _vp), ("z_dtype", _i32), ("ssm_state", _vp), ("y", _vp),
        ("y_dtype", _i32),
        ("discretization", _i32),
    ]


class ChunkParams(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32), ("batch", _i32), ("seqlen", _i32), ("nheads", _i32), ("headdim", _i32),
        ("ngroups", _i32), ("d_state", _i32), ("chunk_size", _i32), ("x", _vp), ("x_dtype", _i32),
        ("dt", _vp), ("dt_bias", _vp), ("dt_softplus", _i32), ("dt_min", _f32), ("dt_max", _f32),
        ("A", _vp), ("B", _vp), ("C", _vp), ("bc_dtype", _i32), ("D", _vp), ("d_per_channel", _i32),
        ("state_in", _vp), ("state_out", _vp), ("out", _vp), ("out_dtype", _i32),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t), ("z", _vp), ("z_dtype", _i32),
        ("segments", _i32),
    ]


class ChunkDecodeParams(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32), ("batch", _i32), ("nheads", _i32), ("headdim", _i32), ("ngroups", _i32),
        ("d_state", _i32), ("x", _vp), ("x_dtype", _i32), ("dt", _vp), ("dt_bias", _vp), ("dt_softplus", _i32),
        ("dt_min", _f32), ("dt_max", _f32), ("A", _vp), ("B", _vp), ("C", _vp), ("bc_dtype", _i32),
        ("D", _vp), ("d_per_channel", _i32), ("z", _vp), ("z_dtype", _i32), ("state", _vp), ("out", _vp),
        ("out_dtype", _i32),
    ]


class LinearParams(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32), ("rows", _i32), ("in_features", _i32), ("out_features", _i32),
        ("x", _vp), ("x_dtype", _i32), ("weight", _vp), ("out", _vp), ("out_dtype", _i32),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
    ]


class LayerParams(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32), ("batch", _i32), ("seqlen", _i32), ("d_model", _i32), ("dim", _i32),
        ("d_state", _i32), ("conv_k", _i32), ("hidden", _vp), ("hidden_dtype", _i32), ("w_in", _vp),
        ("conv_w", _vp), ("conv_b", _vp), ("w_x", _vp), ("dt_w", _vp), ("dt_bias", _vp), ("dt_softplus", _i32),
        ("dt_min", _f32), ("dt_max", _f32), ("A", _vp), ("D", _vp), ("w_out", _vp), ("conv_cache_in", _vp),
        ("conv_cache_out", _vp), ("ssm_state_in", _vp), ("ssm_state_out", _vp), ("out", _vp), ("out_dtype", _i32),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
    ]


class ScanBwdParams(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32), ("batch", _i32), ("seqlen", _i32), ("dim", _i32), ("d_state", _i32),
        ("conv_k", _i32), ("x", _vp), ("x_dtype", _i32), ("conv_w", _vp), ("conv_b", _vp), ("conv_cache_in", _vp),
        ("dt", _vp), ("dt_dtype", _i32), ("dt_rank1", _i32), ("dt_w", _vp), ("dt_bias", _vp), ("dt_softplus", _i32),
        ("dt_min", _f32), ("dt_max", _f32), ("A", _vp), ("B", _vp), ("C", _vp), ("bc_dtype", _i32), ("D", _vp),
        ("z", _vp), ("z_dtype", _i32), ("ssm_state_in", _vp), ("dy", _vp), ("dy_dtype", _i32), ("dstate_out", _vp),
        ("dx", _vp), ("dz", _vp), ("ddt", _vp), ("ddt_w", _vp), ("ddt_bias", _vp), ("dA", _vp), ("dB", _vp),
        ("dC", _vp), ("dD", _vp), ("dconv_w", _vp), ("dconv_b", _vp), ("dconv_cache", _vp), ("dstate_in", _vp),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
    ]


_i64 = ctypes.c_int64
_DELTA_HEAD = [
    ("struct_size", ctypes.c_uint32), ("batch", _i32), ("seqlen", _i32), ("num_seqs", _i32), ("nkheads", _i32),
    ("nheads", _i32), ("d_key", _i32), ("d_value", _i32), ("q", _vp), ("k", _vp), ("v", _vp), ("x_dtype", _i32),
    ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64), ("g", _vp), ("beta", _vp), ("scale", _f32),
    ("qk_norm", _i32), ("eps", _f32), ("cu_seqlens", _vp), ("state_in", _vp),
]


class DeltaChunkParams(ctypes.Structure):
    _fields_ = _DELTA_HEAD + [
        ("state_out", _vp), ("o", _vp), ("o_dtype", _i32), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
    ]


class DeltaChunkBwdParams(ctypes.Structure):
    _fields_ = _DELTA_HEAD + [
        ("dout", _vp), ("dstate_out", _vp), ("dq", _vp), ("dk", _vp), ("dv", _vp), ("grad_dtype", _i32), ("dg", _vp),
        ("dbeta", _vp), ("dstate_in", _vp), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
    ]


class DeltaDecodeParams(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32), ("batch", _i32), ("nkheads", _i32), ("nheads", _i32), ("d_key", _i32),
        ("d_value", _i32), ("q", _vp), ("k", _vp), ("v", _vp), ("x_dtype", _i32), ("q_stride", _i64),
        ("k_stride", _i64), ("v_stride", _i64), ("g", _vp), ("beta", _vp), ("scale", _f32), ("qk_norm", _i32),
        ("eps", _f32), ("state", _vp), ("o", _vp), ("o_dtype", _i32),
    ]


class BlockNormParams(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32), ("rows", _i64), ("width", _i32), ("group_size", _i32), ("x", _vp),
        ("x_dtype", _i32), ("x_stride", _i64), ("z", _vp), ("z_stride", _i64), ("gate_first", _i32), ("norm_w", _vp),
        ("norm_w_len", _i32), ("residual", _vp), ("res_dtype", _i32), ("scale", _vp), ("residual_out", _vp),
        ("out_norm_w", _vp), ("out", _vp), ("out_dtype", _i32), ("eps", _f32),
    ]


class BlockNormBwdParams(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32), ("rows", _i64), ("width", _i32), ("group_size", _i32), ("x", _vp),
        ("x_dtype", _i32), ("x_stride", _i64), ("z", _vp), ("z_stride", _i64), ("gate_first", _i32), ("norm_w", _vp),
        ("norm_w_len", _i32), ("residual", _vp), ("res_dtype", _i32), ("scale", _vp), ("out_norm_w", _vp),
        ("eps", _f32), ("dout", _vp), ("dout_dtype", _i32), ("dresidual_out", _vp), ("dres_dtype", _i32), ("dx", _vp),
        ("dz", _vp), ("grad_dtype", _i32), ("dresidual", _vp), ("dnorm_w", _vp), ("dscale", _vp),
        ("dout_norm_w", _vp), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
    ]


# entry points of the gated delta rule and the block norm: (name, params, has a workspace size)
_DELTA_ENTRIES = [
    ("ssm_delta_chunk_fwd", "ssm_delta_chunk", DeltaChunkParams, True),
    ("ssm_delta_chunk_bwd", "ssm_delta_chunk_bwd", DeltaChunkBwdParams, True),
    ("ssm_delta_decode_step", "ssm_delta_decode", DeltaDecodeParams, False),
    ("ssm_block_norm_fwd", "ssm_block_norm", BlockNormParams, False),
    ("ssm_block_norm_bwd", "ssm_block_norm_bwd", BlockNormBwdParams, True),
]

EXPORTED = [
    "ssm_scan_fwd", "ssm_scan_workspace_size", "ssm_scan_check", "ssm_scan_fwd_noalloc",
    "ssm_decode_step", "ssm_decode_check",
    "ssm_chunk_scan_fwd", "ssm_chunk_scan_workspace_size", "ssm_chunk_scan_check",
    "ssm_chunk_decode_step", "ssm_chunk_decode_check",
    "ssm_linear_fwd", "ssm_linear_workspace_size", "ssm_linear_check",
    "ssm_layer_fwd", "ssm_layer_workspace_size", "ssm_layer_check",
    "ssm_scan_bwd", "ssm_scan_bwd_workspace_size", "ssm_scan_bwd_check",
    "ssm_delta_chunk_fwd", "ssm_delta_chunk_workspace_size", "ssm_delta_chunk_check",
    "ssm_delta_chunk_bwd", "ssm_delta_chunk_bwd_workspace_size", "ssm_delta_chunk_bwd_check",
    "ssm_delta_decode_step", "ssm_delta_decode_check",
    "ssm_block_norm_fwd", "ssm_block_norm_check",
    "ssm_block_norm_bwd", "ssm_block_norm_bwd_workspace_size", "ssm_block_norm_bwd_check",
    "ssm_status_string", "ssm_last_error", "ssm_abi_version", "ssm_params_sizeof", "ssm_set_timing_events",
    "ssm_debug_checks", "ssm_debug_check_scan", "ssm_debug_check_chunk", "ssm_debug_check_scan_bwd",
]

_lib = None


def lib() -> ctypes.CDLL:
    """Load the HIP library (fails loudly when it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"HIP library not built: {LIB_PATH} is missing (build it with selective_state_space_03_amd.build.build())")
    _lib = load(LIB_PATH)
    return _lib


def load(path) -> ctypes.CDLL:
    """Load a build of the library at path (the regular one, or its SSM_DEBUG
    twin) with the argument types of every entry point declared."""
    L = ctypes.CDLL(path)
    L.ssm_scan_fwd.argtypes = [ctypes.POINTER(ScanParams), _vp]
    L.ssm_scan_fwd.restype = _i32
    L.ssm_scan_check.argtypes = [ctypes.POINTER(ScanParams)]
    L.ssm_scan_check.restype = _i32
    L.ssm_scan_workspace_size.argtypes = [ctypes.POINTER(ScanParams)]
    L.ssm_scan_workspace_size.restype = ctypes.c_size_t
    L.ssm_scan_fwd_noalloc.argtypes = [ctypes.POINTER(ScanParams), _vp]
    L.ssm_scan_fwd_noalloc.restype = _i32
    L.ssm_decode_step.argtypes = [ctypes.POINTER(DecodeParams), _vp]
    L.ssm_decode_step.restype = _i32
    L.ssm_decode_check.argtypes = [ctypes.POINTER(DecodeParams)]
    L.ssm_decode_check.restype = _i32
    L.ssm_chunk_scan_fwd.argtypes = [ctypes.POINTER(ChunkParams), _vp]
    L.ssm_chunk_scan_fwd.restype = _i32
    L.ssm_chunk_scan_check.argtypes = [ctypes.POINTER(ChunkParams)]
    L.ssm_chunk_scan_check.restype = _i32
    L.ssm_chunk_scan_workspace_size.argtypes = [ctypes.POINTER(ChunkParams)]
    L.ssm_chunk_scan_workspace_size.restype = ctypes.c_size_t
    L.ssm_chunk_decode_step.argtypes = [ctypes.POINTER(ChunkDecodeParams), _vp]
    L.ssm_chunk_decode_step.restype = _i32
    L.ssm_chunk_decode_check.argtypes = [ctypes.POINTER(ChunkDecodeParams)]
    L.ssm_chunk_decode_check.restype = _i32
    L.ssm_linear_fwd.argtypes = [ctypes.POINTER(LinearParams), _vp]
    L.ssm_linear_fwd.restype = _i32
    L.ssm_linear_workspace_size.argtypes = [ctypes.POINTER(LinearParams)]
    L.ssm_linear_workspace_size.restype = ctypes.c_size_t
    L.ssm_linear_check.argtypes = [ctypes.POINTER(LinearParams)]
    L.ssm_linear_check.restype = _i32
    L.ssm_layer_fwd.argtypes = [ctypes.POINTER(LayerParams), _vp]
    L.ssm_layer_fwd.restype = _i32
    L.ssm_layer_workspace_size.argtypes = [ctypes.POINTER(LayerParams)]
    L.ssm_layer_workspace_size.restype = ctypes.c_size_t
    L.ssm_layer_check.argtypes = [ctypes.POINTER(LayerParams)]
    L.ssm_layer_check.restype = _i32
    L.ssm_scan_bwd.argtypes = [ctypes.POINTER(ScanBwdParams), _vp]
    L.ssm_scan_bwd.restype = _i32
    L.ssm_scan_bwd_workspace_size.argtypes = [ctypes.POINTER(ScanBwdParams)]
    L.ssm_scan_bwd_workspace_size.restype = ctypes.c_size_t
    L.ssm_scan_bwd_check.argtypes = [ctypes.POINTER(ScanBwdParams)]
    L.ssm_scan_bwd_check.restype = _i32
    for run, base, st, sized in _DELTA_ENTRIES:
        ptr = ctypes.POINTER(st)
        getattr(L, run).argtypes, getattr(L, run).restype = [ptr, _vp], _i32
        getattr(L, base + "_check").argtypes, getattr(L, base + "_check").restype = [ptr], _i32
        if sized:
            size = getattr(L, base + "_workspace_size")
            size.argtypes, size.restype = [ptr], ctypes.c_size_t
    L.ssm_status_string.argtypes = [_i32]
    L.ssm_status_string.restype = ctypes.c_char_p
    L.ssm_last_error.argtypes = []
    L.ssm_last_error.restype = ctypes.c_char_p
    L.ssm_abi_version.argtypes = []
    L.ssm_abi_version.restype = _i32
    L.ssm_params_sizeof.argtypes = [_i32]
    L.ssm_params_sizeof.restype = ctypes.c_size_t
    L.ssm_set_timing_events.argtypes = [_vp, _vp]
    L.ssm_set_timing_events.restype = None
    L.ssm_debug_checks.argtypes = []
    L.ssm_debug_checks.restype = ctypes.c_long
    L.ssm_debug_check_scan.argtypes = [ctypes.POINTER(ScanParams)]
    L.ssm_debug_check_scan.restype = _i32
    L.ssm_debug_check_chunk.argtypes = [ctypes.POINTER(ChunkParams)]
    L.ssm_debug_check_chunk.restype = _i32
    L.ssm_debug_check_scan_bwd.argtypes = [ctypes.POINTER(ScanBwdParams)]
    L.ssm_debug_check_scan_bwd.restype = _i32
    for i, st in enumerate((ScanParams, DecodeParams, ChunkParams, ChunkDecodeParams, LinearParams, LayerParams,
                            ScanBwdParams)):
        if L.ssm_params_sizeof(i) != ctypes.sizeof(st):
            raise RuntimeError(f"ctypes mirror of params struct {i} does not match the library")
    for i, (_, _, st, _) in enumerate(_DELTA_ENTRIES):
        if L.ssm_params_sizeof(8 + i) != ctypes.sizeof(st):
            raise RuntimeError(f"ctypes mirror of params struct {8 + i} does not match the library")
    return L


class SsmError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{STATUS.get(status, status)}: {detail}")
        self.status = status


def _raise(status: int):
    if status != 0:
        raise SsmError(status, lib().ssm_last_error().decode())


_DT = {torch.float32: SSM_F32, torch.bfloat16: SSM_BF16}


def _code(t: torch.Tensor, name: str) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"{name}: dtype {t.dtype} not supported (float32 or bfloat16)")
    return _DT[t.dtype]


def _ptr(t, name, shape=None, dtype=None, device=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    return t.data_ptr() if t.numel() > 0 else None


def _discretization(name):
    codes = {"euler": 0, "zoh": 1}
    if name not in codes:
        raise ValueError(f"discretization must be one of {sorted(codes)}, got {name!r}")
    return codes[name]


def _stream(device, stream):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _empty(shape, dtype, device, stream):
    """torch.empty for a buffer the library writes on `stream`.  torch's caching
    allocator ties a block to the stream current at allocation; when the call
    runs on another stream the block is also recorded on that one, so it is not
    handed out again before the work queued there has finished with it."""
    t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None and stream != torch.cuda.current_stream(device):
        t.record_stream(stream)
    return t


class Call:
    """One marshalled entry-point call.  run() enqueues it (again) on the same
    stream with the same buffers and returns the output tensor; the tensors
    the call reads and writes are kept alive here."""

    def __init__(self, fn, params, stream, out, keep):
        self._fn, self._p, self._stream, self.out, self._keep = fn, params, stream, out, keep

    def run(self):
        _raise(self._fn(ctypes.byref(self._p), self._stream))
        return self.out


def set_timing_events(start=None, stop=None):
    """Record two torch.cuda.Event objects around the main kernel of the
    following entry-point calls on this thread (None, None: stop recording)."""
    if (start is None) != (stop is None):
        raise ValueError("give both events or neither")
    if start is None:
        lib().ssm_set_timing_events(None, None)
        return
    for ev in (start, stop):
        if not ev.cuda_event:  # torch creates the HIP event at its first record
            ev.record()
    lib().ssm_set_timing_events(ctypes.c_void_p(start.cuda_event), ctypes.c_void_p(stop.cuda_event))


def _bound(v, default):
    return float(default if v is None else v)


def scan_fwd(x, A, B, C, dt, *, D=None, z=None, conv_w=None, conv_b=None, conv_cache_in=None,
             conv_cache_out=None, dt_rank1=False, dt_w=None, dt_bias=None, dt_softplus=True,
             dt_min=None, dt_max=None, ssm_state_in=None, ssm_state_out=None, y=None,
             y_dtype=None, time_split=0, workspace=None, discretization="euler", stream=None, prepare=False):
    """Full-sequence selective scan (ssm_scan_fwd); discretization "euler" (dt B u) or "zoh"
    (((e^{dt A} - 1) / A) B u).  Returns y (batch, L, E), or
    with prepare=True a Call that enqueues this same call again on each run()."""
    return _scan(False, x, A, B, C, dt, D=D, z=z, conv_w=conv_w, conv_b=conv_b, conv_cache_in=conv_cache_in,
                 conv_cache_out=conv_cache_out, dt_rank1=dt_rank1, dt_w=dt_w, dt_bias=dt_bias,
                 dt_softplus=dt_softplus, dt_min=dt_min, dt_max=dt_max, ssm_state_in=ssm_state_in,
                 ssm_state_out=ssm_state_out, y=y, y_dtype=y_dtype, time_split=time_split, workspace=workspace,
                 discretization=discretization, stream=stream, prepare=prepare)


def scan_fwd_noalloc(x, A, B, C, dt, *, D=None, z=None, conv_w=None, conv_b=None, conv_cache_in=None,
                     conv_cache_out=None, dt_rank1=False, dt_w=None, dt_bias=None, dt_softplus=True,
                     dt_min=None, dt_max=None, ssm_state_in=None, ssm_state_out=None, y=None,
                     y_dtype=None, time_split=0, discretization="euler", stream=None, prepare=False):
    """ssm_scan_fwd_noalloc: scan_fwd with the workspace taken from the library's
    own device scratch (no workspace argument; calls on one GPU must not overlap).
    Returns y, or with prepare=True a Call."""
    return _scan(True, x, A, B, C, dt, D=D, z=z, conv_w=conv_w, conv_b=conv_b, conv_cache_in=conv_cache_in,
                 conv_cache_out=conv_cache_out, dt_rank1=dt_rank1, dt_w=dt_w, dt_bias=dt_bias,
                 dt_softplus=dt_softplus, dt_min=dt_min, dt_max=dt_max, ssm_state_in=ssm_state_in,
                 ssm_state_out=ssm_state_out, y=y, y_dtype=y_dtype, time_split=time_split, workspace=None,
                 discretization=discretization, stream=stream, prepare=prepare)


def _scan(noalloc, x, A, B, C, dt, *, D, z, conv_w, conv_b, conv_cache_in, conv_cache_out, dt_rank1, dt_w, dt_bias,
          dt_softplus, dt_min, dt_max, ssm_state_in, ssm_state_out, y, y_dtype, time_split, workspace,
          discretization, stream, prepare):
    L_ = lib()
    batch, seqlen, dim = x.shape
    dev = x.device
    d_state = A.shape[1]
    if y is None:
        y = _empty((batch, seqlen, dim), y_dtype or x.dtype, dev, stream)
    f32 = torch.float32
    p = ScanParams()
    p.struct_size = ctypes.sizeof(ScanParams)
    p.batch, p.seqlen, p.dim, p.d_state = batch, seqlen, dim, d_state
    p.conv_k = conv_w.shape[1] if conv_w is not None else 0
    p.x = _ptr(x, "x", (batch, seqlen, dim), device=dev)
    p.x_dtype = _code(x, "x")
    p.conv_w = _ptr(conv_w, "conv_w", (dim, p.conv_k) if conv_w is not None else None, f32, dev)
    p.conv_b = _ptr(conv_b, "conv_b", (dim,), f32, dev)
    p.conv_cache_in = _ptr(conv_cache_in, "conv_cache_in", (batch, dim, 3), f32, dev)
    p.conv_cache_out = _ptr(conv_cache_out, "conv_cache_out", (batch, dim, 3), f32, dev)
    p.dt_rank1 = 1 if dt_rank1 else 0
    p.dt = _ptr(dt, "dt", (batch, seqlen) if dt_rank1 else (batch, seqlen, dim), device=dev)
    p.dt_dtype = _code(dt, "dt")
    p.dt_w = _ptr(dt_w, "dt_w", (dim,), f32, dev)
    p.dt_bias = _ptr(dt_bias, "dt_bias", (dim,), f32, dev)
    p.dt_softplus = 1 if dt_softplus else 0
    p.dt_min = _bound(dt_min, -math.inf)
    p.dt_max = _bound(dt_max, math.inf)
    p.A = _ptr(A, "A", (dim, d_state), f32, dev)
    p.B = _ptr(B, "B", (batch, seqlen, d_state), device=dev)
    p.C = _ptr(C, "C", (batch, seqlen, d_state), B.dtype, dev)
    p.bc_dtype = _code(B, "B")
    p.D = _ptr(D, "D", (dim,), f32, dev)
    p.z = _ptr(z, "z", (batch, seqlen, dim), device=dev)
    p.z_dtype = _code(z, "z") if z is not None else 0
    p.ssm_state_in = _ptr(ssm_state_in, "ssm_state_in", (batch, dim, d_state), f32, dev)
    p.ssm_state_out = _ptr(ssm_state_out, "ssm_state_out", (batch, dim, d_state), f32, dev)
    p.y = _ptr(y, "y", (batch, seqlen, dim), device=dev)
    p.y_dtype = _code(y, "y")
    p.time_split = int(time_split)
    p.discretization = _discretization(discretization)
    if not noalloc:
        need = L_.ssm_scan_workspace_size(ctypes.byref(p))
        if workspace is None and need > 0:
            workspace = _empty(need, torch.uint8, dev, stream)
        p.workspace = _ptr(workspace, "workspace", device=dev)
        p.workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    fn = L_.ssm_scan_fwd_noalloc if noalloc else L_.ssm_scan_fwd
    call = Call(fn, p, _stream(dev, stream), y, (x, A, B, C, dt, D, z, conv_w, conv_b, conv_cache_in,
                                                conv_cache_out, dt_w, dt_bias, ssm_state_in, ssm_state_out, workspace))
    return call if prepare else call.run()


def decode_step(x, A, B, C, dt, ssm_state, *, conv_cache=None, D=None, z=None, conv_w=None, conv_b=None,
                dt_rank1=False, dt_w=None, dt_bias=None, dt_softplus=True, dt_min=None, dt_max=None,
                y=None, y_dtype=None, discretization="euler", stream=None, prepare=False):
    """One decode step (ssm_decode_step; discretization as in scan_fwd): updates ssm_state and conv_cache in place, returns y (batch, E)
    (with prepare=True, a Call that enqueues this same step again on each run())."""
    L_ = lib()
    batch, dim = x.shape
    dev = x.device
    d_state = A.shape[1]
    if y is None:
        y = _empty((batch, dim), y_dtype or x.dtype, dev, stream)
    f32 = torch.float32
    p = DecodeParams()
    p.struct_size = ctypes.sizeof(DecodeParams)
    p.batch, p.dim, p.d_state = batch, dim, d_state
    p.conv_k = conv_w.shape[1] if conv_w is not None else 0
    p.x = _ptr(x, "x", (batch, dim), device=dev)
    p.x_dtype = _code(x, "x")
    p.conv_w = _ptr(conv_w, "conv_w", (dim, p.conv_k) if conv_w is not None else None, f32, dev)
    p.conv_b = _ptr(conv_b, "conv_b", (dim,), f32, dev)
    p.conv_cache = _ptr(conv_cache, "conv_cache", (batch, dim, 3), f32, dev)
    p.dt_rank1 = 1 if dt_rank1 else 0
    p.dt = _ptr(dt, "dt", (batch,) if dt_rank1 else (batch, dim), device=dev)
    p.dt_dtype = _code(dt, "dt")
    p.dt_w = _ptr(dt_w, "dt_w", (dim,), f32, dev)
    p.dt_bias = _ptr(dt_bias, "dt_bias", (dim,), f32, dev)
    p.dt_softplus = 1 if dt_softplus else 0
    p.dt_min = _bound(dt_min, -math.inf)
    p.dt_max = _bound(dt_max, math.inf)
    p.A = _ptr(A, "A", (dim, d_state), f32, dev)
    p.B = _ptr(B, "B", (batch, d_state), device=dev)
    p.C = _ptr(C, "C", (batch, d_state), B.dtype, dev)
    p.bc_dtype = _code(B, "B")
    p.D = _ptr(D, "D", (dim,), f32, dev)
    p.z = _ptr(z, "z", (batch, dim), device=dev)
    p.z_dtype = _code(z, "z") if z is not None else 0
    p.ssm_state = _ptr(ssm_state, "ssm_state", (batch, dim, d_state), f32, dev)
    p.y = _ptr(y, "y", (batch, dim), device=dev)
    p.y_dtype = _code(y, "y")
    p.discretization = _discretization(discretization)
    call = Call(L_.ssm_decode_step, p, _stream(dev, stream), y, (x, A, B, C, dt, ssm_state, conv_cache, D, z,
                                                                conv_w, conv_b, dt_w, dt_bias))
    return call if prepare else call.run()


def chunk_scan_fwd(x, dt, A, B, C, *, chunk_size=128, D=None, dt_bias=None, dt_softplus=True, dt_min=None,
                   dt_max=None, state_in=None, state_out=None, out=None, out_dtype=None, z=None, workspace=None,
                   segments=0, stream=None, prepare=False):
    """Multi-head chunked scan (ssm_chunk_scan_fwd).  Returns out (batch, L, H, P), or
    with prepare=True a Call that enqueues this same call again on each run().
    segments: 0 lets the library cut the sequences; n > 0 forces n segments."""
    L_ = lib()
    batch, seqlen, nheads, headdim = x.shape
    ngroups, d_state = B.shape[2], B.shape[3]
    dev = x.device
    if out is None:
        out = _empty((batch, seqlen, nheads, headdim), out_dtype or x.dtype, dev, stream)
    f32 = torch.float32
    p = ChunkParams()
    p.struct_size = ctypes.sizeof(ChunkParams)
    p.batch, p.seqlen, p.nheads, p.headdim = batch, seqlen, nheads, headdim
    p.ngroups, p.d_state, p.chunk_size = ngroups, d_state, int(chunk_size)
    p.x = _ptr(x, "x", (batch, seqlen, nheads, headdim), device=dev)
    p.x_dtype = _code(x, "x")
    p.dt = _ptr(dt, "dt", (batch, seqlen, nheads), f32, dev)
    p.dt_bias = _ptr(dt_bias, "dt_bias", (nheads,), f32, dev)
    p.dt_softplus = 1 if dt_softplus else 0
    p.dt_min = _bound(dt_min, -math.inf)
    p.dt_max = _bound(dt_max, math.inf)
    p.A = _ptr(A, "A", (nheads,), f32, dev)
    p.B = _ptr(B, "B", (batch, seqlen, ngroups, d_state), device=dev)
    p.C = _ptr(C, "C", (batch, seqlen, ngroups, d_state), B.dtype, dev)
    p.bc_dtype = _code(B, "B")
    if D is not None:
        p.d_per_channel = 1 if D.dim() == 2 else 0
        p.D = _ptr(D, "D", (nheads, headdim) if D.dim() == 2 else (nheads,), f32, dev)
    p.state_in = _ptr(state_in, "state_in", (batch, nheads, headdim, d_state), f32, dev)
    p.state_out = _ptr(state_out, "state_out", (batch, nheads, headdim, d_state), f32, dev)
    p.out = _ptr(out, "out", (batch, seqlen, nheads, headdim), device=dev)
    p.out_dtype = _code(out, "out")
    p.z = _ptr(z, "z", (batch, seqlen, nheads, headdim), device=dev)
    p.z_dtype = _code(z, "z") if z is not None else 0
    p.segments = int(segments)
    need = L_.ssm_chunk_scan_workspace_size(ctypes.byref(p))
    if workspace is None and need > 0:
        workspace = _empty(need, torch.uint8, dev, stream)
    p.workspace = _ptr(workspace, "workspace", device=dev)
    p.workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    call = Call(L_.ssm_chunk_scan_fwd, p, _stream(dev, stream), out, (x, dt, A, B, C, D, dt_bias, state_in,
                                                                     state_out, workspace, z))
    return call if prepare else call.run()


def chunk_decode_step(x, dt, A, B, C, state, *, D=None, dt_bias=None, dt_softplus=True, dt_min=None, dt_max=None,
                      z=None, out=None, out_dtype=None, stream=None, prepare=False):
    """One decode step of the multi-head scan (ssm_chunk_decode_step): x (batch, H, P), dt (batch, H),
    B/C (batch, G, N), state (batch, H, P, N) f32 updated in place.  Returns out (batch, H, P), or
    with prepare=True a Call that enqueues this same step again on each run()."""
    L_ = lib()
    batch, nheads, headdim = x.shape
    ngroups, d_state = B.shape[1], B.shape[2]
    dev = x.device
    if out is None:
        out = _empty((batch, nheads, headdim), out_dtype or x.dtype, dev, stream)
    f32 = torch.float32
    p = ChunkDecodeParams()
    p.struct_size = ctypes.sizeof(ChunkDecodeParams)
    p.batch, p.nheads, p.headdim, p.ngroups, p.d_state = batch, nheads, headdim, ngroups, d_state
    p.x = _ptr(x, "x", (batch, nheads, headdim), device=dev)
    p.x_dtype = _code(x, "x")
    p.dt = _ptr(dt, "dt", (batch, nheads), f32, dev)
    p.dt_bias = _ptr(dt_bias, "dt_bias", (nheads,), f32, dev)
    p.dt_softplus = 1 if dt_softplus else 0
    p.dt_min = _bound(dt_min, -math.inf)
    p.dt_max = _bound(dt_max, math.inf)
    p.A = _ptr(A, "A", (nheads,), f32, dev)
    p.B = _ptr(B, "B", (batch, ngroups, d_state), device=dev)
    p.C = _ptr(C, "C", (batch, ngroups, d_state), B.dtype, dev)
    p.bc_dtype = _code(B, "B")
    if D is not None:
        p.d_per_channel = 1 if D.dim() == 2 else 0
        p.D = _ptr(D, "D", (nheads, headdim) if D.dim() == 2 else (nheads,), f32, dev)
    p.z = _ptr(z, "z", (batch, nheads, headdim), device=dev)
    p.z_dtype = _code(z, "z") if z is not None else 0
    p.state = _ptr(state, "state", (batch, nheads, headdim, d_state), f32, dev)
    p.out = _ptr(out, "out", (batch, nheads, headdim), device=dev)
    p.out_dtype = _code(out, "out")
    call = Call(L_.ssm_chunk_decode_step, p, _stream(dev, stream), out, (x, dt, A, B, C, state, D, dt_bias, z))
    return call if prepare else call.run()


def linear_fwd(x, weight, *, out=None, out_dtype=None, workspace=None, stream=None, prepare=False):
    """A projection without bias (ssm_linear_fwd): out[..., o] = sum_i x[..., i] weight[o, i], with x
    (..., in) bf16 or f32 and weight (out, in) bf16.  A workspace of ssm_linear_workspace_size() bytes
    is allocated when none is given (an f32 x needs one; workspace=False passes none).  Returns out (..., out), or
    with prepare=True a Call that enqueues this same call again on each run()."""
    L_ = lib()
    n_out, n_in = weight.shape
    lead = tuple(x.shape[:-1])
    rows = math.prod(lead)
    dev = x.device
    if out is None:
        out = _empty(lead + (n_out,), out_dtype or x.dtype, dev, stream)
    p = LinearParams()
    p.struct_size = ctypes.sizeof(LinearParams)
    p.rows, p.in_features, p.out_features = rows, n_in, n_out
    p.x = _ptr(x, "x", lead + (n_in,), device=dev)
    p.x_dtype = _code(x, "x")
    p.weight = _ptr(weight, "weight", (n_out, n_in), torch.bfloat16, dev)
    p.out = _ptr(out, "out", lead + (n_out,), device=dev)
    p.out_dtype = _code(out, "out")
    if workspace is None:
        need = L_.ssm_linear_workspace_size(ctypes.byref(p))
        workspace = _empty(need, torch.uint8, dev, stream) if need > 0 else False
    if workspace is not False:
        p.workspace = _ptr(workspace, "workspace", device=dev)
        p.workspace_bytes = workspace.numel() * workspace.element_size()
    call = Call(L_.ssm_linear_fwd, p, _stream(dev, stream), out, (x, weight, workspace))
    return call if prepare else call.run()


def layer_fwd(hidden, w_in, conv_w, w_x, dt_w, A, w_out, *, dt_bias=None, D=None, conv_b=None, conv_cache_in=None,
              conv_cache_out=None, ssm_state_in=None, ssm_state_out=None, dt_softplus=True, dt_min=None, dt_max=None,
              out=None, out_dtype=None, workspace=None, stream=None, prepare=False):
    """The whole layer forward (ssm_layer_fwd): in_proj, conv + SiLU, x_proj, scan with the gate, out_proj.
    hidden (batch, L, D); w_in (2E, D), w_x (2N+1, E), w_out (D, E) bf16; conv_w (E, 4), dt_w (E), A (E, N)
    fp32.  Returns out (batch, L, D), or with prepare=True a Call that enqueues this same call again."""
    L_ = lib()
    batch, seqlen, d_model = hidden.shape
    dim, d_state = A.shape
    dev = hidden.device
    if out is None:
        out = _empty((batch, seqlen, d_model), out_dtype or hidden.dtype, dev, stream)
    f32, bf = torch.float32, torch.bfloat16
    p = LayerParams()
    p.struct_size = ctypes.sizeof(LayerParams)
    p.batch, p.seqlen, p.d_model, p.dim, p.d_state = batch, seqlen, d_model, dim, d_state
    p.conv_k = conv_w.shape[1]
    p.hidden = _ptr(hidden, "hidden", (batch, seqlen, d_model), device=dev)
    p.hidden_dtype = _code(hidden, "hidden")
    p.w_in = _ptr(w_in, "w_in", (2 * dim, d_model), bf, dev)
    p.conv_w = _ptr(conv_w, "conv_w", (dim, p.conv_k), f32, dev)
    p.conv_b = _ptr(conv_b, "conv_b", (dim,), f32, dev)
    p.w_x = _ptr(w_x, "w_x", (2 * d_state + 1, dim), bf, dev)
    p.dt_w = _ptr(dt_w, "dt_w", (dim,), f32, dev)
    p.dt_bias = _ptr(dt_bias, "dt_bias", (dim,), f32, dev)
    p.dt_softplus = 1 if dt_softplus else 0
    p.dt_min = _bound(dt_min, -math.inf)
    p.dt_max = _bound(dt_max, math.inf)
    p.A = _ptr(A, "A", (dim, d_state), f32, dev)
    p.D = _ptr(D, "D", (dim,), f32, dev)
    p.w_out = _ptr(w_out, "w_out", (d_model, dim), bf, dev)
    kc = p.conv_k - 1
    p.conv_cache_in = _ptr(conv_cache_in, "conv_cache_in", (batch, dim, kc), f32, dev)
    p.conv_cache_out = _ptr(conv_cache_out, "conv_cache_out", (batch, dim, kc), f32, dev)
    p.ssm_state_in = _ptr(ssm_state_in, "ssm_state_in", (batch, dim, d_state), f32, dev)
    p.ssm_state_out = _ptr(ssm_state_out, "ssm_state_out", (batch, dim, d_state), f32, dev)
    p.out = _ptr(out, "out", (batch, seqlen, d_model), device=dev)
    p.out_dtype = _code(out, "out")
    need = L_.ssm_layer_workspace_size(ctypes.byref(p))
    if workspace is None and need > 0:
        workspace = _empty(need, torch.uint8, dev, stream)
    p.workspace = _ptr(workspace, "workspace", device=dev)
    p.workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    call = Call(L_.ssm_layer_fwd, p, _stream(dev, stream), out,
                (hidden, w_in, conv_w, conv_b, w_x, dt_w, dt_bias, A, D, w_out, conv_cache_in, conv_cache_out,
                 ssm_state_in, ssm_state_out, workspace))
    return call if prepare else call.run()


def scan_bwd(x, A, B, C, dt, dy, *, D=None, z=None, conv_w=None, conv_b=None, conv_cache_in=None, dt_rank1=False,
             dt_w=None, dt_bias=None, dt_softplus=True, dt_min=None, dt_max=None, ssm_state_in=None,
             dstate_out=None, workspace=None, stream=None, prepare=False):
    """Backward of scan_fwd (ssm_scan_bwd): the forward's inputs plus dy (and optionally the gradient on
    the final state).  Returns a dict of fp32 gradients named after the inputs (x, z, dt, dt_w, dt_bias,
    A, B, C, D, conv_w, conv_b, conv_cache, ssm_state), present for the inputs that were given, or with
    prepare=True a Call whose run() enqueues it again (its .out is that dict)."""
    L_ = lib()
    batch, seqlen, dim = x.shape
    d_state = A.shape[1]
    dev = x.device
    f32 = torch.float32
    p = ScanBwdParams()
    p.struct_size = ctypes.sizeof(ScanBwdParams)
    p.batch, p.seqlen, p.dim, p.d_state = batch, seqlen, dim, d_state
    p.conv_k = conv_w.shape[1] if conv_w is not None else 0
    p.x = _ptr(x, "x", (batch, seqlen, dim), device=dev)
    p.x_dtype = _code(x, "x")
    p.conv_w = _ptr(conv_w, "conv_w", (dim, p.conv_k) if conv_w is not None else None, f32, dev)
    p.conv_b = _ptr(conv_b, "conv_b", (dim,), f32, dev)
    p.conv_cache_in = _ptr(conv_cache_in, "conv_cache_in", (batch, dim, 3), f32, dev)
    p.dt_rank1 = 1 if dt_rank1 else 0
    p.dt = _ptr(dt, "dt", (batch, seqlen) if dt_rank1 else (batch, seqlen, dim), device=dev)
    p.dt_dtype = _code(dt, "dt")
    p.dt_w = _ptr(dt_w, "dt_w", (dim,), f32, dev)
    p.dt_bias = _ptr(dt_bias, "dt_bias", (dim,), f32, dev)
    p.dt_softplus = 1 if dt_softplus else 0
    p.dt_min = _bound(dt_min, -math.inf)
    p.dt_max = _bound(dt_max, math.inf)
    p.A = _ptr(A, "A", (dim, d_state), f32, dev)
    p.B = _ptr(B, "B", (batch, seqlen, d_state), device=dev)
    p.C = _ptr(C, "C", (batch, seqlen, d_state), B.dtype, dev)
    p.bc_dtype = _code(B, "B")
    p.D = _ptr(D, "D", (dim,), f32, dev)
    p.z = _ptr(z, "z", (batch, seqlen, dim), device=dev)
    p.z_dtype = _code(z, "z") if z is not None else 0
    p.ssm_state_in = _ptr(ssm_state_in, "ssm_state_in", (batch, dim, d_state), f32, dev)
    p.dy = _ptr(dy, "dy", (batch, seqlen, dim), device=dev)
    p.dy_dtype = _code(dy, "dy")
    p.dstate_out = _ptr(dstate_out, "dstate_out", (batch, dim, d_state), f32, dev)
    e = lambda *shape: _empty(shape, f32, dev, stream)  # noqa: E731
    g = {"x": e(batch, seqlen, dim), "A": e(dim, d_state), "B": e(batch, seqlen, d_state),
         "C": e(batch, seqlen, d_state), "dt": e(batch, seqlen) if dt_rank1 else e(batch, seqlen, dim)}
    if z is not None:
        g["z"] = e(batch, seqlen, dim)
    if dt_rank1:
        g["dt_w"] = e(dim)
    if dt_bias is not None:
        g["dt_bias"] = e(dim)
    if D is not None:
        g["D"] = e(dim)
    if conv_w is not None:
        g["conv_w"] = e(dim, p.conv_k)
        if conv_b is not None:
            g["conv_b"] = e(dim)
        if conv_cache_in is not None:
            g["conv_cache"] = e(batch, dim, 3)
    if ssm_state_in is not None:
        g["ssm_state"] = e(batch, dim, d_state)
    for key, field in (("x", "dx"), ("z", "dz"), ("dt", "ddt"), ("dt_w", "ddt_w"), ("dt_bias", "ddt_bias"),
                       ("A", "dA"), ("B", "dB"), ("C", "dC"), ("D", "dD"), ("conv_w", "dconv_w"),
                       ("conv_b", "dconv_b"), ("conv_cache", "dconv_cache"), ("ssm_state", "dstate_in")):
        if key in g:
            setattr(p, field, g[key].data_ptr() if g[key].numel() > 0 else None)
    need = L_.ssm_scan_bwd_workspace_size(ctypes.byref(p))
    if workspace is None and need > 0:
        workspace = _empty(need, torch.uint8, dev, stream)
    p.workspace = _ptr(workspace, "workspace", device=dev)
    p.workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    call = Call(L_.ssm_scan_bwd, p, _stream(dev, stream), g,
                (x, A, B, C, dt, dy, D, z, conv_w, conv_b, conv_cache_in, dt_w, dt_bias, ssm_state_in, dstate_out,
                 workspace))
    return call if prepare else call.run()
