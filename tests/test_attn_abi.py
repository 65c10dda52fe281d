"""Argument validation, workspace sizes and struct layouts of the window attention's entry points and its cache's on
the CPU: nothing here reaches a GPU (pointers are compared, never dereferenced)."""
import ctypes
import math
import os

import pytest

from selective_state_space_03_amd import binding as b


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(b.LIB_PATH):
        from selective_state_space_03_amd import build

        build.build()
    return b.lib()


def _addr(i):
    return 0x10000000000 + i * 0x100000000


def _fill(st, kw, defaults):
    p = st()
    p.struct_size = ctypes.sizeof(st)
    for k, v in {**defaults, **kw}.items():
        setattr(p, k, v)
    return p


_ATTN = dict(batch=2, seqlen=100, seqlen_k=120, num_seqs=2, nkheads=2, nheads=4, d_head=64, q=_addr(1), k=_addr(2), v=_addr(3),
             x_dtype=1, scale=0.125, window=50, sinks=4, lse=_addr(4), o=_addr(5), o_dtype=1, workspace=_addr(20),
             workspace_bytes=1 << 30)
_POOL = dict(k_cache=_addr(6), v_cache=_addr(7), cache_dtype=2, k_scale=_addr(8), v_scale=_addr(9), page_table=_addr(10),
             lens=_addr(11), table_rows=30, pages=100, page_size=16)


def _fwd(**kw):
    return _fill(b.AttnParams, kw, _ATTN)


def _bwd(**kw):
    return _fill(b.AttnBwdParams, kw, dict(_ATTN, dout=_addr(12), dq=_addr(13), dk=_addr(14), dv=_addr(15), grad_dtype=0))


def _write(**kw):
    return _fill(b.AttnCacheParams, kw, dict(_POOL, batch=2, seqlen=10, num_seqs=2, nkheads=2, d_head=64, k=_addr(2), v=_addr(3),
                                             x_dtype=1))


def _step(**kw):
    return _fill(b.AttnDecodeParams, kw, dict(_POOL, batch=2, nkheads=2, nheads=4, d_head=64, q=_addr(1), x_dtype=1, scale=0.125,
                                              window=0, sinks=0, o=_addr(5), o_dtype=1, workspace=_addr(20),
                                              workspace_bytes=1 << 30))


CHECKS = {_fwd: "ssm_attn", _bwd: "ssm_attn_bwd", _write: "ssm_attn_cache", _step: "ssm_attn_decode"}
RUNS = {_fwd: "ssm_attn_fwd", _bwd: "ssm_attn_bwd", _write: "ssm_attn_cache_write", _step: "ssm_attn_decode_step"}
NAMES = {b.AttnParams: "ssm_attn", b.AttnBwdParams: "ssm_attn_bwd", b.AttnCacheParams: "ssm_attn_cache",
         b.AttnDecodeParams: "ssm_attn_decode"}


def test_sizeof_and_valid_calls(L):
    for i, st in enumerate(NAMES):
        assert L.ssm_params_sizeof(13 + i) == ctypes.sizeof(st)
    assert L.ssm_params_sizeof(17) == 0
    for make, name in CHECKS.items():
        assert getattr(L, name + "_check")(ctypes.byref(make())) == 0, (name, L.ssm_last_error())
        assert L.ssm_last_error() == b""


_SEQ_BAD = [(dict(struct_size=8), 1), (dict(nheads=3), 1), (dict(nkheads=0), 1), (dict(d_head=129), 2), (dict(d_head=0), 1),
            (dict(nheads=1 << 17), 2), (dict(x_dtype=2), 1), (dict(x_dtype=7), 1), (dict(o_dtype=2), 1), (dict(scale=math.inf), 1),
            (dict(scale=math.nan), 1), (dict(scale=-0.5), 1), (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(batch=-1), 1),
            (dict(seqlen=-1), 1), (dict(seqlen_k=-1), 1), (dict(num_seqs=3), 1), (dict(cu_seqlens=_addr(16)), 1),
            (dict(cu_seqlens_k=_addr(16)), 1), (dict(cu_seqlens=_addr(16), batch=1), 1),
            (dict(cu_seqlens=_addr(16) + 2, batch=1, seqlen_k=100), 1), (dict(q_stride=255), 1), (dict(k_stride=127), 1),
            (dict(v_stride=1), 1), (dict(q_stride=1 << 41), 1), (dict(k_stride=1 << 40, batch=1 << 10, num_seqs=1 << 10, seqlen_k=1 << 20), 1),
            (dict(q=None), 1), (dict(v=None), 1), (dict(o=None), 1), (dict(q=_addr(1) + 1), 1), (dict(o=_addr(5) + 1), 1),
            (dict(lse=_addr(4) + 2), 1), (dict(batch=1 << 20, num_seqs=1 << 20, seqlen=1 << 20), 2),
            (dict(seqlen=(1 << 30) + 1), 2), (dict(seqlen_k=(1 << 30) + 1), 2)]
_POOL_BAD = [(dict(struct_size=8), 1), (dict(nkheads=0), 1), (dict(d_head=129), 2), (dict(x_dtype=2), 1), (dict(batch=-1), 1),
             (dict(table_rows=-1), 1), (dict(pages=-1), 1), (dict(page_size=0), 1), (dict(page_size=65537), 2),
             (dict(table_rows=1 << 30, page_size=2), 2), (dict(cache_dtype=3), 1), (dict(cache_dtype=1), 1),
             (dict(cache_dtype=0, k_scale=None, v_scale=None), 2), (dict(k_scale=None), 1), (dict(v_scale=None), 1),
             (dict(k_cache=None), 1), (dict(lens=None), 1), (dict(page_table=None), 1), (dict(k_scale=_addr(8) + 2), 1),
             (dict(lens=_addr(11) + 1), 1), (dict(page_table=_addr(10) + 2), 1),
             (dict(cache_dtype=1, k_cache=_addr(6) + 1, k_scale=None, v_scale=None), 1), (dict(pages=(1 << 31) - 1, page_size=65536, d_head=128, nkheads=1 << 15), 1)]
BAD = (
    [(_fwd, *c) for c in _SEQ_BAD] + [(_bwd, *c) for c in _SEQ_BAD] + [(_write, *c) for c in _POOL_BAD]
    + [(_step, *c) if "nkheads" not in c[0] or c[0]["nkheads"] == 0 else (_step, {**c[0], "nheads": c[0]["nkheads"]}, c[1])
       for c in _POOL_BAD]
    + [(_fwd, dict(o=_addr(2) + 64), 1), (_fwd, dict(lse=_addr(5) + 4), 1), (_fwd, dict(o=_addr(1)), 1),
       (_fwd, dict(o_rest=_addr(17) + 1), 1), (_fwd, dict(o_rest=_addr(17), o_dtype=0), 1), (_fwd, dict(o_rest=_addr(5) + 64), 1),
       (_fwd, dict(o_rest=_addr(2)), 1), (_fwd, dict(seqlen_k=4096, window=0, workspace=None), 3),
       (_fwd, dict(seqlen_k=4096, window=0, workspace_bytes=1000), 3), (_fwd, dict(seqlen_k=4096, window=0, workspace=_addr(20) + 64), 1),
       (_fwd, dict(seqlen_k=4096, window=0, workspace=_addr(2)), 1), (_bwd, dict(o_rest=_addr(17) + 1), 1), (_bwd, dict(o_rest=_addr(17), o_dtype=0), 1),
       (_bwd, dict(o_rest=_addr(17), dq=_addr(17)), 1),
       (_bwd, dict(dout=None), 1), (_bwd, dict(lse=None), 1), (_bwd, dict(grad_dtype=2), 1), (_bwd, dict(dq=_addr(12)), 1),
       (_bwd, dict(dk=_addr(15)), 1), (_bwd, dict(dv=_addr(15) + 2), 1), (_bwd, dict(dout=_addr(12) + 1), 1),
       (_bwd, dict(dq=_addr(5)), 1), (_bwd, dict(workspace=None), 3), (_bwd, dict(workspace_bytes=100), 3),
       (_bwd, dict(workspace=_addr(20) + 64), 1), (_bwd, dict(dk=_addr(20)), 1),
       (_bwd, dict(batch=1 << 12, num_seqs=1 << 12, seqlen=1 << 14, seqlen_k=1 << 14, nkheads=16, nheads=16, window=1, sinks=1), 2),
       (_write, dict(num_seqs=3), 1), (_write, dict(cu_seqlens=_addr(16)), 1), (_write, dict(cu_seqlens=_addr(16) + 2, batch=1), 1),
       (_write, dict(k=None), 1), (_write, dict(k_stride=5), 1), (_write, dict(v=_addr(3) + 1), 1), (_write, dict(k_cache=_addr(2)), 1),
       (_write, dict(k_cache=_addr(7)), 1), (_write, dict(k_scale=_addr(11)), 1), (_write, dict(seqlen=-1), 1),
       (_write, dict(batch=1 << 23, num_seqs=1 << 23), 2),
       (_step, dict(nheads=3), 1), (_step, dict(scale=-1.0), 1), (_step, dict(window=-2), 1), (_step, dict(sinks=-1), 1),
       (_step, dict(q=None), 1), (_step, dict(o=None), 1), (_step, dict(q_stride=255), 1), (_step, dict(o_dtype=2), 1),
       (_step, dict(o=_addr(6)), 1), (_step, dict(o=_addr(10) + 2), 1), (_step, dict(q=_addr(1) + 1), 1), (_step, dict(batch=1 << 23), 2),
       (_step, dict(table_rows=300, workspace=None), 3), (_step, dict(table_rows=300, workspace=_addr(20) + 4), 1),
       (_step, dict(table_rows=300, workspace_bytes=64), 3)])


@pytest.mark.parametrize("make,kw,status", BAD, ids=[f"{m.__name__}-{i}" for i, (m, _, _) in enumerate(BAD)])
def test_refusals(L, make, kw, status):
    """The check and the entry point itself refuse alike, before anything is launched."""
    p = make(**kw)
    assert getattr(L, CHECKS[make] + "_check")(ctypes.byref(p)) == status, L.ssm_last_error()
    assert L.ssm_last_error() != b""
    assert getattr(L, RUNS[make])(ctypes.byref(p), None) == status


def test_null_params(L):
    for make in CHECKS:
        assert getattr(L, CHECKS[make] + "_check")(None) == 1


def test_allowed_forms(L):
    none = dict(k_scale=None, v_scale=None)
    ok = [_fwd(lse=None), _fwd(window=0, sinks=9), _fwd(scale=0.0), _fwd(seqlen_k=50), _fwd(batch=0, num_seqs=0),
          _fwd(seqlen=0, q=None, o=None), _fwd(seqlen_k=0, k=None, v=None), _fwd(cu_seqlens=_addr(16), batch=1, num_seqs=7, seqlen_k=100),
          _fwd(cu_seqlens=_addr(16), cu_seqlens_k=_addr(17), batch=1, num_seqs=0), _fwd(q_stride=1000, k_stride=128, v_stride=130),
          _bwd(dq=None, dk=None, dv=None), _bwd(seqlen=0, q=None, o=None, dout=None, lse=None),
          _write(cache_dtype=1, **none), _write(x_dtype=0), _write(batch=0, num_seqs=0, lens=None), _write(table_rows=0, page_table=None),
          _write(pages=0, k_cache=None, v_cache=None, **none), _write(cu_seqlens=_addr(16), batch=1, num_seqs=5),
          _step(cache_dtype=1, **none), _step(x_dtype=0), _step(x_dtype=0, cache_dtype=1, **none), _step(x_dtype=0, cache_dtype=0, **none),
          _step(batch=0, q=None, o=None, lens=None), _step(nheads=80), _step(table_rows=0, page_table=None)]
    for p in ok:
        assert getattr(L, NAMES[type(p)] + "_check")(ctypes.byref(p)) == 0, (type(p), L.ssm_last_error())


def test_workspace_sizes(L):
    for p, name in ((_fwd(), "ssm_attn"), (_bwd(), "ssm_attn_bwd"), (_bwd(seqlen=5000, seqlen_k=5000), "ssm_attn_bwd"), (_step(), "ssm_attn_decode"),
                    (_step(table_rows=4096, batch=1), "ssm_attn_decode")):
        need = getattr(L, name + "_workspace_size")(ctypes.byref(p))
        p.workspace_bytes = need
        p.workspace = _addr(20) if need else None
        assert getattr(L, name + "_check")(ctypes.byref(p)) == 0
        if need:
            p.workspace_bytes = need - 1
            assert getattr(L, name + "_check")(ctypes.byref(p)) == 3
    size = lambda p: L.ssm_attn_bwd_workspace_size(ctypes.byref(p))  # noqa: E731
    assert size(_bwd(seqlen=5000, seqlen_k=5000)) > size(_bwd(seqlen=5000, seqlen_k=5000, sinks=0)) > 0
    assert size(_bwd(d_head=200)) == 0 and size(_bwd(struct_size=4)) == 0
    assert L.ssm_attn_decode_workspace_size(ctypes.byref(_step(d_head=200))) == 0
    # sizes past 32 bits
    assert size(_bwd(batch=1, num_seqs=1, seqlen=1 << 26, seqlen_k=1 << 20, nkheads=1, nheads=15, window=1000)) >= 1 << 32
