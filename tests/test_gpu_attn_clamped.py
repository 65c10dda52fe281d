"""Offsets out of range in packed calls of the window attention and in writes to its cache: they are clamped, and no
access leaves the tensors.  Every tensor that a call reads or writes lies between guards: NaN around the inputs, a known
value around the outputs and the workspace."""
import ctypes

import pytest
import torch

import selective_state_space_03_amd as ssm
from gpu_util import DEV
from selective_state_space_03_amd import attn

pytestmark = pytest.mark.gpu
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
GUARD = 1 << 16  # elements on either side
BAD = [[-5, 40, 300], [0, 90, 20, 100], [50, 10, 2 ** 31 - 1], [-2 ** 31, -7, 2 ** 31 - 1], [2 ** 31 - 1, 0, -1, 60]]


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class _Guarded:
    """Tensors in the middle of longer ones; outputs filled with 7 inside and out."""

    def __init__(self):
        self.all = []

    def put(self, t):
        whole = torch.full((t.numel() + 2 * GUARD,), float("nan"), device=DEV).to(t.dtype)
        inside = whole[GUARD:GUARD + t.numel()].view(t.shape)
        inside.copy_(t)
        self.all.append((whole, whole.view(torch.uint8).clone(), t.numel()))
        return inside

    def empty(self, shape, dtype, *_):
        shape = (shape,) if isinstance(shape, int) else tuple(shape)
        n = torch.Size(shape).numel()
        whole = torch.full((n + 2 * GUARD,), 7.0, device=DEV).to(dtype)
        self.all.append((whole, whole.view(torch.uint8).clone(), n))
        return whole[GUARD:GUARD + n].view(shape)

    def intact(self):
        torch.cuda.synchronize()
        for whole, was, n in self.all:
            now, e = whole.view(torch.uint8), whole.element_size()
            assert torch.equal(now[:GUARD * e], was[:GUARD * e]) and torch.equal(now[(GUARD + n) * e:], was[(GUARD + n) * e:])


def _both(q, k, v, do, cu, g, cu_k=None, **kw):
    o, lse = g.empty(q.shape, q.dtype), g.empty(q.shape[:3], F32)
    kw.update(cu_seqlens=_dev(cu), cu_seqlens_k=None if cu_k is None else _dev(cu_k))
    ssm.attn_fwd(q, k, v, o=o, lse=lse, **kw)
    return [o, lse, *ssm.attn_bwd(q, k, v, o, lse, do, grad_dtype=q.dtype, **kw).values()]


def _guard_the_binding(g, monkeypatch):
    """Gradients and workspaces that the binding allocates lie between guards too."""
    monkeypatch.setattr(attn, "_empty", g.empty)

    def workspace(p, need, given, dev, stream):
        t = g.empty(need, torch.uint8) if need else None
        if t is not None:
            assert t.data_ptr() % 256 == 0
            p.workspace, p.workspace_bytes = t.data_ptr(), need
        return t

    monkeypatch.setattr(attn, "_workspace", workspace)


@pytest.mark.parametrize("dtype,D", [(BF, 32), (BF, 128), (BF, 33), (F32, 64)])
@pytest.mark.parametrize("window,sinks", [(9, 2), (None, 0)])
def test_offsets_leave_everything_else_alone(dtype, D, window, sinks, monkeypatch):
    gen = torch.Generator(device=DEV).manual_seed(D)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV).to(dtype)  # noqa: E731
    for cu in BAD:
        g = _Guarded()
        _guard_the_binding(g, monkeypatch)
        q, k, v, do = g.put(rnd(1, 100, 2, D)), g.put(rnd(1, 100, 1, D)), g.put(rnd(1, 100, 1, D)), g.put(rnd(1, 100, 2, D))
        _both(q, k, v, do, cu, g, window=window, sinks=sinks)
        k, v = g.put(rnd(1, 210, 1, D)), g.put(rnd(1, 210, 1, D))
        _both(q, k, v, do, cu, g, cu_k=cu[:1] + [x + 3 if 0 <= x < 1000 else x for x in cu[1:]], window=window, sinks=sinks)
        g.intact()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_offsets_past_the_ends_are_the_ends(dtype):
    """Rising offsets that only reach over the tensors' ends: as the ends themselves, bit for bit."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV).to(dtype)  # noqa: E731
    q, k, v, do = rnd(1, 300, 2, 64), rnd(1, 300, 1, 64), rnd(1, 300, 1, 64), rnd(1, 300, 2, 64)
    for cu, means in (([-5, 140, 900], [0, 140, 300]), ([-9, -3, 20, 2 ** 31 - 1], [0, 0, 20, 300]), ([299, 300, 301, 400], [299, 300, 300, 300])):
        got = _both(q, k, v, do, cu, _Guarded(), window=50, sinks=3)
        want = _both(q, k, v, do, means, _Guarded(), window=50, sinks=3)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), cu


@pytest.mark.parametrize("dtype,kind,D", [(BF, E4, 64), (F32, E4, 40), (BF, BF, 33), (F32, F32, 128)])
def test_writes_leave_everything_else_alone(dtype, kind, D):
    """Offsets, lengths and entries out of range."""
    gen = torch.Generator(device=DEV).manual_seed(D)
    pages, hk, page = 9, 2, 16
    for cu in BAD:
        g = _Guarded()
        k, v = (g.put(torch.randn((1, 100, hk, D), generator=gen, device=DEV).to(dtype)) for _ in range(2))
        kc, vc = (g.empty((pages, hk, page, D), kind) for _ in range(2))
        ks, vs = (g.empty((pages, hk), F32) for _ in range(2)) if kind == E4 else (None, None)
        n = len(cu) - 1
        table = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)[:2 * n].view(n, 2)
        table[0, 1] = 2 ** 31 - 1
        lens = g.put(_dev([2 ** 31 - 1, -2 ** 31, 17, 5][:n]))
        ssm.attn_cache_write(k, v, kc, vc, g.put(table), lens, cu_seqlens=g.put(_dev(cu)), k_scale=ks, v_scale=vs)
        q, o = g.put(torch.randn((n, 4, D), generator=gen, device=DEV).to(dtype)), g.empty((n, 4, D), F32)
        ssm.attn_decode_step(q, kc, vc, g.put(table), lens, k_scale=ks, v_scale=vs, o=o)
        g.intact()
