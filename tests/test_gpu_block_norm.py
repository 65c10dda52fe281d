"""GPU parity of the block norm (ssm_block_norm_fwd / _bwd) against the float64 oracle, through the C ABI.

Bounds, set before the first run: all arithmetic is f32 on exact inputs, a row's sums run over at most 16384
values in registers and a tree (a few hundred roundings), column sums over at most a few hundred rows in a row:
1e-5 of the result's largest value; a bf16 result adds its own rounding, 2^-8 of each value."""
import numpy as np
import pytest
import torch

import selective_state_space_03_amd as ssm
from gpu_util import DEV, check, np64
from oracle import delta_oracle as D

pytestmark = pytest.mark.gpu
TOL = 1e-5
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _seed():
    torch.manual_seed(0)


def _inputs(seed, rows, d, dtype, opt, res_dtype=F32):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    c = {"x": rnd(rows, d).to(dtype)}
    if opt.get("z"):
        c["z"] = rnd(rows, d).to(dtype)
    if opt.get("norm_w"):
        c["norm_w"] = 1.0 + 0.3 * rnd(d if opt["norm_w"] == "all" else opt.get("group_size", d))
    if opt.get("residual"):
        c["residual"] = (2.0 * rnd(rows, d)).to(res_dtype)
    if opt.get("scale"):
        c["scale"] = rnd(d)
    if opt.get("out_norm_w"):
        c["out_norm_w"] = 1.0 + 0.3 * rnd(d)
    return c


def _kw(opt):
    return {k: opt[k] for k in ("gate_first", "group_size") if k in opt}


def _ref_in(c):
    return {k: np64(t) for k, t in c.items()}


def _check(c, opt, dout_dtype=None, grad_dtype=None, what=""):
    kw = _kw(opt)
    out, res = ssm.block_norm_fwd(**c, **kw)
    torch.cuda.synchronize()
    ro, rt = D.block_norm(**_ref_in(c), **kw)
    if out is not None:
        check(np64(out), ro, TOL, what + " out", out_bf16=out.dtype == BF)
    assert (res is not None) == ("residual" in c)
    if res is not None:
        check(np64(res), rt, TOL, what + " residual", out_bf16=res.dtype == BF)
    dt = c["x"].dtype
    dout = torch.randn(c["x"].shape, device=DEV).to(dout_dtype or dt) if out is not None else None
    dres = torch.randn(c["x"].shape, device=DEV).to(c["residual"].dtype) if res is not None else None
    g = ssm.block_norm_bwd(**c, **kw, dout=dout, dresidual=dres, grad_dtype=grad_dtype)
    torch.cuda.synchronize()
    r = D.block_norm_backward(**_ref_in(c), **kw, dout=None if dout is None else np64(dout),
                              dt=None if dres is None else np64(dres))
    assert set(g) == set(c)
    for x in g:
        check(np64(g[x]), r[x], TOL, f"{what} d{x}", out_bf16=g[x].dtype == BF)


OPTS = {
    "bare": dict(norm_w=1),
    "gated": dict(norm_w=1, z=1),
    "gate_first": dict(norm_w=1, z=1, gate_first=True),
    "no_norm": dict(z=1),
    "residual": dict(residual=1),
    "scaled": dict(residual=1, scale=1),
    "end": dict(residual=1, scale=1, out_norm_w=1),
    "all": dict(norm_w=1, z=1, residual=1, scale=1, out_norm_w=1),
    "all_first": dict(norm_w=1, z=1, gate_first=True, residual=1, scale=1, out_norm_w=1),
    "no_residual": dict(z=1, scale=1, out_norm_w=1),
}


@pytest.mark.parametrize("name", list(OPTS))
@pytest.mark.parametrize("dtype,res", [(F32, F32), (BF, F32), (BF, BF)])
def test_parts(name, dtype, res):
    _check(_inputs(1, 33, 320, dtype, OPTS[name], res), OPTS[name], what=name)


@pytest.mark.parametrize("d", [1, 2, 7, 8, 12, 100, 128, 129, 256, 260, 512, 1000, 1499, 2048, 2560, 4100, 8192, 16384])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_widths(d, dtype):
    opt = OPTS["all"]
    for rows in (1, 5):
        _check(_inputs(d, rows, d, dtype, opt), opt, grad_dtype=dtype, what=f"d={d} rows={rows}")


@pytest.mark.parametrize("d", [264, 640, 1111, 1600, 2000, 2560, 2700, 4096])
def test_many_rows(d):
    """More rows than the backward has workgroups: each walks several."""
    opt = OPTS["all"]
    _check(_inputs(d, 1027, d, BF, opt), opt, what=f"d={d}")


@pytest.mark.parametrize("d", [4104, 5120, 8192, 9001])
@pytest.mark.parametrize("dtype,grads", [(F32, F32), (BF, F32), (BF, BF)])
@pytest.mark.parametrize("name", ["all", "all_first"])
def test_many_long_rows(d, dtype, grads, name):
    """Rows long enough for the widest team, more of them than workgroups."""
    _check(_inputs(d, 519, d, dtype, OPTS[name], dtype), OPTS[name], grad_dtype=grads, what=f"{name} d={d}")


@pytest.mark.parametrize("group,groups", [(1, 5), (8, 3), (96, 10), (100, 3), (128, 32), (257, 3), (600, 2)])
@pytest.mark.parametrize("whole", [False, True])
def test_groups(group, groups, whole):
    """Weights shared by the groups, or one for every channel; gate before and after."""
    for first in (False, True):
        opt = dict(norm_w="all" if whole else 1, z=1, gate_first=first, group_size=group)
        _check(_inputs(group, 41, group * groups, F32, opt), opt, what=f"{group}x{groups} whole={whole}")


def test_group_size_follows_the_weight():
    c = _inputs(3, 6, 64, F32, dict(norm_w=1, z=1, group_size=16))
    a, _ = ssm.block_norm_fwd(**c)
    b, _ = ssm.block_norm_fwd(**c, group_size=16)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_strided_rows():
    for pad in (8, 3):
        wide = torch.randn(2, 9, 3 * 40 + pad, device=DEV).to(BF)
        x, z = wide[..., 40:80], wide[..., 80:120]
        w = torch.rand(40, device=DEV)
        a, _ = ssm.block_norm_fwd(x, z=z, norm_w=w)
        b, _ = ssm.block_norm_fwd(x.contiguous(), z=z.contiguous(), norm_w=w)
        do = torch.randn(2, 9, 40, device=DEV).to(BF)
        ga = ssm.block_norm_bwd(x, z=z, norm_w=w, dout=do)
        gb = ssm.block_norm_bwd(x.contiguous(), z=z.contiguous(), norm_w=w, dout=do)
        torch.cuda.synchronize()
        assert torch.equal(a, b) and all(torch.equal(ga[k], gb[k]) for k in gb)


def test_unaligned_bases():
    c = _inputs(4, 5, 64, F32, OPTS["all"])
    def shifted(t):
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        b[1:] = t.flatten()
        return b[1:].view(t.shape)
    a, b = ssm.block_norm_fwd(**{k: shifted(t) for k, t in c.items()}), ssm.block_norm_fwd(**c)
    torch.cuda.synchronize()
    check(np64(a[0]), np64(b[0]), 1e-6, "unaligned out")
    assert torch.equal(a[1], b[1])


def test_residual_in_place_and_one_gradient_only():
    c = _inputs(5, 20, 320, BF, OPTS["end"], BF)
    out, res = ssm.block_norm_fwd(**c)
    mine = c["residual"].clone()
    out2, res2 = ssm.block_norm_fwd(**dict(c, residual=mine), residual_out=mine)
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(res, res2) and res2.data_ptr() == mine.data_ptr()
    do = torch.randn(20, 320, device=DEV)
    for kw, ref in ((dict(dout=do), dict(dout=np64(do))), (dict(dresidual=do), dict(dt=np64(do)))):
        g = ssm.block_norm_bwd(**c, **kw)
        torch.cuda.synchronize()
        r = D.block_norm_backward(**_ref_in(c), **ref)
        for x in g:
            if np.any(r[x]):
                check(np64(g[x]), r[x], TOL, f"{list(kw)} d{x}", out_bf16=g[x].dtype == BF)
            else:
                assert not g[x].any()


def test_extreme_rows():
    """Zero rows (the epsilon alone), large and tiny values, a gate far out on both sides."""
    x = torch.zeros(4, 64, device=DEV)
    x[1], x[2], x[3] = 1e15, 1e-15, torch.randn(64, device=DEV)
    z = torch.tensor([[0.0], [80.0], [-80.0], [-300.0]], device=DEV).expand(4, 64).contiguous()
    w = torch.rand(64, device=DEV)
    for first in (False, True):
        out, _ = ssm.block_norm_fwd(x, z=z, norm_w=w, gate_first=first)
        torch.cuda.synchronize()
        ro, _ = D.block_norm(np64(x), z=np64(z), norm_w=np64(w), gate_first=first)
        for i in range(4):
            check(np64(out[i]), ro[i], TOL, f"row {i} first={first}") if np.any(np.abs(ro[i]) > 1e-30) else None


def test_no_rows():
    c = _inputs(6, 0, 320, BF, OPTS["all"])
    out, res = ssm.block_norm_fwd(**c)
    g = ssm.block_norm_bwd(**c, dout=out, dresidual=res)
    torch.cuda.synchronize()
    assert out.shape == (0, 320) and not g["norm_w"].any() and not g["scale"].any() and not g["out_norm_w"].any()


def test_repeatable_streams_and_graph():
    c = _inputs(7, 3000, 640, BF, OPTS["all"])
    do = torch.randn(3000, 640, device=DEV).to(BF)
    want = ssm.block_norm_bwd(**c, dout=do)
    fw = ssm.block_norm_fwd(**c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = ssm.block_norm_bwd(**c, dout=do, stream=s)
    fo = ssm.block_norm_fwd(**c, stream=s)
    s.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want) and torch.equal(fo[0], fw[0]) and torch.equal(fo[1], fw[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        go = ssm.block_norm_fwd(**c, stream=s)
        gg = ssm.block_norm_bwd(**c, dout=do, stream=s)
    for _ in range(3):
        c["x"].normal_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        w, f = ssm.block_norm_bwd(**c, dout=do), ssm.block_norm_fwd(**c)
        torch.cuda.synchronize()
        assert all(torch.equal(gg[k], w[k]) for k in w) and torch.equal(go[0], f[0]) and torch.equal(go[1], f[1])
