"""GPU parity of the block norm at its edges, against the float64 oracle, through the C ABI.

Bounds, set before the first run: all arithmetic is f32 on exact inputs, 1e-5 of the result's largest value; a
bf16 result adds its own rounding, 2^-8 of each value."""
import numpy as np
import pytest
import torch

import selective_state_space_03_amd as ssm
from gpu_util import DEV, check, np64
from oracle import delta_oracle as D

pytestmark = pytest.mark.gpu
TOL = 1e-5
BF, F32 = torch.bfloat16, torch.float32
CODE = {F32: 0, BF: 1}


def _inputs(seed, rows, d, dtype):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    return {"x": rnd(rows, d).to(dtype), "z": rnd(rows, d).to(dtype), "norm_w": 1.0 + 0.3 * rnd(d), "scale": rnd(d),
            "out_norm_w": 1.0 + 0.3 * rnd(d)}


def _guarded(shape, dtype):
    """A NaN-filled tensor and the elements behind it in the same allocation, twice its bytes and more."""
    n = shape[0] * shape[1]
    whole = torch.full((4 * n + 64,), 7.0, dtype=dtype, device=DEV)
    whole[:n] = float("nan")
    return whole[:n].view(shape), whole[n:]


@pytest.mark.parametrize("d", [96, 100, 97, 2560])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("res", [F32, BF])
def test_residual_out_without_residual_takes_res_dtype(d, dtype, res):
    """t goes out in res_dtype, whatever the type of x, also where no residual comes in."""
    c = _inputs(d, 5, d, dtype)
    t, guard = _guarded((5, d), res)
    call = ssm.block_norm_fwd(**c, residual_out=t, prepare=True)
    call._p.res_dtype = CODE[res]
    out, got = call.run()
    torch.cuda.synchronize()
    ro, rt = D.block_norm(**{k: np64(v) for k, v in c.items()})
    assert got is t and (guard == 7).all()
    check(np64(got), rt, TOL, "t", out_bf16=res == BF)
    check(np64(out), ro, TOL, "out", out_bf16=dtype == BF)


@pytest.mark.parametrize("d", [96, 100, 97])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("res", [F32, BF])
def test_binding_passes_residual_outs_type(d, dtype, res):
    """The type of a residual_out given by the caller is the one the kernel writes."""
    c = _inputs(d, 5, d, dtype)
    t, guard = _guarded((5, d), res)
    call = ssm.block_norm_fwd(**c, residual_out=t, prepare=True)
    assert call._p.res_dtype == CODE[res]
    call.run()
    torch.cuda.synchronize()
    assert (guard == 7).all()
    check(np64(t), D.block_norm(**{k: np64(v) for k, v in c.items()})[1], TOL, "t", out_bf16=res == BF)
    with pytest.raises(TypeError):
        ssm.block_norm_fwd(**c, residual_out=torch.empty(5, d, dtype=torch.float16, device=DEV))
    with pytest.raises(TypeError):
        ssm.block_norm_fwd(**c, residual=torch.empty(5, d, dtype=F32 if res == BF else BF, device=DEV), residual_out=t)


def test_more_rows_than_a_launch_holds():
    """2^28 groups and some, 16 lanes each: the threads of one launch would be 2^32.  Every row equals that of a
    call on a part of the rows."""
    rows, d, n = (1 << 25) + 9, 64, 8
    gen = torch.Generator(device=DEV).manual_seed(8)
    x = torch.randn(rows, d, generator=gen, device=DEV, dtype=BF)
    w = 1.0 + 0.3 * torch.randn(n, generator=gen, device=DEV)
    out, _ = ssm.block_norm_fwd(x, norm_w=w)
    for a, b in ((0, 1 << 23), (1 << 23, 1 << 24), (1 << 24, 3 << 23), (3 << 23, rows)):
        part, _ = ssm.block_norm_fwd(x[a:b], norm_w=w)
        torch.cuda.synchronize()
        assert torch.equal(part, out[a:b]), (a, b)
    last = slice(rows - 20, rows)
    check(np64(out[last]), D.block_norm(np64(x[last]), norm_w=np64(w), group_size=n)[0], TOL, "last rows", out_bf16=True)


@pytest.mark.parametrize("groups,n", [(65535, 2), (65536, 2), (70001, 3)])
def test_gradients_of_many_weight_rows(groups, n):
    """A weight per channel in more groups than a launch holds workgroups along y."""
    gen = torch.Generator(device=DEV).manual_seed(n)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    x, w, do = rnd(3, groups * n), 1.0 + 0.3 * rnd(groups * n), rnd(3, groups * n)
    g = ssm.block_norm_bwd(x, norm_w=w, group_size=n, dout=do)
    torch.cuda.synchronize()
    r = D.block_norm_backward(np64(x), norm_w=np64(w), group_size=n, dout=np64(do))
    assert set(g) == {"x", "norm_w"}
    check(np64(g["norm_w"]), r["norm_w"], TOL, "dnorm_w")
    check(np64(g["x"]), r["x"], TOL, "dx")


@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_gradients_of_single_values(eps):
    """A row of one value is normalised to its sign: without an epsilon its gradient is 0 at every size of value, and
    with one eps / (y^2 + eps)^1.5."""
    x = torch.tensor([3.0, -1e-3, 1e-14, -1e-18, 1e15], device=DEV).view(5, 1)
    w, do = torch.full((1,), 1.5, device=DEV), torch.tensor([1.0, -2.0, 0.5, 1.0, 1.0], device=DEV).view(5, 1)
    g = ssm.block_norm_bwd(x, norm_w=w, dout=do, eps=eps)
    torch.cuda.synchronize()
    y = np64(x)
    # (eps as the kernel holds it, in 32 bits)
    e = float(np.float32(eps))
    check(np64(g["x"]), 1.5 * np64(do) * e / (y * y + e) ** 1.5 if eps else np.zeros((5, 1)), TOL, "dx")
    check(np64(g["norm_w"]), (np64(do) * y / np.sqrt(y * y + e)).sum(0), TOL, "dnorm_w")


def test_rows_past_31_bits_are_refused():
    """2^32 + 64 values a row (of no memory here) are not taken for 64."""
    x = torch.empty(1, 1, dtype=BF, device=DEV).expand(1, (1 << 32) + 64)
    for call in (ssm.block_norm_fwd, ssm.block_norm_bwd):
        with pytest.raises(ValueError, match="values a row, more than"):
            call(x, group_size=64)
