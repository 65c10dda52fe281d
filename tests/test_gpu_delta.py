"""GPU parity of the gated delta rule (ssm_delta_chunk_fwd / _bwd, ssm_delta_decode_step) against the float64
oracle, through the C ABI.

Bounds, set before the first run: every 32-bit operand of a matrix product keeps 24 bits (three bf16 parts) and
sums are 32-bit, so an f32 result is off by a few times 2^-23 per product of the longest chain (norm, L, the
inverse, three products a chunk): 1e-5 of the result's largest value, as for the framework's other f32 paths.
With bf16 inputs the operands that only reach o keep two parts (2^-16 each, four of them in a product): 1e-4 of
the largest value.  A bf16 result adds its own rounding, 2^-8 of each value."""
import numpy as np
import pytest
import torch

import selective_state_space_03_amd as ssm
from gpu_util import DEV, check, np64
from oracle import delta_oracle as D

pytestmark = pytest.mark.gpu
TOL_F32 = 1e-5
TOL_O_BF16 = 1e-4


@pytest.fixture(autouse=True)
def _seed():
    torch.manual_seed(0)


def _case(seed, n, L, Hk, H, K, V, dtype=torch.float32, unit=True, cu=None, state=True, gmin=-1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    sc = 1.0 if unit else K ** -0.5
    c = dict(q=(rnd(n, L, Hk, K) * sc).to(dtype), k=(rnd(n, L, Hk, K) * sc).to(dtype), v=rnd(n, L, H, V).to(dtype),
             g=gmin * torch.rand((n, L, H), generator=gen, device=DEV), beta=torch.sigmoid(rnd(n, L, H)))
    seqs = n if cu is None else len(cu) - 1
    st = rnd(seqs, H, V, K) if state else None
    return c, st


def _ref(c, st, **kw):
    cu = kw.pop("cu", None)
    return D.delta_rule(*(np64(c[x]) for x in ("q", "k", "v", "g", "beta")), cu=cu,
                        state=None if st is None else np64(st), **kw)


def _cu(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)


def _run(c, st, cu=None, **kw):
    seqs = c["q"].shape[0] if cu is None else len(cu) - 1
    out = torch.full((seqs, c["v"].shape[2], c["v"].shape[3], c["q"].shape[3]), float("nan"), device=DEV)
    o = ssm.delta_chunk_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], cu_seqlens=_cu(cu), state_in=st, state_out=out, **kw)
    torch.cuda.synchronize()
    return o, out


def _check(c, st, cu=None, what="", **kw):
    o, s = _run(c, st, cu, **kw)
    kw.pop("o_dtype", None)
    ro, rs = _ref(c, st, cu=cu, **kw)
    bf = o.dtype == torch.bfloat16
    check(np64(o), ro, TOL_O_BF16 if c["q"].dtype == torch.bfloat16 else TOL_F32, what + " o", out_bf16=bf)
    check(np64(s), rs, TOL_F32, what + " state")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 130, 200])
def test_lengths(dtype, L):
    c, st = _case(L, 2, L, 2, 4, 64, 48, dtype)
    _check(c, st, qk_norm=True, what=f"L={L}")


@pytest.mark.parametrize("K,V", [(1, 1), (7, 5), (16, 16), (33, 17), (64, 96), (65, 33), (100, 40), (128, 128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_head_sizes(K, V, dtype):
    c, st = _case(K * V, 1, 97, 1, 2, K, V, dtype, unit=False)
    _check(c, st, what=f"K={K} V={V}")


@pytest.mark.parametrize("Hk,H", [(1, 1), (1, 7), (3, 9), (5, 5)])
def test_shared_heads_and_wide_slices(Hk, H):
    """Few groups take 16 value channels per workgroup, many take 32: both, with a ragged last slice."""
    for n in (1, 60):
        c, st = _case(H, n, 70, Hk, H, 32, 72, torch.bfloat16)
        _check(c, st, qk_norm=True, what=f"Hk={Hk} H={H} n={n}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_packed_with_empty_and_ragged_sequences(dtype):
    cu = [0, 0, 1, 64, 64, 129, 200, 331, 331]
    c, st = _case(9, 1, 331, 2, 4, 48, 40, dtype, cu=cu)
    _check(c, st, cu, qk_norm=True, what="packed")
    c, _ = _case(10, 1, 331, 2, 4, 48, 40, dtype, cu=cu)
    _check(c, None, cu, qk_norm=True, what="packed from zero")


def test_packed_equals_each_alone():
    cu = [0, 77, 205, 206]
    c, st = _case(11, 1, 206, 2, 2, 64, 32, torch.bfloat16, cu=cu)
    o, s = _run(c, st, cu, qk_norm=True)
    for i, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        one = {x: t[:, a:b].contiguous() for x, t in c.items()}
        oi, si = _run(one, st[i:i + 1].contiguous(), qk_norm=True)
        assert torch.equal(oi, o[:, a:b]) and torch.equal(si[0], s[i])


def test_tokens_outside_the_sequences_are_neither_read_nor_written():
    c, st = _case(12, 1, 150, 1, 2, 32, 32, torch.float32, cu=[0, 1])
    for x in ("q", "k", "v", "g", "beta"):
        c[x][:, :10] = float("nan")
        c[x][:, 101:] = float("nan")
    o = torch.full_like(c["v"], 7.0)
    cu = [10, 50, 101]
    st = torch.randn(2, 2, 32, 32, device=DEV)
    out = torch.empty_like(st)
    ssm.delta_chunk_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], cu_seqlens=_cu(cu), state_in=st, state_out=out, o=o,
                        qk_norm=True)
    torch.cuda.synchronize()
    assert (o[:, :10] == 7).all() and (o[:, 101:] == 7).all()
    inner = {x: t[:, 10:101].contiguous() for x, t in c.items()}
    ro, rs = _ref(inner, st, cu=[0, 40, 91], qk_norm=True)
    check(np64(o[:, 10:101]), ro, TOL_F32, "inner o")
    check(np64(out), rs, TOL_F32, "inner state")


def test_offsets_out_of_range_stay_inside():
    """cu_seqlens is read on the device only: offsets out of range or order are clamped, nothing outside is touched."""
    c, _ = _case(13, 1, 100, 1, 1, 16, 16)
    guard = torch.full((300, 1, 16), 3.0, device=DEV)
    o = guard[100:200].unsqueeze(0)
    for cu in ([-5, 40, 1000], [90, 20, 60], [2 ** 31 - 1, -2 ** 31, 50]):
        ssm.delta_chunk_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], cu_seqlens=_cu(cu), o=o)
        torch.cuda.synchronize()
        assert (guard[:100] == 3).all() and (guard[200:] == 3).all()


def test_slices_of_a_wider_projection():
    n, L, Hk, H, K, V = 2, 130, 2, 4, 32, 24
    c, st = _case(14, n, L, Hk, H, K, V, torch.bfloat16)
    for pad in (0, 3):  # even strides, and ones that allow no wide loads
        wide = torch.full((n, L, 2 * Hk * K + H * V + pad), float("nan"), device=DEV, dtype=torch.bfloat16)
        wide[..., :Hk * K] = c["q"].flatten(2)
        wide[..., Hk * K:2 * Hk * K] = c["k"].flatten(2)
        wide[..., 2 * Hk * K:2 * Hk * K + H * V] = c["v"].flatten(2)
        s = dict(c, q=wide[..., :Hk * K].unflatten(-1, (Hk, K)), k=wide[..., Hk * K:2 * Hk * K].unflatten(-1, (Hk, K)),
                 v=wide[..., 2 * Hk * K:2 * Hk * K + H * V].unflatten(-1, (H, V)))
        a, b = _run(s, st, qk_norm=True), _run(c, st, qk_norm=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        do = torch.randn(n, L, H, V, device=DEV).to(torch.bfloat16)
        ga = ssm.delta_chunk_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], do, qk_norm=True, state_in=st)
        gb = ssm.delta_chunk_bwd(c["q"], c["k"], c["v"], c["g"], c["beta"], do, qk_norm=True, state_in=st)
        torch.cuda.synchronize()
        assert all(torch.equal(ga[x], gb[x]) for x in gb)


def test_unaligned_bases():
    c, st = _case(15, 1, 70, 1, 2, 24, 24)
    def shifted(t):
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        b[1:] = t.flatten()
        return b[1:].view(t.shape)
    a, b = _run({x: shifted(t) for x, t in c.items()}, shifted(st)), _run(c, st)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("gmin", [0.0, -30.0, -200.0, -1e6])
def test_decays_from_none_to_total(gmin):
    """exp(G_t - G_s) above the diagonal would overflow, and a 32-bit running sum would lose the small gaps."""
    c, st = _case(16, 1, 150, 1, 2, 32, 32, gmin=gmin)
    _check(c, st, qk_norm=True, what=f"g to {gmin}")


def test_resets_and_no_writes():
    c, st = _case(17, 1, 150, 1, 2, 32, 32, gmin=-0.1)
    c["g"][:, 70] = float("-inf")
    c["g"][:, 100, 1] = -1e30
    c["beta"][:, 20:90, 0] = 0.0
    c["k"][:, 30:40] = 0.0
    _check(c, st, qk_norm=True, what="resets")
    do = torch.randn_like(c["v"])
    _check_grads(c, st, do, torch.randn_like(st), qk_norm=True, what="resets")


def test_equal_keys():
    """Every key of a chunk alike (L is full of ones): the inverse is taken by substitution, not by powers of L."""
    c, st = _case(18, 1, 128, 1, 1, 32, 16, gmin=0.0)
    c["k"] = c["k"][:, :1].expand(1, 128, 1, 32).contiguous()
    c["beta"].fill_(1.0)
    _check(c, st, qk_norm=True, what="equal keys")


def test_output_types_default_scale_and_scale():
    c, st = _case(19, 1, 66, 1, 2, 32, 20, torch.bfloat16)
    _check(c, st, o_dtype=torch.float32, qk_norm=True, what="bf16 in, f32 out")
    _check(c, st, qk_norm=True, scale=0.75, what="scale")
    _check({x: t.float() for x, t in c.items()}, st, o_dtype=torch.bfloat16, qk_norm=True, what="f32 in, bf16 out")


def test_state_in_place_and_empty_calls():
    c, st = _case(20, 2, 70, 1, 2, 32, 20)
    o, s = _run(c, st)
    mine = st.clone()
    o2 = ssm.delta_chunk_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], state_in=mine, state_out=mine)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(s, mine)
    none = {x: t[:, :0].contiguous() for x, t in c.items()}
    o, s = _run(none, st)
    assert o.shape == (2, 0, 2, 20) and torch.equal(s, st)
    g = ssm.delta_chunk_bwd(none["q"], none["k"], none["v"], none["g"], none["beta"], none["v"], state_in=st, dstate_out=st)
    torch.cuda.synchronize()
    assert torch.equal(g["state_in"], st)
    o, s = _run({x: t[:0].contiguous() for x, t in c.items()}, None)
    assert o.shape == (0, 70, 2, 20)


# ---------------------------------------------------------------- backward

def _check_grads(c, st, do, ds, cu=None, grad_dtype=None, what="", **kw):
    g = ssm.delta_chunk_bwd(c["q"], c["k"], c["v"], c["g"], c["beta"], do, cu_seqlens=_cu(cu), state_in=st, dstate_out=ds,
                            grad_dtype=grad_dtype, **kw)
    torch.cuda.synchronize()
    r = D.delta_rule_backward(*(np64(c[x]) for x in ("q", "k", "v", "g", "beta")), np64(do), cu=cu,
                              state=None if st is None else np64(st), dstate=None if ds is None else np64(ds), **kw)
    for x in g:
        check(np64(g[x]), r[x], TOL_F32, f"{what} d{x}", out_bf16=g[x].dtype == torch.bfloat16)
    assert ("state_in" in g) == (st is not None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L", [1, 2, 17, 64, 65, 150])
def test_grads_lengths(dtype, L):
    c, st = _case(30 + L, 2, L, 2, 4, 64, 48, dtype)
    do, ds = torch.randn_like(c["v"]), torch.randn_like(st)
    _check_grads(c, st, do, ds, qk_norm=True, what=f"L={L}")


@pytest.mark.parametrize("K,V", [(1, 1), (7, 5), (33, 17), (100, 40), (128, 128), (64, 130)])
def test_grads_head_sizes(K, V):
    c, st = _case(K * V, 1, 97, 1, 3, K, V, unit=False)
    _check_grads(c, st, torch.randn_like(c["v"]), torch.randn_like(st), what=f"K={K} V={V}")
    _check_grads(c, None, torch.randn_like(c["v"]), None, what=f"K={K} V={V} from zero")


def test_grads_packed_shared_heads_bf16():
    cu = [0, 0, 1, 65, 129, 200]
    c, st = _case(41, 1, 200, 2, 6, 48, 40, torch.bfloat16, cu=cu)
    do, ds = torch.randn_like(c["v"]), torch.randn_like(st)
    _check_grads(c, st, do, ds, cu, qk_norm=True, what="packed")
    _check_grads(c, st, do, None, cu, grad_dtype=torch.bfloat16, qk_norm=True, what="packed bf16")


def test_grads_against_differences():
    """The forward kernel's own change along a direction, against the gradients' inner product with it.  A step h
    leaves an error of h^2 times the third derivative and the f32 results' rounding over h: 2e-3 at h = 1e-2."""
    c, st = _case(43, 1, 90, 1, 2, 32, 24, gmin=-0.5)
    do, ds = torch.randn_like(c["v"]), torch.randn_like(st)
    g = ssm.delta_chunk_bwd(c["q"], c["k"], c["v"], c["g"], c["beta"], do, qk_norm=True, state_in=st, dstate_out=ds)
    g = dict(g, state=g.pop("state_in"))
    loss = lambda r: float((r[0].double() * do.double()).sum() + (r[1].double() * ds.double()).sum())  # noqa: E731
    for x in ("q", "k", "v", "g", "beta", "state"):
        t = st if x == "state" else c[x]
        e = torch.randn_like(t) * (0.1 if x in ("g", "beta") else 1.0)
        h = 1e-2
        if x == "state":
            num = (loss(_run(c, st + h * e, qk_norm=True)) - loss(_run(c, st - h * e, qk_norm=True))) / (2 * h)
        else:
            num = (loss(_run(dict(c, **{x: t + h * e}), st, qk_norm=True))
                   - loss(_run(dict(c, **{x: t - h * e}), st, qk_norm=True))) / (2 * h)
        want = float((g[x].double() * e.double()).sum())
        size = float(g[x].double().norm() * e.double().norm())
        assert abs(num - want) <= 2e-3 * size, (x, num, want, size)


def test_repeatable():
    c, st = _case(44, 2, 300, 2, 8, 64, 64, torch.bfloat16)
    do = torch.randn_like(c["v"])
    runs = [ssm.delta_chunk_bwd(c["q"], c["k"], c["v"], c["g"], c["beta"], do, qk_norm=True, state_in=st) for _ in range(3)]
    fwd = [_run(c, st, qk_norm=True) for _ in range(3)]
    torch.cuda.synchronize()
    for r in runs[1:]:
        assert all(torch.equal(r[x], runs[0][x]) for x in r)
    for r in fwd[1:]:
        assert torch.equal(r[0], fwd[0][0]) and torch.equal(r[1], fwd[0][1])


# ---------------------------------------------------------------- one token

@pytest.mark.parametrize("K,V", [(1, 1), (7, 5), (33, 17), (64, 96), (100, 40), (128, 128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch", [1, 3, 70])
def test_step(K, V, dtype, batch):
    c, st = _case(50 + K, batch, 1, 2, 4, K, V, dtype)
    ro, rs = _ref(c, st, qk_norm=True)
    tok = {x: t[:, 0].contiguous() for x, t in c.items()}
    o = ssm.delta_decode_step(tok["q"], tok["k"], tok["v"], tok["g"], tok["beta"], st, qk_norm=True)
    torch.cuda.synchronize()
    check(np64(o), ro[:, 0], TOL_F32, "step o", out_bf16=dtype == torch.bfloat16)
    check(np64(st), rs, TOL_F32, "step state")


def test_step_wide_rows_and_strides():
    """Many rows, token rows taken from a wider projection."""
    n, Hk, H, K, V = 64, 4, 16, 64, 50
    c, st = _case(60, n, 1, Hk, H, K, V, torch.bfloat16)
    wide = torch.full((n, 2 * Hk * K + H * V + 8), float("nan"), device=DEV, dtype=torch.bfloat16)
    wide[:, :Hk * K] = c["q"].flatten(1)
    wide[:, Hk * K:2 * Hk * K] = c["k"].flatten(1)
    wide[:, 2 * Hk * K:2 * Hk * K + H * V] = c["v"].flatten(1)
    ro, rs = _ref(c, st)
    o = ssm.delta_decode_step(wide[:, :Hk * K].unflatten(-1, (Hk, K)), wide[:, Hk * K:2 * Hk * K].unflatten(-1, (Hk, K)),
                              wide[:, 2 * Hk * K:2 * Hk * K + H * V].unflatten(-1, (H, V)), c["g"][:, 0].contiguous(),
                              c["beta"][:, 0].contiguous(), st, o_dtype=torch.float32)
    torch.cuda.synchronize()
    check(np64(o), ro[:, 0], TOL_F32, "wide o")
    check(np64(st), rs, TOL_F32, "wide state")


def test_prefill_then_steps_equal_a_longer_prefill():
    c, st = _case(61, 2, 140, 2, 4, 64, 32)
    o, s = _run(c, st, qk_norm=True)
    a = {x: t[:, :130].contiguous() for x, t in c.items()}
    _, mid = _run(a, st, qk_norm=True)
    for t in range(130, 140):
        tok = {x: y[:, t].contiguous() for x, y in c.items()}
        ot = ssm.delta_decode_step(tok["q"], tok["k"], tok["v"], tok["g"], tok["beta"], mid, qk_norm=True)
        torch.cuda.synchronize()
        check(np64(ot), np64(o[:, t]), 2 * TOL_F32, f"token {t}")
    check(np64(mid), np64(s), 2 * TOL_F32, "state")


# ---------------------------------------------------------------- streams, graphs, long calls

def test_on_another_stream():
    c, st = _case(70, 2, 200, 2, 4, 64, 32, torch.bfloat16)
    want = _run(c, st, qk_norm=True)
    do = torch.randn_like(c["v"])
    gw = ssm.delta_chunk_bwd(c["q"], c["k"], c["v"], c["g"], c["beta"], do, qk_norm=True, state_in=st)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):  # workspaces handed back between calls must not be reused while the other stream works
        out = torch.empty_like(st)
        o = ssm.delta_chunk_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], state_in=st, state_out=out, qk_norm=True, stream=s)
        g = ssm.delta_chunk_bwd(c["q"], c["k"], c["v"], c["g"], c["beta"], do, qk_norm=True, state_in=st, stream=s)
        junk = [torch.full((1 << 20,), float("nan"), device=DEV) for _ in range(8)]
    s.synchronize()
    del junk
    assert torch.equal(o, want[0]) and torch.equal(out, want[1])
    assert all(torch.equal(g[x], gw[x]) for x in gw)


def test_packed_gradients_on_another_stream():
    """The zeros that tokens outside the sequences get are written on the call's stream too."""
    cu = [3, 70, 190]
    c, st = _case(73, 1, 200, 2, 4, 48, 40, torch.bfloat16, cu=cu)
    do = torch.randn_like(c["v"])
    want = ssm.delta_chunk_bwd(c["q"], c["k"], c["v"], c["g"], c["beta"], do, qk_norm=True, cu_seqlens=_cu(cu), state_in=st)
    for x in ("q", "k", "v", "g", "beta"):
        assert not want[x][:, :3].any() and not want[x][:, 190:].any() and want[x][:, 3:190].any()
    offsets = _cu(cu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    spin = torch.randn(4096, 4096, device=DEV)
    for _ in range(4):
        for _ in range(8):
            spin = torch.tanh(spin @ spin)  # work that keeps the current stream behind
        got = ssm.delta_chunk_bwd(c["q"], c["k"], c["v"], c["g"], c["beta"], do, qk_norm=True, cu_seqlens=offsets,
                                  state_in=st, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(got[x], want[x]) for x in want)


def test_no_sequence_at_all():
    """One offset, no sequence: nothing is read or written, gradients are zeros."""
    c, _ = _case(74, 1, 100, 1, 2, 32, 16, state=False)
    o = torch.full_like(c["v"], 5.0)
    cu = _cu([0])
    out = torch.empty((0, 2, 16, 32), device=DEV)
    ssm.delta_chunk_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], cu_seqlens=cu, o=o, state_out=out)
    g = ssm.delta_chunk_bwd(c["q"], c["k"], c["v"], c["g"], c["beta"], c["v"], cu_seqlens=cu)
    torch.cuda.synchronize()
    assert (o == 5).all() and not any(t.any() for t in g.values())


def test_graph_replays():
    """Prefill, backward and a decode step recorded in one graph, replayed with eager work between."""
    c, st = _case(71, 1, 200, 2, 4, 64, 32, torch.bfloat16)
    do = torch.randn_like(c["v"])
    dec = st.clone()
    tok = {x: t[:, 0].contiguous() for x, t in c.items()}
    out = torch.empty_like(st)
    f = ssm.delta_chunk_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], state_in=st, state_out=out, qk_norm=True, prepare=True)
    b = ssm.delta_chunk_bwd(c["q"], c["k"], c["v"], c["g"], c["beta"], do, qk_norm=True, state_in=st, prepare=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        for call in (f, b):
            call._stream = __import__("ctypes").c_void_p(s.cuda_stream)
            call.run()
        od = ssm.delta_decode_step(tok["q"], tok["k"], tok["v"], tok["g"], tok["beta"], dec, qk_norm=True, stream=s)
    eager = st.clone()
    for i in range(3):
        c["v"].normal_()
        tok["v"].normal_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        wo, ws = _run(c, st, qk_norm=True)
        gw = ssm.delta_chunk_bwd(c["q"], c["k"], c["v"], c["g"], c["beta"], do, qk_norm=True, state_in=st)
        ow = ssm.delta_decode_step(tok["q"], tok["k"], tok["v"], tok["g"], tok["beta"], eager, qk_norm=True)
        torch.cuda.synchronize()
        assert torch.equal(f.out, wo) and torch.equal(out, ws), i
        assert all(torch.equal(b.out[x], gw[x]) for x in gw), i
        assert torch.equal(od, ow) and torch.equal(dec, eager), i


def test_offsets_past_32_bits():
    """v, o and the workspace beyond 2^31 elements: the last heads equal a call on those heads alone."""
    L, H, K, V = 68000, 256, 16, 128
    gen = torch.Generator(device=DEV).manual_seed(72)
    q, k = (torch.randn((1, L, 1, K), generator=gen, device=DEV).to(torch.bfloat16) for _ in range(2))
    v = torch.randn((1, L, H, V), generator=gen, device=DEV, dtype=torch.bfloat16)
    g = -0.1 * torch.rand((1, L, H), generator=gen, device=DEV)
    beta = torch.rand((1, L, H), generator=gen, device=DEV)
    assert v.numel() > 2 ** 31
    o = ssm.delta_chunk_fwd(q, k, v, g, beta, qk_norm=True)
    a = ssm.delta_chunk_fwd(q, k, v[:, :, -2:].contiguous(), g[..., -2:].contiguous(), beta[..., -2:].contiguous(), qk_norm=True)
    torch.cuda.synchronize()
    assert torch.equal(o[:, :, -2:], a)
