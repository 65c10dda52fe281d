"""The float64 oracle of the gated delta rule and the block norm, pinned on the CPU: gradients against central
differences, the recurrence against its chunk form and closed cases, the norm against hand-written sums."""
import numpy as np
import pytest

from oracle import delta_oracle as D


def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def _delta_case(seed, n=1, L=7, Hk=2, H=4, K=5, V=3):
    r = _rng(seed)
    return dict(q=r.standard_normal((n, L, Hk, K)), k=r.standard_normal((n, L, Hk, K)) * 0.5,
                v=r.standard_normal((n, L, H, V)), g=-r.uniform(0.01, 1.0, (n, L, H)), beta=r.uniform(0, 1, (n, L, H)))


@pytest.mark.parametrize("qk_norm", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_backward_against_differences(qk_norm, packed):
    c = _delta_case(1)
    r = _rng(2)
    cu = np.array([0, 3, 3, 7]) if packed else None
    n = 3 if packed else 1
    c["state"] = r.standard_normal((n, 4, 3, 5))
    do, ds = r.standard_normal(c["v"].shape), r.standard_normal(c["state"].shape)
    g = D.delta_rule_backward(c["q"], c["k"], c["v"], c["g"], c["beta"], do, qk_norm=qk_norm, cu=cu, state=c["state"],
                              dstate=ds)

    def loss(**kw):
        a = dict(c, **kw)
        o, s = D.delta_rule(a["q"], a["k"], a["v"], a["g"], a["beta"], qk_norm=qk_norm, cu=cu, state=a["state"])
        return (o * do).sum() + (s * ds).sum()

    for name in c:
        got = g["state_in" if name == "state" else name]
        for at in [tuple(r.integers(0, s) for s in c[name].shape) for _ in range(6)]:
            e = np.zeros(c[name].shape)
            e[at] = 1e-5
            num = (loss(**{name: c[name] + e}) - loss(**{name: c[name] - e})) / 2e-5
            assert abs(num - got[at]) <= 1e-7 * max(1.0, abs(num)), (name, at)


def test_chunk_form_equals_recurrence():
    """Within a chunk the corrections solve (I + L) u = beta (v - e^G k S)."""
    c = _delta_case(3, L=9, Hk=1, H=1)
    r = _rng(4)
    S0 = r.standard_normal((1, 1, 3, 5))
    o, s = D.delta_rule(c["q"], c["k"], c["v"], c["g"], c["beta"], state=S0, scale=1.0)
    q, k, v, g, b = (c[x][0, :, 0] for x in ("q", "k", "v", "g", "beta"))
    G = np.cumsum(g)
    E = np.tril(np.exp(np.tril(G[:, None] - G)))
    Lm = np.tril(b[:, None] * E * (k @ k.T), -1)
    u = np.linalg.solve(np.eye(9) + Lm, b[:, None] * (v - np.exp(G)[:, None] * (k @ S0[0, 0].T)))
    np.testing.assert_allclose(np.exp(G)[:, None] * (q @ S0[0, 0].T) + (E * (q @ k.T)) @ u, o[0, :, 0], rtol=1e-11, atol=1e-11)
    np.testing.assert_allclose(np.exp(G[-1]) * S0[0, 0] + (np.exp(G[-1] - G)[:, None] * u).T @ k, s[0, 0], rtol=1e-11, atol=1e-11)


def test_closed_cases():
    c = _delta_case(5)
    zero = dict(c, beta=np.zeros(c["beta"].shape))
    S0 = _rng(6).standard_normal((1, 4, 3, 5))
    _, s = D.delta_rule(zero["q"], zero["k"], zero["v"], zero["g"], zero["beta"], state=S0)
    np.testing.assert_allclose(s[0], S0[0] * np.exp(c["g"][0].sum(0))[:, None, None], rtol=1e-12)  # no writes: decay only
    one = dict(c, beta=np.ones(c["beta"].shape))
    o, _ = D.delta_rule(one["k"], one["k"], one["v"], one["g"], one["beta"], scale=1.0, qk_norm=True, eps=0.0)
    np.testing.assert_allclose(o, one["v"], rtol=1e-10, atol=1e-10)  # a full write is read back by its own key
    reset = dict(c, g=np.where(np.arange(7)[None, :, None] == 4, -np.inf, c["g"]))
    a, _ = D.delta_rule(*[reset[x] for x in ("q", "k", "v", "g", "beta")], state=S0)
    b, _ = D.delta_rule(*[reset[x][:, 4:] for x in ("q", "k", "v", "g", "beta")])
    np.testing.assert_allclose(a[:, 4:], b, rtol=1e-12)  # a reset forgets everything before it


NORMS = [dict(), dict(z=1, norm_w=1), dict(z=1, norm_w=1, gate_first=True), dict(norm_w=1, z=1, group_size=3),
         dict(norm_w="all", z=1, group_size=3, gate_first=True), dict(residual=1), dict(residual=1, scale=1, out_norm_w=1),
         dict(norm_w=1, z=1, residual=1, scale=1, out_norm_w=1), dict(z=1, gate_first=True, out_norm_w=1)]


@pytest.mark.parametrize("opt", NORMS, ids=[str(i) for i in range(len(NORMS))])
def test_norm_backward_against_differences(opt):
    r = _rng(7)
    rows, d = 4, 12
    n = opt.get("group_size", d)
    c = {"x": r.standard_normal((rows, d))}
    for k, v in opt.items():
        if k in ("z", "residual"):
            c[k] = r.standard_normal((rows, d))
        elif k == "norm_w":
            c[k] = r.standard_normal(d if v == "all" else n)
        elif k in ("scale", "out_norm_w"):
            c[k] = r.standard_normal(d)
    kw = {k: opt[k] for k in ("gate_first", "group_size") if k in opt}
    do, dt = r.standard_normal((rows, d)), r.standard_normal((rows, d)) if "residual" in c else None
    g = D.block_norm_backward(c["x"], dout=do, dt=dt, **{k: v for k, v in c.items() if k != "x"}, **kw)
    assert set(g) == set(c)

    def loss(a):
        out, t = D.block_norm(a["x"], **{k: v for k, v in a.items() if k != "x"}, **kw)
        return (out * do).sum() + (0.0 if dt is None else (t * dt).sum())

    for name in c:
        for at in [tuple(r.integers(0, s) for s in c[name].shape) for _ in range(6)]:
            e = np.zeros(c[name].shape)
            e[at] = 1e-5
            num = (loss(dict(c, **{name: c[name] + e})) - loss(dict(c, **{name: c[name] - e}))) / 2e-5
            assert abs(num - g[name][at]) <= 1e-7 * max(1.0, abs(num)), (name, at)


def test_norm_by_hand():
    x, z, w = np.array([[3.0, 4.0]]), np.array([[0.0, 2.0]]), np.array([1.0, 2.0])
    out, _ = D.block_norm(x, norm_w=w, z=z, eps=0.0)
    rms = np.sqrt(12.5)
    np.testing.assert_allclose(out, [[0.0, 4.0 / rms * 2.0 * 2.0 / (1 + np.exp(-2.0))]], rtol=1e-14)
    out, t = D.block_norm(x, residual=np.array([[1.0, -1.0]]), scale=np.array([0.5, 2.0]), out_norm_w=w, eps=0.0)
    np.testing.assert_allclose(t, [[2.5, 7.0]])
    np.testing.assert_allclose(out, t * w / np.sqrt((2.5 ** 2 + 49) / 2), rtol=1e-14)
