"""GPU parity of attention with a sliding window and sinks (ssm_attn_fwd, ssm_attn_bwd) against the float64 oracle,
through the C ABI.

Bounds, set before the first run.  f32 inputs: products and sums in f32, scores of a few units whose error of about
D 2^-24 enters P relatively; 1e-5 of the result's largest value, as for the framework's other f32 paths.  bf16 inputs
with f32 results: P and dS keep 24 bits, the same bound.  bf16 results: P and dS keep 16 bits (2^-16 each, of values
up to a few times the result's largest: 1e-4 of that), and the result's own rounding, 2^-8 of each value."""
import numpy as np
import pytest
import torch

import selective_state_space_03_amd as ssm
from gpu_util import DEV, check, np64
from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL_F32, TOL_BF16 = 1e-5, 1e-4


def _case(seed, n, L, Lk, Hk, H, D, dtype):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV).to(dtype)  # noqa: E731
    return rnd(n, L, H, D), rnd(n, Lk, Hk, D), rnd(n, Lk, Hk, D), rnd(n, L, H, D)


def _cu(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)


def _inside(t, cu):
    """Whether a row of a packed tensor lies in a sequence."""
    if cu is None:
        return np.ones(t.shape[:2], bool)
    at = np.arange(t.shape[1])
    return np.array([[any(a <= x < b for a, b in zip(cu[:-1], cu[1:])) for x in at]])


def _run(c, out=None, cu=None, cu_k=None, grads=True, o_dtype=None, grad_dtype=None, rest=False, **kw):
    """Forward (and backward), both against the oracle; o and lse start as NaN.  rest: with what rounding took from o,
    so that the gradients are those of an exact o."""
    q, k, v, do = c
    o = torch.full(q.shape, float("nan"), dtype=o_dtype or q.dtype, device=DEV)
    lse = torch.full(q.shape[:3], float("nan"), device=DEV)
    orest = torch.full_like(o, float("nan")) if rest else None
    ssm.attn_fwd(q, k, v, lse=lse, o=o, o_rest=orest, cu_seqlens=_cu(cu), cu_seqlens_k=_cu(cu_k), **kw)
    torch.cuda.synchronize()
    ok = dict(kw, cu=cu, cu_k=cu_k)
    ok["window"] = kw.get("window") or 0
    ro, rl = A.attention(*(np64(x) for x in (q, k, v)), **ok)
    inq = _inside(q, cu)
    got, gl = np64(o), np64(lse)
    assert np.isnan(got[~inq]).all() and np.isnan(gl[~inq]).all()  # rows of no sequence are left as they were
    bf = o.dtype == BF
    check(got[inq], ro[inq], TOL_BF16 if bf else TOL_F32, "o", out_bf16=bf)
    if rest:
        assert np.isnan(np64(orest)[~inq]).all()
        check((got + np64(orest))[inq], ro[inq], TOL_BF16, "o + rest")
    none = np.isneginf(rl[inq])
    assert np.array_equal(np.isneginf(gl[inq]), none) and not got[inq][none].any()
    check(gl[inq][~none], rl[inq][~none], TOL_F32, "lse")
    if not grads:
        return
    gd = grad_dtype or q.dtype
    g = ssm.attn_bwd(q, k, v, o, lse, do, o_rest=orest, grad_dtype=gd, cu_seqlens=_cu(cu), cu_seqlens_k=_cu(cu_k), **kw)
    torch.cuda.synchronize()
    rg = A.attention_backward(*(np64(x) for x in (q, k, v, do)), o=None if rest else np64(o), **ok)
    for x in g:
        assert g[x].dtype == gd
        check(np64(g[x]), rg[x], TOL_BF16 if gd == BF else TOL_F32, "d" + x, out_bf16=gd == BF)


DTYPES = pytest.mark.parametrize("dtype", [F32, BF])


@DTYPES
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200, 333])
def test_lengths(dtype, L):
    _run(_case(L, 2, L, L, 2, 4, 64, dtype))
    _run(_case(L, 1, L, L, 1, 3, 64, dtype), window=max(1, L // 3), sinks=3)


@DTYPES
@pytest.mark.parametrize("D", [1, 7, 8, 16, 31, 32, 33, 40, 64, 66, 80, 96, 100, 127, 128])
def test_head_sizes(dtype, D):
    _run(_case(D, 1, 97, 97, 1, 2, D, dtype), window=40, sinks=2)


@DTYPES
@pytest.mark.parametrize("Hk,H", [(1, 1), (1, 7), (3, 9), (5, 5), (8, 16)])
def test_shared_heads(dtype, Hk, H):
    _run(_case(H, 2, 70, 70, Hk, H, 32, dtype), window=20, sinks=1)


@DTYPES
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (1, 70), (2, 0), (5, 200), (63, 0), (64, 4), (65, 64), (100, 65),
                                          (128, 0), (299, 3), (300, 3), (10 ** 9, 5)])
def test_masks(dtype, window, sinks):
    _run(_case(window % 1000 + sinks, 1, 300, 300, 1, 2, 64, dtype), window=window, sinks=sinks)


@DTYPES
@pytest.mark.parametrize("L,Lk", [(1, 1), (1, 100), (16, 333), (100, 101), (130, 900), (40, 30), (200, 1), (65, 64), (70, 0)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (50, 3)])
def test_more_and_fewer_keys(dtype, L, Lk, window, sinks):
    """The queries are the last positions; with fewer keys the first queries see nothing."""
    _run(_case(L + Lk, 2, L, Lk, 2, 4, 64, dtype), window=window, sinks=sinks)


PACKED = [[0, 5, 5, 70, 71, 200], [0, 200], [0, 0, 0, 64, 128, 200], [0, 130, 190]]


@DTYPES
@pytest.mark.parametrize("cu", PACKED)
@pytest.mark.parametrize("window,sinks", [(None, 0), (33, 2)])
def test_packed(dtype, cu, window, sinks):
    """Empty sequences, sequences that end inside a tile, rows behind the last one (200 in all)."""
    _run(_case(len(cu), 1, 200, 200, 2, 4, 48, dtype), cu=cu, window=window, sinks=sinks)


@DTYPES
def test_packed_keys_of_their_own(dtype):
    cu, cu_k = [0, 3, 3, 60, 100], [0, 90, 95, 130, 300]
    _run(_case(3, 1, 100, 310, 1, 4, 64, dtype), cu=cu, cu_k=cu_k, window=70, sinks=5)


@pytest.mark.parametrize("window,sinks", [(None, 0), (100, 4)])
def test_f32_results_of_bf16_inputs(window, sinks):
    """P and dS keep 24 bits where the results do."""
    _run(_case(1, 1, 300, 300, 2, 4, 128, BF), window=window, sinks=sinks, o_dtype=F32, grad_dtype=F32)
    _run(_case(2, 1, 90, 90, 1, 2, 100, F32), window=window, sinks=sinks, o_dtype=BF, grad_dtype=BF)


@DTYPES
@pytest.mark.parametrize("sinks", [1, 64, 65, 256, 257])
def test_sinks_seen_by_many_queries(dtype, sinks):
    """The sinks' tiles are cut into pieces of queries (up to four tiles, more than 512 queries)."""
    _run(_case(sinks, 2, 1300, 1300, 1, 2, 32, dtype), window=20, sinks=sinks)
    _run(_case(sinks, 1, 1300, 1300, 2, 2, 32, dtype), window=20, sinks=sinks, cu=[0, 10, 700, 700, 1290])


@DTYPES
def test_a_query_that_sees_one_key_has_no_gradient(dtype):
    """P = 1 whatever q and k are: exactly zero, also where o was rounded."""
    q, k, v, do = _case(5, 3, 1, 1, 2, 4, 64, dtype)
    lse = torch.empty(q.shape[:3], device=DEV)
    o = ssm.attn_fwd(q, k, v, lse=lse)
    assert torch.equal(o, v.repeat_interleave(2, 2))
    g = ssm.attn_bwd(q, k, v, o, lse, do)
    assert not g["q"].any() and not g["k"].any()
    q, k, v, do = _case(6, 1, 90, 90, 1, 2, 64, dtype)
    lse = torch.empty(q.shape[:3], device=DEV)
    o = ssm.attn_fwd(q, k, v, lse=lse, window=1)
    g = ssm.attn_bwd(q, k, v, o, lse, do, window=1)
    assert not g["q"].any() and not g["k"].any()


@DTYPES
def test_slices_of_a_projection(dtype):
    """q, k and v side by side in one tensor, at an odd offset too."""
    H, Hk, D, L = 4, 2, 64, 150
    for extra in (0, 1, 3):
        w = (H + 2 * Hk) * D
        x = torch.randn(1, L, w + extra, device=DEV).to(dtype)
        x = x[..., extra:]
        q, k, v = x[..., :H * D].unflatten(-1, (H, D)), x[..., H * D:(H + Hk) * D].unflatten(-1, (Hk, D)), x[..., (H + Hk) * D:].unflatten(-1, (Hk, D))
        _run((q, k, v, torch.randn(1, L, H, D, device=DEV).to(dtype)), window=30, sinks=1)


@DTYPES
def test_large_scores(dtype):
    """Scores of hundreds: one key takes a row, the others vanish; a new maximum moves by steps."""
    q, k, v, do = _case(9, 1, 200, 200, 1, 2, 64, dtype)
    k = k * (torch.arange(200, device=DEV)[None, :, None, None] * 0.05 + 1).to(dtype)
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    ssm.attn_fwd(q, k, v, lse=lse, o=o, scale=1.0)
    ro, rl = A.attention(np64(q), np64(k), np64(v), scale=1.0)
    # a score s of 64 products is off by 64 |q||k| 2^-24, of |q||k| <= 64 * 11 here: P by 64 * 700 * 6e-8 = 2.7e-3 at most
    check(np64(o), ro, 3e-3, "o", out_bf16=dtype == BF)
    check(np64(lse), rl, TOL_F32, "lse")


@DTYPES
def test_infinities_and_nan_in_rows_that_nobody_sees(dtype):
    """Keys and values of other sequences, and behind the last one, never reach a query."""
    q, k, v, do = _case(11, 1, 200, 200, 1, 2, 64, dtype)
    cu = [0, 70, 150]
    o1, l1 = torch.zeros_like(q), torch.zeros(q.shape[:3], device=DEV)
    ssm.attn_fwd(q, k, v, o=o1, lse=l1, cu_seqlens=_cu(cu))
    g1 = ssm.attn_bwd(q, k, v, o1, l1, do, cu_seqlens=_cu(cu))
    for bad in (float("nan"), float("inf")):
        k2, v2, q2, d2 = k.clone(), v.clone(), q.clone(), do.clone()
        for t in (k2, v2, q2, d2):
            t[:, 70:150] = bad
            t[:, 150:] = bad
        o2, l2 = torch.zeros_like(q), torch.zeros(q.shape[:3], device=DEV)
        ssm.attn_fwd(q2, k2, v2, o=o2, lse=l2, cu_seqlens=_cu(cu))
        g2 = ssm.attn_bwd(q2, k2, v2, o2, l2, d2, cu_seqlens=_cu(cu))
        assert torch.equal(o1[:, :70], o2[:, :70]) and torch.equal(l1[:, :70], l2[:, :70])
        assert not o2[:, 150:].any()
        for x in g1:
            assert torch.equal(g1[x][:, :70], g2[x][:, :70])


def test_offsets_out_of_range_are_clamped():
    q, k, v, do = _case(12, 1, 100, 100, 1, 1, 32, BF)
    lse = torch.zeros(q.shape[:3], device=DEV)
    for cu in ([-5, 40, 300], [0, 90, 20, 100], [50, 10, 2 ** 31 - 1]):
        o = ssm.attn_fwd(q, k, v, lse=lse, cu_seqlens=_cu(cu), window=9, sinks=2)
        ssm.attn_bwd(q, k, v, o, lse, do, cu_seqlens=_cu(cu), window=9, sinks=2)
    torch.cuda.synchronize()


def test_repeats_bit_for_bit():
    q, k, v, do = _case(13, 2, 700, 700, 2, 6, 64, BF)
    def once():
        lse = torch.empty(q.shape[:3], device=DEV)
        o = ssm.attn_fwd(q, k, v, lse=lse, window=100, sinks=4)
        return [o, lse, *ssm.attn_bwd(q, k, v, o, lse, do, window=100, sinks=4).values()]
    first = once()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, once()))


def test_gradients_against_differences():
    """d(sum o do) along a random direction of each input, by central differences of the forward in f32."""
    q, k, v, do = _case(14, 1, 60, 75, 2, 4, 32, F32)
    kw = dict(window=20, sinks=3)
    lse = torch.empty(q.shape[:3], device=DEV)
    o = ssm.attn_fwd(q, k, v, lse=lse, **kw)
    g = ssm.attn_bwd(q, k, v, o, lse, do, **kw)
    ins = {"q": q, "k": k, "v": v}
    for x in ins:
        d = torch.randn_like(ins[x])
        f = lambda e: (ssm.attn_fwd(**{**ins, x: ins[x] + e * d}, **kw).double() * do.double()).sum().item()  # noqa: E731
        h = 1e-2
        num, ana = (f(h) - f(-h)) / (2 * h), (g[x].double() * d.double()).sum().item()
        # the third derivative's term h^2 / 6 and the forward's 1e-6 / h of a sum of 60 * 4 * 32 values of order 1
        assert abs(num - ana) <= 2e-2 * max(1.0, abs(ana)), (x, num, ana)


def test_another_stream_and_a_graph():
    """A forward and backward on a stream of their own, and replayed from a graph; eager work in between."""
    q, k, v, do = _case(15, 1, 300, 300, 2, 4, 64, BF)
    kw = dict(window=50, sinks=2)
    lse = torch.empty(q.shape[:3], device=DEV)
    o = ssm.attn_fwd(q, k, v, lse=lse, **kw)
    want = [o, lse, *ssm.attn_bwd(q, k, v, o, lse, do, **kw).values()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lse2 = torch.empty_like(lse)
    s.wait_stream(torch.cuda.current_stream())
    o2 = ssm.attn_fwd(q, k, v, lse=lse2, stream=s, **kw)
    g2 = ssm.attn_bwd(q, k, v, o2, lse2, do, stream=s, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, [o2, lse2, *g2.values()]))
    x = [t.clone() for t in (q, k, v, do)]
    lse3 = torch.zeros_like(lse)
    with torch.cuda.stream(s):  # (the allocations of the capture come from a warm-up)
        ssm.attn_bwd(*x[:3], ssm.attn_fwd(*x[:3], lse=lse3, **kw), lse3, x[3], **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3 = ssm.attn_fwd(*x[:3], lse=lse3, **kw)
        g3 = ssm.attn_bwd(*x[:3], o3, lse3, x[3], **kw)
    for i in range(3):
        for t, u in zip(x, (q, k, v, do)):
            t.copy_(u * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        le = torch.empty_like(lse)
        e = ssm.attn_fwd(*x[:3], lse=le, **kw)
        ge = ssm.attn_bwd(*x[:3], e, le, x[3], **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([o3, lse3, *g3.values()], [e, le, *ge.values()])), i


@pytest.mark.parametrize("D", [24, 64, 96, 128])
@pytest.mark.parametrize("window,sinks", [(None, 0), (70, 3), (1, 2)])
def test_forward_of_many_workgroups(D, window, sinks):
    """Whole sequences and packed ones, empty ones among them, that fill the GPU (512 workgroups of 128 queries)."""
    _run(_case(D, 8, 200, 200, 4, 32, D, BF), grads=False, window=window, sinks=sinks)
    cu = [0, 300, 300, 429, 430, 900, 1156, 1190]
    _run(_case(D, 1, 1200, 1200, 4, 40, D, BF), grads=False, window=window, sinks=sinks, cu=cu)


@pytest.mark.parametrize("D", [24, 64, 96, 128])
@pytest.mark.parametrize("window,sinks", [(None, 0), (1100, 3)])
def test_few_queries_of_many_keys(D, window, sinks):
    for L, Lk in ((1, 1024), (60, 1500), (130, 2049), (1500, 1400)):
        _run(_case(L, 1, L, Lk, 1, 2, D, BF), grads=False, window=window, sinks=sinks)
    _run(_case(D, 1, 200, 4000, 1, 3, D, BF), grads=False, window=window, sinks=sinks, cu=[0, 1, 1, 130, 190], cu_k=[0, 1500, 1502, 1520, 3900])


@pytest.mark.parametrize("D", [24, 64, 96, 128])
@pytest.mark.parametrize("n,Hk,H", [(4, 2, 4), (1, 1, 3), (1, 3, 3)])
def test_gradients_over_many_tiles(D, n, Hk, H):
    """Shared heads in pairs and odd ones, key heads that fall evenly on the XCDs and not, more queries than a workgroup."""
    for window, sinks in ((None, 0), (150, 70)):
        _run(_case(D + H, n, 400, 400, Hk, H, D, BF), window=window, sinks=sinks)
    _run(_case(D, 1, 700, 800, Hk, H, D, BF), window=100, sinks=5, cu=[0, 300, 301, 690], cu_k=[0, 400, 401, 790])


@DTYPES
@pytest.mark.parametrize("scale", [0.0, 1e-20, 1e-4])
def test_small_scales(dtype, scale):
    """Scores that vanish: P averages the visible values."""
    _run(_case(3, 1, 150, 150, 1, 2, 64, dtype), window=40, sinks=2, scale=scale)


@pytest.mark.parametrize("D", [40, 64, 66, 96, 127, 128])
def test_gradients_of_an_exact_o(D):
    """With what rounding took from o, narrow, wide and long kernels: gradients as of an o in 64 bits."""
    _run(_case(D, 2, 90, 90, 2, 4, D, BF), rest=True, window=30, sinks=2)
    _run(_case(D, 1, 200, 200, 1, 3, D, BF), rest=True, cu=[0, 1, 14, 14, 150, 190])
    _run(_case(D, 8, 200, 200, 4, 32, D, BF), rest=True, grads=False)
    _run(_case(D, 1, 60, 1500, 1, 2, D, BF), rest=True)


@DTYPES
def test_no_queries(dtype):
    """Keys that no query sees have gradients of zero."""
    q, k, v, do = _case(1, 2, 0, 70, 2, 4, 64, dtype)
    lse = torch.empty(q.shape[:3], device=DEV)
    o = ssm.attn_fwd(q, k, v, lse=lse, window=20, sinks=2)
    g = ssm.attn_bwd(q, k, v, o, lse, do, window=20, sinks=2, grad_dtype=dtype)
    assert o.shape == q.shape and g["q"].shape == q.shape and g["k"].shape == k.shape
    assert not g["k"].any() and not g["v"].any()


def test_two_calls_at_once():
    """Forward and backward of two inputs on two streams side by side, several times: the results of each alone."""
    cases = [_case(s, 2, 900, 900, 2, 4, 64, BF) for s in (20, 21)]
    kw = dict(window=200, sinks=4)

    def one(c, stream=None):
        lse, rest = torch.empty(c[0].shape[:3], device=DEV), torch.empty_like(c[0])
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        o = ssm.attn_fwd(*c[:3], lse=lse, o_rest=rest, stream=stream, **kw)
        return [o, lse, rest, *ssm.attn_bwd(*c[:3], o, lse, c[3], o_rest=rest, stream=stream, **kw).values()]

    want = [one(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(4):
        got = [one(c, s) for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


@pytest.mark.parametrize("D", [24, 64, 66, 96, 128])
def test_keys_split_over_workgroups(D):
    """Few queries of many keys, whose parts a second kernel joins; some parts hold no visible key, some rows see none."""
    for n, L, Lk, Hk, H, kw in ((1, 1, 8192, 1, 2, {}), (2, 5, 3000, 2, 4, {}), (1, 200, 2500, 1, 3, dict(window=2300, sinks=5)),
                                (1, 130, 5000, 2, 2, dict(window=1950, sinks=1)), (1, 2300, 2100, 1, 1, {})):
        _run(_case(L + D, n, L, Lk, Hk, H, D, BF), grads=False, rest=True, **kw)
