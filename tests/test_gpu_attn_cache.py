"""GPU parity of the attention's paged cache (ssm_attn_cache_write, ssm_attn_decode_step) against the float64 oracle,
through the C ABI.

Bounds, set before the first run.  Codes and scales are equal: scales are powers of two, so the only rounding is the
one to 8 bits.  A step keeps 24 bits of every operand and f32 sums: 1e-5 of the largest value, and the rounding of an
o in bf16, 2^-8 of each value."""
import numpy as np
import pytest
import torch

import selective_state_space_03_amd as ssm
from gpu_util import DEV, check, np64
from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TOL = 1e-5
KINDS = [(F32, F32), (BF, BF), (F32, E4), (BF, E4)]


def _pool(seed, pages, hk, page, D, kind):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    out = []
    for _ in range(2):
        x = torch.randn((pages, hk, page, D), generator=gen, device=DEV)
        s = None
        if kind == E4:
            s = torch.exp2(torch.randint(-9, -5, (pages, hk), generator=gen, device=DEV).float())
            x = (x / s[..., None, None]).clamp(-448, 448)
        out.append((x.to(kind), s))
    return out


def _table(seed, held, new, page, pages, rows=None):
    """Pages of their own for every sequence, in any order; -1 past its end."""
    rows = max(1, max(-(-(a + b) // page) for a, b in zip(held, new))) if rows is None else rows
    ids = np.random.default_rng(seed).permutation(pages).astype(np.int32)
    t, at = np.full((len(held), rows), -1, np.int32), 0
    for i, (a, b) in enumerate(zip(held, new)):
        n = min(rows, -(-(a + b) // page))
        t[i, :n] = ids[at:at + n]
        at += n
    assert at <= pages
    return t


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _values(t):
    return np64(t.float())


def _write(seed, held, new, hk, page, D, dtype, kind, packed, k=None, v=None, table=None, tokens=None):
    pages = sum(-(-(a + b) // page) for a, b in zip(held, new)) + 2
    (kc, ks), (vc, vs) = _pool(seed, pages, hk, page, D, kind)
    table = _table(seed, held, new, page, pages) if table is None else table
    gen = torch.Generator(device=DEV).manual_seed(seed + 1)
    lead = (1, sum(new) if tokens is None else tokens) if packed else (len(held), new[0])
    mk = lambda: (torch.randn((*lead, hk, D), generator=gen, device=DEV) * 3).to(dtype)  # noqa: E731
    k, v = mk() if k is None else k, mk() if v is None else v
    cu = [0, *np.cumsum(new).tolist()] if packed else None
    want = []
    for x, c, s in ((k, kc, ks), (v, vc, vs)):
        want.append(A.cache_write(np64(x), _values(c), None if s is None else np64(s), table, held, cu))
    lens = _dev(held)
    got = ssm.attn_cache_write(k, v, kc, vc, _dev(table), lens, cu_seqlens=None if cu is None else _dev(cu), k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    assert got[0] is kc and got[1] is vc and lens.tolist() == list(held)
    for (c, s), (wc, ws) in zip(((kc, ks), (vc, vs)), want):
        assert np.array_equal(_values(c), wc, equal_nan=True)
        if s is not None:
            assert np.array_equal(np64(s), ws)
    return kc, vc, ks, vs


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("page", [1, 5, 16, 24, 64])
def test_write_one_token(dtype, kind, page):
    held = [0, 1, page - 1, page, page + 1, 3 * page, 4 * page - 1, 37]
    _write(page, held, [1] * len(held), 2, page, 64, dtype, kind, False)


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("page,D", [(16, 64), (64, 128), (24, 40), (7, 33), (16, 1), (128, 100)])
def test_write_packed(dtype, kind, page, D):
    """Empty sequences, sequences that begin and end inside a page, and ones that stay inside one."""
    _write(D, [0, 3, 0, page, 5 * page - 1, 2, page - 1], [200, 0, 1, 65, 2, 3 * page, 150], 3, page, D, dtype, kind, True)


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_write_whole_sequences(dtype, kind):
    _write(1, [0, 7, 30], [50, 50, 50], 2, 16, 64, dtype, kind, False)


def test_tokens_outside_every_sequence_and_pages_that_are_not_kept():
    """Tokens behind the last sequence, entries out of range, and positions past the table are not written."""
    held, new, page = [0, 20, 5], [40, 30, 100], 16
    table = _table(2, held, new, page, 14, rows=4)
    table[0, 1], table[1, 2], table[2, 0] = -1, 14 + 9, -7
    _write(2, held, new, 2, page, 32, BF, E4, True, table=table, tokens=200)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_scales_follow_growing_values(dtype):
    """Token by token with growing values: the scale of a page grows, its codes follow; a zero page has the least."""
    page, D = 8, 32
    (kc, ks), (vc, vs) = _pool(3, 3, 1, page, D, E4)
    table, wk, wv = np.array([[2, 0]], np.int32), _values(kc), _values(vc)
    sk, sv = np64(ks), np64(vs)
    gen = torch.Generator(device=DEV).manual_seed(4)
    for t in range(12):
        k = (torch.randn((1, 1, 1, D), generator=gen, device=DEV) * 1.9 ** t).to(dtype)
        v = torch.zeros_like(k) if t < 9 else k
        ssm.attn_cache_write(k, v, kc, vc, _dev(table), _dev([t]), k_scale=ks, v_scale=vs)
        wk, sk = A.cache_write(np64(k), wk, sk, table, [t])
        wv, sv = A.cache_write(np64(v), wv, sv, table, [t])
        assert np.array_equal(_values(kc), wk) and np.array_equal(np64(ks), sk)
        assert np.array_equal(_values(vc), wv) and np.array_equal(np64(vs), sv)
    assert sv[2, 0] == 2.0 ** -100


def test_values_at_the_borders_of_the_scale():
    """448 s exactly, just above, the largest and smallest numbers, infinities and NaN, ties of the rounding."""
    rows = [[448.0, 1.0], [448.0 * 2 ** 5, 3.0], [450.0, 1.0], [448.00003, 17.0], [3.4e38, -3.4e38], [1e-38, 1e-45], [float("inf"), 2.0],
            [float("nan"), -0.5], [2.0 ** -92 * 448, 2.0 ** -100], [0.0, -0.0], [17.0, 19.0], [1.0625, 448.0]]
    x = torch.tensor(rows, device=DEV).reshape(len(rows), 1, 1, 2)
    _write(5, [0] * len(rows), [1] * len(rows), 1, 4, 2, F32, E4, False, k=x, v=x.flip(-1).contiguous())


def _step(seed, lens, h, hk, page, D, dtype, kind, window=None, sinks=0, o_dtype=None, table=None, rows=None, q=None, spread=True, **kw):
    pages = sum(-(-n // page) for n in lens) + 2
    (kc, ks), (vc, vs) = _pool(seed, pages, hk, page, D, kind)
    table = _table(seed, lens, [0] * len(lens), page, pages, rows) if table is None else table
    gen = torch.Generator(device=DEV).manual_seed(seed + 7)
    q = torch.randn((len(lens), h, D), generator=gen, device=DEV).to(dtype) if q is None else q
    # rows that no query sees: behind the last token, behind the window, in pages of nobody
    seen = np.zeros((pages, page), bool)
    for i, n in enumerate(lens):
        j = np.arange(min(max(n, 0), table.shape[1] * page))
        if window:
            j = j[(j >= len(j) - window) | (j < sinks)]
        at = table[i, j // page]
        fine = (at >= 0) & (at < pages)
        seen[at[fine], (j % page)[fine]] = True
    hide = torch.tensor(~seen, device=DEV)[:, None, :, None].expand(kc.shape)
    for c in (kc, vc):
        c.view(torch.uint8 if kind == E4 else c.dtype)[hide] = 0x7f if kind == E4 else float("nan")
    o = torch.full((len(lens), h, D), float("nan"), dtype=o_dtype or dtype, device=DEV)
    ssm.attn_decode_step(q, kc, vc, _dev(table), _dev(lens), k_scale=ks, v_scale=vs, window=window, sinks=sinks, o=o, **kw)
    torch.cuda.synchronize()
    want = A.decode_step(np64(q), _values(kc), _values(vc), table, lens, k_scale=None if ks is None else np64(ks),
                         v_scale=None if vs is None else np64(vs), window=window or 0, sinks=sinks, scale=kw.get("scale"))
    check(np64(o), want, TOL, "o", out_bf16=o.dtype == BF)


STEPS = KINDS + [(F32, BF)]


@pytest.mark.parametrize("dtype,kind", STEPS)
@pytest.mark.parametrize("page,D", [(1, 32), (16, 64), (24, 40), (64, 128), (7, 33), (128, 100), (16, 1), (33, 96)])
def test_step(dtype, kind, page, D):
    _step(page + D, [1, 2, 15, 33, 0, 128, 300], 4, 2, page, D, dtype, kind)


@pytest.mark.parametrize("dtype,kind", STEPS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (100, 3), (31, 64), (299, 1), (300, 0), (10 ** 9, 2)])
def test_step_masks(dtype, kind, window, sinks):
    _step(window % 997, [300, 1, 64, 130], 4, 2, 16, 64, dtype, kind, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype,kind", STEPS)
@pytest.mark.parametrize("scale", [0.0, 1e-20])
def test_step_small_scales(dtype, kind, scale):
    """The mean of the visible values."""
    _step(3, [300, 1, 64, 0], 4, 2, 16, 64, dtype, kind, window=50, sinks=3, scale=scale)


@pytest.mark.parametrize("dtype,kind", STEPS)
@pytest.mark.parametrize("hk,h", [(1, 1), (1, 16), (1, 17), (2, 80), (3, 15)])
def test_step_shared_heads(dtype, kind, hk, h):
    _step(h, [100, 41], h, hk, 16, 64, dtype, kind, window=64, sinks=2)


@pytest.mark.parametrize("dtype,kind", STEPS)
def test_step_parts(dtype, kind):
    """Long sequences are cut into parts that a second kernel joins; short ones beside them leave most empty."""
    _step(1, [5000, 3, 0, 257, 2048], 8, 2, 64, 128, dtype, kind)
    _step(2, [5000, 3, 700], 2, 1, 16, 64, dtype, kind, window=1500, sinks=9)


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_step_results_in_the_other_type(dtype, kind):
    _step(4, [90, 1000], 4, 2, 32, 64, dtype, kind, o_dtype=BF if dtype == F32 else F32)


def test_step_pages_out_of_range_and_lengths_past_the_table():
    """Keys in pages out of range are left out; a length past the table counts as the table's; below zero as zero."""
    lens, page = [100, 64, 1000, -3, 50], 16
    table = _table(8, [100, 64, 64, 1, 50], [0] * 5, page, 20, rows=7)
    table[0, 2], table[0, 6], table[1, :] = -1, 20 + 5, 2 ** 31 - 1
    _step(8, [100, 64, 64, 1, 50], 4, 2, page, 64, BF, E4, table=table)
    table[2, 4:] = -1
    (kc, ks), (vc, vs) = _pool(9, 20, 2, page, 64, E4)
    q = torch.randn(5, 4, 64, device=DEV).to(BF)
    o = ssm.attn_decode_step(q, kc, vc, _dev(table), _dev(lens), k_scale=ks, v_scale=vs)
    want = A.decode_step(np64(q), _values(kc), _values(vc), table, lens, k_scale=np64(ks), v_scale=np64(vs))
    check(np64(o), want, TOL, "o", out_bf16=True)
    assert not o[1].any() and not o[3].any()


def test_step_q_inside_a_projection():
    for extra in (0, 3):
        x = torch.randn(3, 6 * 64 + extra + 10, device=DEV).to(BF)
        _step(5, [70, 20, 33], 6, 2, 16, 64, BF, BF, q=x[:, extra:extra + 6 * 64].unflatten(-1, (6, 64)))


def test_offsets_past_32_bits():
    """A pool of more than 2^32 elements: the last pages are read and written where they are."""
    pages, hk, page, D = 2 ** 20 + 3, 1, 32, 130 - 2
    kc = torch.zeros((pages, hk, page, D), dtype=BF, device=DEV)
    vc = torch.zeros_like(kc)
    assert kc.numel() > 2 ** 32
    table = np.array([[pages - 1, 0, pages - 2]], np.int32)
    k, v = (torch.randn((1, 90, hk, D), device=DEV).to(BF) for _ in range(2))
    ssm.attn_cache_write(k, v, kc, vc, _dev(table), _dev([0]))
    assert torch.equal(kc[pages - 1, 0], k[0, :32, 0]) and torch.equal(vc[pages - 2, 0, :26], v[0, 64:, 0])
    q = torch.randn((1, 2, D), device=DEV).to(BF)
    o = ssm.attn_decode_step(q, kc, vc, _dev(table), _dev([90]))
    ro, _ = A.attention(np64(q)[:, None], np64(k), np64(v))
    check(np64(o), ro[:, 0], TOL, "o", out_bf16=True)


def test_prefill_write_and_steps_equal_the_whole_sequence():
    """A prompt's attention, its keys and values into the cache, then token by token: the rows of one call over the
    whole sequence (a cache in f32 holds the values as they are)."""
    n, L, more, h, hk, D, page = 2, 70, 20, 4, 2, 64, 16
    q, k, v = (torch.randn((n, L + more, x, D), device=DEV) for x in (h, hk, hk))
    kw = dict(window=40, sinks=3)
    whole = ssm.attn_fwd(q, k, v, **kw)
    rows = -(-(L + more) // page)
    table = _dev(np.random.default_rng(0).permutation(n * rows + 3)[:n * rows].reshape(n, rows))
    kc, vc = (torch.full((n * rows + 3, hk, page, D), float("nan"), device=DEV) for _ in range(2))
    lens = _dev([0] * n)
    ssm.attn_cache_write(k[:, :L].contiguous(), v[:, :L].contiguous(), kc, vc, table, lens)
    lens += L
    for t in range(L, L + more):
        ssm.attn_cache_write(k[:, t:t + 1].contiguous(), v[:, t:t + 1].contiguous(), kc, vc, table, lens)
        lens += 1
        o = ssm.attn_decode_step(q[:, t].contiguous(), kc, vc, table, lens, **kw)
        check(np64(o), np64(whole[:, t]), 2 * TOL, f"token {t}")


@pytest.mark.parametrize("kind", [BF, E4])
def test_step_graph_with_growing_lengths(kind):
    """A decode step (write, length, attention) captured once and replayed token by token, each replay against the
    eager step on caches of its own; two graphs with workspaces of their own in turn."""
    n, h, hk, D, page, start = 3, 8, 2, 64, 16, 1000
    rows = -(-(start + 40) // page)
    table = _dev(np.random.default_rng(1).permutation(n * rows).reshape(n, rows))

    def state():
        (kc, ks), (vc, vs) = _pool(6, n * rows, hk, page, D, kind)
        return dict(kc=kc, vc=vc, ks=ks, vs=vs, lens=_dev([start, 5, 600]), q=torch.zeros(n, h, D, dtype=BF, device=DEV),
                    k=torch.zeros(n, 1, hk, D, dtype=BF, device=DEV), v=torch.zeros(n, 1, hk, D, dtype=BF, device=DEV))

    def step(s):
        ssm.attn_cache_write(s["k"], s["v"], s["kc"], s["vc"], table, s["lens"], k_scale=s["ks"], v_scale=s["vs"])
        s["lens"].add_(1)
        return ssm.attn_decode_step(s["q"], s["kc"], s["vc"], table, s["lens"], k_scale=s["ks"], v_scale=s["vs"], window=700, sinks=4)

    eager, graphs = state(), []
    for _ in range(2):
        s = state()
        warm = state()
        step(warm)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = step(s)
        graphs.append((g, s, o))
    gen = torch.Generator(device=DEV).manual_seed(3)
    for t in range(6):
        new = [torch.randn(eager[x].shape, generator=gen, device=DEV).to(BF) for x in ("q", "k", "v")]
        for s in (eager, graphs[0][1], graphs[1][1]):
            for x, y in zip(("q", "k", "v"), new):
                s[x].copy_(y)
        for g, _, _ in graphs:
            g.replay()
        want = step(eager)
        torch.cuda.synchronize()
        for _, s, o in graphs:
            assert torch.equal(o, want), t
            for x in ("kc", "vc"):
                a, b = (y[x].view(torch.uint8) if kind == E4 else y[x] for y in (s, eager))
                assert torch.equal(a, b), (t, x)
