"""Where a NaN or an infinity in the window attention's inputs may reach (ssm_attn_fwd, ssm_attn_bwd): a row of v only the queries of
tiles (of 128 from the sequence's first query on) in which some query sees it, a row of k only the queries that see it.

With v, everything else has to equal the result of clean inputs bit for bit: a hidden pair adds an exact zero.  With k,
the scores of other queries may change when a row's running maximum moves: f32 1e-5 of the largest value, bf16 16 bits of
P (1e-4) and the rounding of both results, 2^-8 of each value."""
import pytest
import torch

import selective_state_space_03_amd as ssm
from gpu_util import DEV, check, np64
from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


def _case(seed, n, L, Lk, Hk, H, D, dtype):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV).to(dtype)  # noqa: E731
    return rnd(n, L, H, D), rnd(n, Lk, Hk, D), rnd(n, Lk, Hk, D), rnd(n, L, H, D)


def _visible(L, Lk, window, sinks):
    return torch.from_numpy(A.visible(L, Lk, window or 0, sinks))


# (sequences, queries, keys, key heads, heads, channels, types of q and o, window, sinks): the kernels for f32, for rows
# that are not aligned, for results in f32, for many workgroups, for few queries of many keys, for keys in parts
CASES = [
    (1, 1, 100, 1, 2, 64, F32, None, 50, 0), (1, 1, 100, 1, 2, 64, BF, None, 50, 0), (1, 300, 300, 1, 2, 64, F32, None, 40, 4),
    (1, 300, 305, 2, 4, 66, F32, None, 40, 4), (1, 300, 300, 1, 2, 40, BF, None, 40, 4), (1, 300, 331, 2, 4, 66, BF, None, 45, 70),
    (1, 300, 303, 1, 2, 128, BF, F32, 70, 5), (2, 150, 161, 1, 1, 64, BF, None, None, 0), (1, 290, 290, 1, 2, 64, BF, None, 10, 9),
    (8, 200, 207, 4, 32, 64, BF, None, 50, 3), (8, 200, 200, 4, 32, 128, BF, None, 33, 0), (4, 400, 433, 4, 32, 96, BF, None, 130, 65),
    (8, 150, 170, 4, 32, 32, BF, None, None, 0), (8, 200, 220, 4, 32, 64, BF, None, 7, 5),
    (1, 130, 1501, 1, 2, 64, BF, None, 1100, 3), (1, 300, 1707, 1, 2, 128, BF, None, 1024, 65), (1, 260, 1290, 1, 2, 96, BF, None, None, 0),
    (1, 5, 3000, 2, 4, 64, BF, None, 2300, 5), (1, 130, 5000, 2, 2, 128, BF, None, 1950, 1),
]


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_rows_of_v_that_no_query_of_a_tile_sees(case, bad):
    n, L, Lk, Hk, H, D, dtype, o_dtype, window, sinks = case
    q, k, v, _ = _case(L + Lk, n, L, Lk, Hk, H, D, dtype)
    kw = dict(window=window, sinks=sinks, o_dtype=o_dtype)
    lse = torch.empty(q.shape[:3], device=DEV)
    want, see = ssm.attn_fwd(q, k, v, lse=lse, **kw), _visible(L, Lk, window, sinks)
    assert torch.isfinite(want).all()
    for i in range(0, L, 128):
        hidden = (~see[i:i + 128].any(0)).to(DEV)
        v2, l2 = v.clone(), torch.empty_like(lse)
        v2[:, hidden] = bad
        got = ssm.attn_fwd(q, k, v2, lse=l2, **kw)
        assert torch.equal(got[:, i:i + 128], want[:, i:i + 128]), (i, int(hidden.sum()))
        assert torch.equal(l2, lse)


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_rows_of_k_that_a_query_does_not_see(case, bad):
    n, L, Lk, Hk, H, D, dtype, o_dtype, window, sinks = case
    q, k, v, _ = _case(L + Lk, n, L, Lk, Hk, H, D, dtype)
    kw = dict(window=window, sinks=sinks, o_dtype=o_dtype)
    want, see = ssm.attn_fwd(q, k, v, **kw), _visible(L, Lk, window, sinks)
    for i in {0, L // 3, L - 1}:
        k2 = k.clone()
        k2[:, (~see[i]).to(DEV)] = bad
        got, ref = ssm.attn_fwd(q, k2, v, **kw)[:, i].double(), want[:, i].double()
        bound = 1e-5 * ref.abs().max() if want.dtype == F32 else 1e-4 * ref.abs().max() + 2.0 ** -7 * ref.abs()
        assert ((got - ref).abs() <= bound).all(), i


@pytest.mark.parametrize("dtype", [F32, BF])
def test_rows_of_v_hidden_in_packed_sequences(dtype):
    """Sequences that begin inside a tile of their neighbours, with keys of their own."""
    cu, cu_k = [0, 140, 141, 300], [0, 150, 333, 500]
    q, k, v, _ = _case(5, 1, 300, 500, 2, 4, 64, dtype)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    kw = dict(window=30, sinks=2, cu_seqlens=dev(cu), cu_seqlens_k=dev(cu_k))
    want = ssm.attn_fwd(q, k, v, **kw)
    for (a, b), (c, d) in zip(zip(cu, cu[1:]), zip(cu_k, cu_k[1:])):
        see = _visible(b - a, d - c, 30, 2)
        for i in range(0, b - a, 128):
            v2, end = torch.full_like(v, NAN), min(b, a + i + 128)
            seen = see[i:i + 128].any(0).to(DEV)
            v2[:, c:d][:, seen] = v[:, c:d][:, seen]
            assert torch.equal(ssm.attn_fwd(q, k, v2, **kw)[:, a + i:end], want[:, a + i:end]), (a, i)


def _grads(c, o, lse, kw, **new):
    q, k, v, do = (new.get(x, t) for x, t in zip(("q", "k", "v", "do"), c))
    return ssm.attn_bwd(q, k, v, o, lse, do, **kw)


# as above, with the type of the gradients: f32, rows that are not aligned, gradients in f32, aligned bf16 with sinks in
# pieces and not, two heads a workgroup and one
GRADS = [
    (1, 300, 305, 1, 2, 64, F32, F32, 40, 4), (1, 300, 300, 2, 4, 66, F32, F32, None, 0), (1, 300, 331, 1, 3, 66, BF, BF, 45, 70),
    (1, 300, 303, 1, 2, 128, BF, F32, 70, 5), (1, 600, 600, 1, 2, 64, BF, BF, 40, 4), (1, 600, 633, 1, 3, 128, BF, BF, 100, 65),
    (2, 400, 410, 2, 4, 96, BF, BF, None, 0), (1, 500, 450, 1, 1, 32, BF, BF, 33, 300), (1, 400, 407, 1, 2, 64, BF, BF, 7, 5),
]


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("case", GRADS, ids=[str(i) for i in range(len(GRADS))])
def test_gradients(case, bad):
    """A row of k reaches the dq of the queries of tiles of 256 in which some query sees it (and its own dk, dv); a row
    of q or dout the dk and dv of the tiles of 64 keys of which it sees some (and its own dq); a row of v the dq of
    the queries that see it and its own dk."""
    n, L, Lk, Hk, H, D, dtype, gd, window, sinks = case
    c = _case(L + Lk, n, L, Lk, Hk, H, D, dtype)
    mask = dict(window=window, sinks=sinks)
    lse = torch.empty(c[0].shape[:3], device=DEV)
    o, see = ssm.attn_fwd(*c[:3], lse=lse, **mask), _visible(L, Lk, window, sinks)
    kw = dict(mask, grad_dtype=gd)
    want = _grads(c, o, lse, kw)
    poisoned = lambda t, rows: t.masked_fill(rows.to(DEV)[None, :, None, None], bad)  # noqa: E731
    for i in range(0, L, 256):
        got = _grads(c, o, lse, kw, k=poisoned(c[1], ~see[i:i + 256].any(0)))
        assert torch.equal(got["q"][:, i:i + 256], want["q"][:, i:i + 256]), i
    for j in range(0, Lk, 64):
        blind = ~see[:, j:j + 64].any(1)
        for x, t in (("q", c[0]), ("do", c[3])):
            got = _grads(c, o, lse, kw, **{x: poisoned(t, blind)})
            for g in ("k", "v"):
                assert torch.equal(got[g][:, j:j + 64], want[g][:, j:j + 64]), (x, g, j)
            assert torch.equal(got["q"][:, ~blind], want["q"][:, ~blind]), (x, j)
    for i in {0, L // 2, L - 1}:
        got = _grads(c, o, lse, kw, v=poisoned(c[2], ~see[i]))
        assert torch.equal(got["q"][:, i], want["q"][:, i]) and torch.equal(got["v"], want["v"])
        assert torch.equal(got["k"][:, see[i]], want["k"][:, see[i]])
        got = _grads(c, o, lse, kw, k=poisoned(c[1], ~see[i]))
        assert torch.equal(got["k"][:, see[i]], want["k"][:, see[i]]) and torch.equal(got["v"][:, see[i]], want["v"][:, see[i]])


@pytest.mark.parametrize("dtype,D", [(BF, 40), (BF, 80), (BF, 64), (BF, 66), (F32, 40), (F32, 36), (F32, 100), (F32, 64)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_a_step_over_infinite_keys(dtype, D, sign):
    """A key whose score is -infinity vanishes from the step: infinite channels, the first and the last among them,
    against queries of the other sign there.  Cache and queries of one type."""
    lens, page, hk, h = [100, 33, 7], 16, 2, 4
    gen = torch.Generator(device=DEV).manual_seed(D)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    table = torch.randperm(21, generator=gen, device=DEV).to(torch.int32).view(3, 7)
    q, kc, vc = rnd(3, h, D).to(dtype), rnd(21, hk, page, D).to(dtype), rnd(21, hk, page, D).to(dtype)
    for ch, pages in ((0, table[:, 0]), (D - 1, table[:, 1])):
        q[..., ch] = -sign * (q[..., ch].abs() + 0.5)
        kc[pages.long(), :, 3, ch] = sign * INF
    o = ssm.attn_decode_step(q, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device=DEV))
    want = A.decode_step(np64(q), np64(kc), np64(vc), table.cpu().numpy(), lens)
    check(np64(o), want, 1e-5, "o", out_bf16=dtype == BF)
