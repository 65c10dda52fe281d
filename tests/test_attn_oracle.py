"""The attention oracle's own pins: gradients against central differences, the masks by hand, the 8-bit rounding
against torch's cast, the cache against its definition."""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as A


def _draw(seed, n, L, Lk, hk, h, d):
    rng = np.random.default_rng(seed)
    return [rng.standard_normal(s) for s in ((n, L, h, d), (n, Lk, hk, d), (n, Lk, hk, d), (n, L, h, d))]


def test_visible_by_hand():
    assert A.visible(3, 3, 0, 0).tolist() == [[1, 0, 0], [1, 1, 0], [1, 1, 1]]
    assert A.visible(4, 4, 2, 1).tolist() == [[1, 0, 0, 0], [1, 1, 0, 0], [1, 1, 1, 0], [1, 0, 1, 1]]
    assert A.visible(1, 4, 1, 0).tolist() == [[0, 0, 0, 1]]
    assert A.visible(3, 2, 0, 0).tolist() == [[0, 0], [1, 0], [1, 1]]


def test_uniform_scores_average_the_visible_values():
    q, k, v, _ = _draw(0, 1, 6, 6, 1, 1, 3)
    o, lse = A.attention(0 * q, k, v, window=3, sinks=1)
    assert np.allclose(o[0, 5, 0], v[0, [0, 3, 4, 5], 0].mean(0)) and np.isclose(lse[0, 5, 0], np.log(4))
    o, lse = A.attention(q, k[:, :0], v[:, :0])
    assert not o.any() and np.isneginf(lse).all()


@pytest.mark.parametrize("cu,cu_k,L,Lk", [(None, None, 7, 7), (None, None, 3, 8), (None, None, 6, 4), ([0, 2, 2, 7], None, 7, 7),
                                          ([0, 2, 5], [0, 6, 9], 6, 9)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (2, 1), (1, 0)])
def test_gradients_against_differences(cu, cu_k, L, Lk, window, sinks):
    n = 1 if cu else 2
    ins = dict(zip("qkv", _draw(1, n, L, Lk, 2, 4, 3)))
    do = np.random.default_rng(2).standard_normal(ins["q"].shape)
    kw = dict(window=window, sinks=sinks, cu=cu, cu_k=cu_k, scale=0.7)
    g = A.attention_backward(*ins.values(), do, **kw)
    f = lambda **c: np.nansum(A.attention(**{**ins, **c}, **kw)[0] * do)  # noqa: E731
    for x in ins:
        for at in np.random.default_rng(3).integers(0, ins[x].size, 25):
            e = np.zeros(ins[x].size)
            e[at] = 1e-5
            e = e.reshape(ins[x].shape)
            num = (f(**{x: ins[x] + e}) - f(**{x: ins[x] - e})) / 2e-5
            assert abs(num - g[x].reshape(-1)[at]) < 1e-8


def test_e4m3_is_torchs_cast():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    fin = codes[torch.isfinite(codes)].double().numpy()
    assert np.array_equal(A.e4m3(fin), fin)
    mid = np.sort(np.unique(fin))
    x = np.concatenate([(mid[1:] + mid[:-1]) / 2, np.random.default_rng(0).uniform(-448, 448, 5000),
                        np.random.default_rng(1).standard_normal(5000) * 1e-2]).astype(np.float32)
    assert np.array_equal(A.e4m3(x), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())
    assert np.isnan(A.e4m3([np.inf, np.nan])).all()


@pytest.mark.parametrize("top,want", [(448.0, 1.0), (449.0, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8), (0.875, 2.0 ** -9),
                                      (0.8750001, 2.0 ** -8), (0.0, 2.0 ** -100), (1e-40, 2.0 ** -100), (3.4e38, 2.0 ** 120)])
def test_page_scale(top, want):
    assert A.page_scale([0.0, -top, np.nan, np.inf]) == want
    assert want == 2.0 ** -100 or (top <= 448 * want and top > 224 * want)


def test_writes_in_parts_equal_one_write():
    """A cache of whole values, and one of codes whose scale does not grow: token by token as all at once."""
    rng = np.random.default_rng(4)
    k = rng.uniform(1, 2, (1, 11, 1, 4))
    k[0, ::4] = 448.0 / 256  # every page of 4 begins with its largest value, 448 2^-8
    k = np.minimum(k, 448.0 / 256)
    table = np.array([[2, 0, 3]])
    for scaled in (False, True):
        empty = np.zeros((4, 1, 4, 4)), np.zeros((4, 1)) if scaled else None
        whole, ws = A.cache_write(k, *empty, table, [0])
        c, s = empty
        for t in range(11):
            c, s = A.cache_write(k[:, t:t + 1], c, s, table, [t])
        assert np.array_equal(whole, c) and (s is None or np.array_equal(ws, s))


def test_decode_step_is_the_last_row():
    q, k, v, _ = _draw(5, 2, 13, 13, 2, 4, 3)
    table = np.array([[4, 1, 0, 6], [2, 3, 5, 7]])
    empty = np.zeros((8, 2, 4, 3))
    kc, _ = A.cache_write(k, empty, None, table, [0, 0])
    vc, _ = A.cache_write(v, empty, None, table, [0, 0])
    for kw in (dict(), dict(window=5, sinks=2)):
        o, _ = A.attention(q, k, v, **kw)
        assert np.allclose(A.decode_step(q[:, -1], kc, vc, table, [13, 13], **kw), o[:, -1])
