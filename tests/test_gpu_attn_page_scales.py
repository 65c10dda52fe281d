"""The attention's decode step over an 8-bit cache (ssm_attn_decode_step): scales of pages that no visible key lies in
never reach a result, whatever they hold.

Bounds as for the step's other tests, set before the first run: 24 bits of every operand and f32 sums, 1e-5 of the
largest value, and the rounding of an o in bf16, 2^-8 of each value."""
import numpy as np
import pytest
import torch

import selective_state_space_03_amd as ssm
from gpu_util import DEV, check, np64
from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TOL = 1e-5


def _step(seed, lens, h, hk, page, D, dtype, bad, drop=(), window=None, sinks=0, own_first=0):
    """Pages own_first .. belong to the sequences in a random order; drop: (sequence, table row) whose entry is -1.
    All scales of pages without a visible key are `bad`, those of page 0 (own_first > 0) among them."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    counts = [-(-n // page) for n in lens]
    pages, rows = own_first + sum(counts) + 2, max(1, max(counts))
    ids, at = own_first + rng.permutation(sum(counts)).astype(np.int32), 0
    table = np.full((len(lens), rows), -1, np.int32)
    for i, n in enumerate(counts):
        table[i, :n] = ids[at:at + n]
        at += n
    for i, r in drop:
        table[i, r] = -1 if r % 2 else pages + 3
    seen = np.zeros(pages, bool)
    for i, n in enumerate(lens):
        j = np.arange(n)
        if window:
            j = j[(j >= n - window) | (j < sinks)]
        e = table[i, j // page]
        seen[e[(e >= 0) & (e < pages)]] = True
    assert own_first == 0 or not seen[0]
    pool = []
    for _ in range(2):
        s = torch.exp2(torch.randint(-9, -5, (pages, hk), generator=gen, device=DEV).float())
        x = torch.randn((pages, hk, page, D), generator=gen, device=DEV) / s[..., None, None]
        s[torch.tensor(~seen, device=DEV)] = bad
        pool += [x.clamp(-448, 448).to(E4), s]
    kc, ks, vc, vs = pool
    q = torch.randn((len(lens), h, D), generator=gen, device=DEV).to(dtype)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    o = ssm.attn_decode_step(q, kc, vc, dev(table), dev(lens), k_scale=ks, v_scale=vs, window=window, sinks=sinks)
    torch.cuda.synchronize()
    want = A.decode_step(np64(q), np64(kc.float()), np64(vc.float()), table, lens, k_scale=np64(ks), v_scale=np64(vs),
                         window=window or 0, sinks=sinks)
    check(np64(o), want, TOL, "o", out_bf16=dtype == BF)


ANY = pytest.mark.parametrize("dtype", [F32, BF])
BAD = pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])


@ANY
@BAD
@pytest.mark.parametrize("D", [32, 40, 64, 128])
def test_lengths_that_end_inside_a_tile(dtype, bad, D):
    _step(D, [1, 31, 33, 100, 0, 7], 4, 2, 16, D, dtype, bad, own_first=1)


@ANY
@BAD
def test_entries_out_of_range_between_visible_keys(dtype, bad):
    _step(1, [96, 64, 128], 4, 2, 16, 64, dtype, bad, drop=[(0, 2), (1, 0), (2, 3), (2, 5)], own_first=1)


@ANY
@BAD
@pytest.mark.parametrize("window,sinks", [(40, 0), (33, 3), (1, 1)])
def test_pages_behind_the_window(dtype, bad, window, sinks):
    """Pages that only the window hides, page 0 among them, keep their entries and hold scales that are no numbers."""
    _step(2, [300, 161, 70], 4, 2, 24, 64, dtype, bad, window=window, sinks=sinks)
    _step(3, [300, 161, 70], 4, 2, 24, 64, dtype, bad, window=window, sinks=sinks, own_first=1)


@ANY
@BAD
def test_parts_of_long_sequences(dtype, bad):
    _step(4, [5000, 3, 2049], 8, 2, 64, 128, dtype, bad, own_first=1)
