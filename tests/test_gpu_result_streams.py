"""Results of calls on a stream of their own (the binding's stream argument): their memory is neither what earlier work of
the current stream still uses, nor handed out again while work of the current stream reads them."""
import pytest
import torch

import selective_state_space_03_amd as ssm
from gpu_util import DEV

pytestmark = pytest.mark.gpu
NAN = float("nan")


def _rnd(*s):
    return torch.randn(s, device=DEV)


def _attn_fwd():
    q, k, v = _rnd(1, 2000, 4, 64), _rnd(1, 2000, 4, 64), _rnd(1, 2000, 4, 64)
    return lambda **kw: ssm.attn_fwd(q, k, v, window=100, **kw)


def _delta_fwd():
    q, k, v, g = _rnd(1, 2000, 4, 64), _rnd(1, 2000, 4, 64), _rnd(1, 2000, 4, 64), -torch.rand(1, 2000, 4, device=DEV)
    beta = -g
    return lambda **kw: ssm.delta_chunk_fwd(q, k, v, g, beta, qk_norm=True, **kw)


def _scan_fwd():
    x, A, B, C, dt = _rnd(2, 1000, 256), -torch.rand(256, 16, device=DEV), _rnd(2, 1000, 16), _rnd(2, 1000, 16), _rnd(2, 1000, 256)
    return lambda **kw: ssm.scan_fwd(x, A, B, C, dt, **kw)


CALLS = pytest.mark.parametrize("make", [_attn_fwd, _delta_fwd, _scan_fwd])


def _ahead(x):
    """Some tens of milliseconds of work on the current stream."""
    for _ in range(8):
        x = x @ x * 1e-2
    return x


@CALLS
def test_memory_that_the_current_stream_still_uses(make):
    run, busy, s = make(), _rnd(6144, 6144) * 1e-2, torch.cuda.Stream()
    want = run()
    _ahead(busy)
    run(stream=s)
    torch.cuda.synchronize()
    for _ in range(3):
        before = torch.empty_like(want)
        _ahead(busy)
        before.fill_(NAN)
        kept = before + 0.0
        del before
        got = run(stream=s)  # (its inputs have long been there)
        torch.cuda.synchronize()
        assert torch.isnan(kept).all() and torch.equal(got, want)
        del got


@CALLS
def test_results_that_the_current_stream_reads_later(make):
    first, second, busy, s = make(), make(), _rnd(6144, 6144) * 1e-2, torch.cuda.Stream()
    want = first()
    _ahead(busy)
    torch.cuda.synchronize()
    for _ in range(3):
        got = first(stream=s)
        torch.cuda.current_stream().wait_stream(s)
        _ahead(busy)
        copy = got + 0.0
        del got
        other = [second(stream=s) for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(copy, want)
        del other
