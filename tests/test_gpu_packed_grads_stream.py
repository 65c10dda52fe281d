"""Packed backward calls (ssm_attn_bwd, ssm_delta_chunk_bwd) clear the rows of no sequence in the order of their stream:
neither before work that was queued ahead of the call, nor after the call's own results."""
import pytest
import torch

import selective_state_space_03_amd as ssm
from gpu_util import DEV

pytestmark = pytest.mark.gpu
F32 = torch.float32
L, END = 2000, 1700
CU = [150, 900, END]
NAN = float("nan")


def _rnd(*s):
    return torch.randn(s, device=DEV)


def _attn():
    q, k, v, do = _rnd(1, L, 4, 64), _rnd(1, L, 4, 64), _rnd(1, L, 4, 64), _rnd(1, L, 4, 64)
    cu = torch.tensor(CU, dtype=torch.int32, device=DEV)
    lse = torch.zeros(q.shape[:3], device=DEV)
    o = ssm.attn_fwd(q, k, v, lse=lse, cu_seqlens=cu, window=100)
    return lambda **kw: ssm.attn_bwd(q, k, v, o, lse, do, cu_seqlens=cu, window=100, **kw)


def _delta():
    q, k, v, do = _rnd(1, L, 4, 64), _rnd(1, L, 4, 64), _rnd(1, L, 4, 64), _rnd(1, L, 4, 64)
    g, beta = -torch.rand(1, L, 4, device=DEV), torch.rand(1, L, 4, device=DEV)
    cu = torch.tensor(CU, dtype=torch.int32, device=DEV)
    return lambda **kw: ssm.delta_chunk_bwd(q, k, v, g, beta, do, qk_norm=True, cu_seqlens=cu, **kw)


CALLS = pytest.mark.parametrize("make", [_attn, _delta])


def _ahead(x):
    """Some tens of milliseconds of work on the current stream."""
    for _ in range(8):
        x = x @ x * 1e-2
    return x


@CALLS
@pytest.mark.parametrize("on", ["default", "side", "given"])
def test_memory_that_earlier_work_still_writes(make, on):
    """Gradients come to lie where tensors lay that queued work has yet to write and read: that work reads what it
    wrote, and the rows of no sequence are zero in the end."""
    run, busy = make(), _rnd(6144, 6144) * 1e-2
    want = run()
    _ahead(busy)
    torch.cuda.synchronize()
    want = {x: t.clone() for x, t in want.items()}
    side = torch.cuda.Stream()
    given = dict(stream=torch.cuda.default_stream()) if on == "given" else {}
    with torch.cuda.stream(side if on == "side" else torch.cuda.default_stream()):
        run()  # (the allocator's blocks of this stream)
        torch.cuda.synchronize()
        for _ in range(3):
            before = {x: torch.empty_like(t) for x, t in want.items()}
            at = {t.data_ptr() for t in before.values()}
            _ahead(busy)
            for t in before.values():
                t.fill_(NAN)
            kept = {x: t + 0.0 for x, t in before.items()}
            del before, t
            got = run(**given)
            assert at & {t.data_ptr() for t in got.values()}, "the gradients lie elsewhere: nothing is tested"
            torch.cuda.synchronize()
            assert all(torch.isnan(t).all() for t in kept.values())
            for x, t in got.items():
                assert torch.equal(t, want[x]), x
                assert not t[:, :CU[0]].any() and not t[:, END:].any(), x
            del got, t, kept


@CALLS
def test_a_prepared_call_behind_queued_work(make):
    """run() of a prepared call, again and again while earlier work runs: each the results of a call alone."""
    run, busy = make(), _rnd(6144, 6144) * 1e-2
    call = run(prepare=True)
    want = {x: t.clone() for x, t in call.run().items()}
    for _ in range(3):
        _ahead(busy)
        for t in call.out.values():
            t.fill_(NAN)
        got = call.run()
        copy = {x: t.clone() for x, t in got.items()}
        torch.cuda.synchronize()
        for x in want:
            assert torch.equal(got[x], want[x]) and torch.equal(copy[x], want[x]), x


@pytest.mark.parametrize("grad_dtype", [F32, torch.bfloat16])
def test_rows_of_no_sequence_in_both_types(grad_dtype):
    """Gradients in bf16 beside ones that stay f32 (the delta rule's g and beta), and calls without any token."""
    for make in (_attn, _delta):
        got = make()(grad_dtype=grad_dtype)
        torch.cuda.synchronize()
        assert got["q"].dtype == grad_dtype
        for x, t in got.items():
            assert not t[:, :CU[0]].any() and not t[:, END:].any() and torch.isfinite(t).all() and t.any(), x
    cu = torch.zeros(3, dtype=torch.int32, device=DEV)
    q = torch.empty(1, 0, 2, 16, device=DEV)
    g = ssm.attn_bwd(q, q, q, q, q[..., 0], q, cu_seqlens=cu, grad_dtype=grad_dtype)
    assert all(t.shape == q.shape for t in g.values())
    g = ssm.delta_chunk_bwd(q, q, q, q[..., 0], q[..., 0], q, cu_seqlens=cu, grad_dtype=grad_dtype)
    assert g["k"].shape == q.shape and g["beta"].shape == q.shape[:3]
    torch.cuda.synchronize()
