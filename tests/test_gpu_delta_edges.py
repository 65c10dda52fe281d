"""GPU parity of the gated delta rule at its edges, against the float64 oracle, through the C ABI.

Bounds, set before the first run: the operands of every matrix product keep 24 bits and sums are 32-bit, so a
result before its rounding is off by a few times 2^-23 per product of the longest chain, 1e-5 of the result's
largest value, whatever the inputs' type.  A bf16 result adds its own rounding, 2^-8 of each value."""
import numpy as np
import pytest
import torch

import selective_state_space_03_amd as ssm
from gpu_util import DEV, check, np64
from oracle import delta_oracle as D

pytestmark = pytest.mark.gpu
TOL = 1e-5
BF, F32 = torch.bfloat16, torch.float32
NAMES = ("q", "k", "v", "g", "beta")


def _case(seed, n, L, Hk, H, K, V, dtype, seqs=None):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    c = dict(q=rnd(n, L, Hk, K).to(dtype), k=rnd(n, L, Hk, K).to(dtype), v=rnd(n, L, H, V).to(dtype),
             g=-torch.rand((n, L, H), generator=gen, device=DEV), beta=torch.sigmoid(rnd(n, L, H)))
    return c, rnd(seqs or n, H, V, K), rnd(n, L, H, V).to(dtype), rnd(seqs or n, H, V, K)


def _args(c):
    return [c[x] for x in NAMES]


def _ref(c):
    return [np64(c[x]) for x in NAMES]


@pytest.mark.parametrize("K,V,L", [(128, 128, 700), (64, 96, 700), (100, 40, 300)])
def test_o_of_bf16_inputs_keeps_32_bits(K, V, L):
    """An f32 o carries f32 accuracy, and a bf16 o is that o rounded once."""
    c, st, _, _ = _case(K, 1, L, 1, 2, K, V, BF)
    o = ssm.delta_chunk_fwd(*_args(c), qk_norm=True, state_in=st, o_dtype=F32)
    ob = ssm.delta_chunk_fwd(*_args(c), qk_norm=True, state_in=st)
    torch.cuda.synchronize()
    ro, _ = D.delta_rule(*_ref(c), qk_norm=True, state=np64(st))
    check(np64(o), ro, TOL, "f32 o")
    assert ob.dtype == BF and torch.equal(ob, o.to(BF))


def _grads(c, do, st, ds, cu=None, **kw):
    off = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    g = ssm.delta_chunk_bwd(*_args(c), do, cu_seqlens=off, state_in=st, dstate_out=ds, **kw)
    torch.cuda.synchronize()
    return g, D.delta_rule_backward(*_ref(c), np64(do), cu=cu, state=np64(st), dstate=np64(ds), **kw)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("L,cu,Hk", [(1, None, 2), (63, None, 2), (64, None, 4), (65, None, 4), (77, None, 2),
                                     (200, [0, 1, 64, 64, 200], 2)])
def test_unit_rows_without_epsilon(dtype, L, cu, Hk):
    """qk_norm with eps = 0 is x / |x|: the rows that fill a sequence's last chunk have no length to divide by, and
    reach neither its results nor its gradients."""
    n = 2 if cu is None else 1
    c, st, do, ds = _case(L, n, L, Hk, 4, 48, 40, dtype, None if cu is None else len(cu) - 1)
    off = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    end = torch.empty_like(st)
    o = ssm.delta_chunk_fwd(*_args(c), qk_norm=True, eps=0.0, cu_seqlens=off, state_in=st, state_out=end)
    torch.cuda.synchronize()
    ro, rs = D.delta_rule(*_ref(c), qk_norm=True, eps=0.0, cu=cu, state=np64(st))
    check(np64(o), ro, TOL, "o", out_bf16=dtype == BF)
    check(np64(end), rs, TOL, "state")
    g, r = _grads(c, do, st, ds, cu, qk_norm=True, eps=0.0)
    for x in g:
        check(np64(g[x]), r[x], TOL, "d" + x)


def test_prepared_packed_gradients_follow_the_offsets():
    """A prepared backward call run again with other offsets in the same buffer: tokens that left the sequences have
    zeros, not the gradients of the run before; so too in a graph that records the call."""
    c, st, do, _ = _case(21, 1, 130, 1, 2, 32, 24, F32, seqs=2)
    cu = torch.tensor([0, 50, 130], dtype=torch.int32, device=DEV)
    call = ssm.delta_chunk_bwd(*_args(c), do, qk_norm=True, cu_seqlens=cu, state_in=st, prepare=True)
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        rec = ssm.delta_chunk_bwd(*_args(c), do, qk_norm=True, cu_seqlens=cu, state_in=st, stream=s)
    for off in ([0, 50, 130], [20, 60, 100], [0, 1, 64], [5, 5, 130]):
        cu.copy_(torch.tensor(off, dtype=torch.int32))
        graph.replay()
        got = call.run()
        want = ssm.delta_chunk_bwd(*_args(c), do, qk_norm=True, cu_seqlens=torch.tensor(off, dtype=torch.int32, device=DEV),
                                   state_in=st)
        torch.cuda.synchronize()
        for x in want:
            assert torch.equal(got[x], want[x]) and torch.equal(rec[x], want[x]), (off, x)
        for x in NAMES:
            assert not got[x][:, :off[0]].any() and not got[x][:, off[-1]:].any(), (off, x)


def test_sizes_past_31_bits_are_refused():
    """2^32 + 64 tokens or sequences (of no memory here) are not taken for 64."""
    n = (1 << 32) + 64
    q, v = torch.empty(1, 1, 1, 8, device=DEV), torch.empty(1, 1, 1, 4, device=DEV)
    g = torch.empty(1, 1, 1, device=DEV)
    for dims in ((1, n), (n, 1)):
        args = [t.expand(*dims, *t.shape[2:]) for t in (q, q, v, g, g)]
        with pytest.raises(ValueError, match="tokens, more than"):
            ssm.delta_chunk_fwd(*args)
        with pytest.raises(ValueError, match="tokens, more than"):
            ssm.delta_chunk_bwd(*args, args[2])
    one = [t[0].expand(n, *t.shape[2:]) for t in (q, q, v, g, g)]
    with pytest.raises(ValueError, match="sequences, more than"):
        ssm.delta_decode_step(*one, torch.empty(1, 1, 4, 8, device=DEV).expand(n, 1, 4, 8))
