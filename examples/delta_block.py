"""A block of a recurrent language model built from the package's operators: projections
(linear_fwd), the gated delta rule (delta_chunk_fwd, delta_decode_step), the mixer's gated norm and
the end-of-block norm (block_norm_fwd), and the mixer's gradients (delta_chunk_bwd, block_norm_bwd).

    python examples/delta_block.py

prefills a packed batch of prompts of unlike lengths, decodes a few tokens from the states it leaves,
checks them against a prefill of the longer prompts, and takes one gradient step through the mixer.
Weights are random."""
from __future__ import annotations

import math
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_03_amd as ssm  # noqa: E402

EPS = 1e-6


@dataclass
class DeltaBlock:
    """One block: x -> norm(residual) is taken by the block before; this one turns its normalised input
    into the next block's and updates the residual stream.

    In one projection of the input, per token: q, k (key heads), v and the gate z (value heads), and two
    numbers per value head, the time step and the write strength."""

    d_model: int = 512
    key_heads: int = 2
    heads: int = 4
    d_key: int = 64
    d_value: int = 96
    seed: int = 0

    def __post_init__(self):
        dev, gen = torch.device("cuda:0"), torch.Generator(device="cuda:0").manual_seed(self.seed)
        rnd = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
        self.kw, self.vw = self.key_heads * self.d_key, self.heads * self.d_value
        # (rounded up to 8 outputs: the projection's rows stay 16-byte aligned)
        self.width = (2 * self.kw + 2 * self.vw + 2 * self.heads + 7) // 8 * 8
        bf = torch.bfloat16
        self.w_in = (rnd(self.width, self.d_model) / math.sqrt(self.d_model)).to(bf)
        self.w_out = (rnd(self.d_model, self.vw) / math.sqrt(self.vw)).to(bf)
        self.rate = torch.exp(torch.rand(self.heads, generator=gen, device=dev) * math.log(16.0))
        self.head_norm = 1.0 + 0.1 * rnd(self.d_value)
        self.res_scale = torch.full((self.d_model,), 0.5, device=dev)
        self.next_norm = 1.0 + 0.1 * rnd(self.d_model)

    def project(self, x):
        """q, k, v and z as slices of the projection (their rows are read in place), g and beta."""
        y = ssm.linear_fwd(x, self.w_in)
        kw, vw, lead = self.kw, self.vw, x.shape[:-1]
        q = y[..., :kw].unflatten(-1, (self.key_heads, self.d_key))
        k = y[..., kw:2 * kw].unflatten(-1, (self.key_heads, self.d_key))
        v = y[..., 2 * kw:2 * kw + vw].unflatten(-1, (self.heads, self.d_value))
        z = y[..., 2 * kw + vw:2 * kw + 2 * vw]
        ab = y[..., 2 * kw + 2 * vw:2 * kw + 2 * vw + 2 * self.heads].float().reshape(*lead, 2, self.heads)
        g = -self.rate * torch.nn.functional.softplus(ab[..., 0, :] - 4.0)
        return q, k, v, z, g.contiguous(), torch.sigmoid(ab[..., 1, :]).contiguous()

    def finish(self, o, z, residual):
        """Gated norm per head, output projection, residual and the next block's norm."""
        a, _ = ssm.block_norm_fwd(o.flatten(-2), z=z, norm_w=self.head_norm, eps=EPS)
        y = ssm.linear_fwd(a, self.w_out)
        return ssm.block_norm_fwd(y, residual=residual, scale=self.res_scale, out_norm_w=self.next_norm, eps=EPS)

    def prefill(self, x, residual, cu_seqlens):
        """x, residual (1, tokens, d_model) of packed prompts; returns (x', residual', state)."""
        q, k, v, z, g, beta = self.project(x)
        state = torch.empty((cu_seqlens.numel() - 1, self.heads, self.d_value, self.d_key), device=x.device)
        o = ssm.delta_chunk_fwd(q, k, v, g, beta, qk_norm=True, cu_seqlens=cu_seqlens, state_out=state)
        return (*self.finish(o, z, residual), state)

    def step(self, x, residual, state):
        """One token of each sequence: x, residual (sequences, d_model); state in place."""
        q, k, v, z, g, beta = self.project(x)
        o = ssm.delta_decode_step(q, k, v, g, beta, state, qk_norm=True)
        return self.finish(o, z, residual)

    def mixer_grads(self, x, da, cu_seqlens):
        """Gradients of sum(da * a) with respect to q, k, v, g, beta, z and the head norm's weight, where a
        is the gated norm's output (1, tokens, heads * d_value)."""
        q, k, v, z, g, beta = self.project(x)
        o = ssm.delta_chunk_fwd(q, k, v, g, beta, qk_norm=True, cu_seqlens=cu_seqlens)
        n = ssm.block_norm_bwd(o.flatten(-2), z=z, norm_w=self.head_norm, dout=da, eps=EPS, grad_dtype=torch.bfloat16)
        d = ssm.delta_chunk_bwd(q, k, v, g, beta, n["x"].unflatten(-1, (self.heads, self.d_value)), qk_norm=True,
                                cu_seqlens=cu_seqlens, grad_dtype=torch.bfloat16)
        return {**d, "z": n["z"], "head_norm": n["norm_w"]}


def main(lengths=(70, 1, 200, 33), extra=3):
    """Returns the largest difference between decoded and prefilled tokens and the gradients' names."""
    block = DeltaBlock()
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(1)
    whole = [n + extra for n in lengths]
    make = lambda *s: torch.randn(s, generator=gen, device=dev).to(torch.bfloat16)  # noqa: E731
    xs, rs = [make(n, block.d_model) for n in whole], [make(n, block.d_model) for n in whole]
    offsets = lambda ns: torch.tensor([0, *ns]).cumsum(0).to(device=dev, dtype=torch.int32)  # noqa: E731
    pack = lambda ts: torch.cat(ts).unsqueeze(0)  # noqa: E731
    want, want_res, _ = block.prefill(pack(xs), pack(rs), offsets(whole))
    _, _, state = block.prefill(pack([x[:n] for x, n in zip(xs, lengths)]), pack([r[:n] for r, n in zip(rs, lengths)]),
                                offsets(lengths))
    worst = 0.0
    ends = torch.tensor([0, *whole]).cumsum(0)
    for i in range(extra):
        x, res = (torch.stack([t[n + i] for t, n in zip(ts, lengths)]) for ts in (xs, rs))
        got, got_res = block.step(x, res, state)
        at = [int(ends[j]) + n + i for j, n in enumerate(lengths)]
        worst = max(worst, float((got.float() - want[0, at].float()).abs().max()),
                    float((got_res.float() - want_res[0, at].float()).abs().max()))
    grads = block.mixer_grads(pack(xs), make(1, sum(whole), block.vw), offsets(whole))
    torch.cuda.synchronize()
    assert all(bool(torch.isfinite(t).all()) for t in grads.values())
    return worst, sorted(grads)


if __name__ == "__main__":
    worst, names = main()
    print(f"decoded tokens match the longer prefill to {worst:.3g}; gradients of {', '.join(names)}")
