"""Float64 oracle of the gated delta rule and the block norm (test infrastructure
only; shares nothing with the HIP path).

Per sequence and head, state S (V, K):
    S <- e^{g_t} S;  u_t = beta_t (v_t - S k_t);  S <- S + u_t k_t^T;  o_t = scale S q_t
taken token by token, and its reverse, derived from those four lines."""
from __future__ import annotations

import numpy as np


def _unit(x, eps):
    r = 1.0 / np.sqrt((x * x).sum(-1, keepdims=True) + eps)
    return x * r, r


def _bounds(q, cu):
    n, L = q.shape[:2]
    if cu is None:
        return [(b, 0, L) for b in range(n)]
    return [(0, int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


def delta_rule(q, k, v, g, beta, *, scale=None, qk_norm=False, eps=1e-6, cu=None, state=None, keep=None):
    """o (batch, L, H, V) and the final states (sequences, H, V, K).  keep: a list that receives, per
    sequence, the states before each token and after the last."""
    q, k, v, g, beta = (np.asarray(t, np.float64) for t in (q, k, v, g, beta))
    H, K, V = v.shape[2], q.shape[3], v.shape[3]
    rep = H // q.shape[2]
    scale = K ** -0.5 if scale is None else scale
    if qk_norm:
        q, k = _unit(q, eps)[0], _unit(k, eps)[0]
    q, k = np.repeat(q, rep, 2), np.repeat(k, rep, 2)
    seqs = _bounds(q, cu)
    o = np.zeros(v.shape)
    out = np.zeros((len(seqs), H, V, K))
    for i, (b, t0, t1) in enumerate(seqs):
        S = np.zeros((H, V, K)) if state is None else np.asarray(state[i], np.float64).copy()
        kept = [S]
        for t in range(t0, t1):
            S = S * np.exp(g[b, t])[:, None, None]
            u = beta[b, t][:, None] * (v[b, t] - np.einsum("hvk,hk->hv", S, k[b, t]))
            S = S + u[:, :, None] * k[b, t][:, None, :]
            o[b, t] = scale * np.einsum("hvk,hk->hv", S, q[b, t])
            kept.append(S)
        out[i] = S
        if keep is not None:
            keep.append(kept)
    return o, out


def delta_rule_backward(q, k, v, g, beta, do, *, scale=None, qk_norm=False, eps=1e-6, cu=None, state=None,
                        dstate=None):
    """Gradients of sum(do * o) + sum(dstate * final state): a dict named after the inputs."""
    q, k, v, g, beta, do = (np.asarray(t, np.float64) for t in (q, k, v, g, beta, do))
    Hk, H, K = q.shape[2], v.shape[2], q.shape[3]
    rep = H // Hk
    scale = K ** -0.5 if scale is None else scale
    keep = []
    delta_rule(q, k, v, g, beta, scale=scale, qk_norm=qk_norm, eps=eps, cu=cu, state=state, keep=keep)
    qn, rq = _unit(q, eps) if qk_norm else (q, None)
    kn, rk = _unit(k, eps) if qk_norm else (k, None)
    qh, kh = np.repeat(qn, rep, 2), np.repeat(kn, rep, 2)
    dq, dk = np.zeros(qh.shape), np.zeros(kh.shape)
    dv, dg, db = np.zeros(v.shape), np.zeros(g.shape), np.zeros(beta.shape)
    ds = np.zeros((len(keep), H, v.shape[3], K))
    for i, (b, t0, t1) in enumerate(_bounds(q, cu)):
        D = np.zeros(ds[i].shape) if dstate is None else np.asarray(dstate[i], np.float64).copy()
        for t in range(t1 - 1, t0 - 1, -1):
            before, after = keep[i][t - t0], keep[i][t - t0 + 1]
            a = np.exp(g[b, t])[:, None, None]
            E = a * before
            miss = v[b, t] - np.einsum("hvk,hk->hv", E, kh[b, t])
            u = beta[b, t][:, None] * miss
            dq[b, t] = scale * np.einsum("hvk,hv->hk", after, do[b, t])
            D = D + scale * do[b, t][:, :, None] * qh[b, t][:, None, :]
            du = np.einsum("hvk,hk->hv", D, kh[b, t])
            dk[b, t] = np.einsum("hvk,hv->hk", D, u)
            db[b, t] = (du * miss).sum(-1)
            dv[b, t] = beta[b, t][:, None] * du
            dk[b, t] -= np.einsum("hvk,hv->hk", E, dv[b, t])
            D = D - dv[b, t][:, :, None] * kh[b, t][:, None, :]
            dg[b, t] = (D * E).sum((1, 2))
            D = D * a
        ds[i] = D
    fold = lambda x: x.reshape(*x.shape[:2], Hk, rep, K).sum(3)  # noqa: E731
    dq, dk = fold(dq), fold(dk)
    if qk_norm:
        dq = rq * (dq - qn * (qn * dq).sum(-1, keepdims=True))
        dk = rk * (dk - kn * (kn * dk).sum(-1, keepdims=True))
    return {"q": dq, "k": dk, "v": dv, "g": dg, "beta": db, "state_in": ds}


def _gate(z):
    s = 1.0 / (1.0 + np.exp(-z))
    return z * s, s


def block_norm(x, *, norm_w=None, z=None, gate_first=False, residual=None, scale=None, out_norm_w=None,
               group_size=None, eps=1e-6, parts=None):
    """(out, t): out = norm(t) out_norm_w, t = residual + scale a.  parts: a dict that receives the values
    the backward needs."""
    x = np.asarray(x, np.float64)
    rows, d = x.shape
    n = group_size or d
    y = x if not gate_first else x * _gate(np.asarray(z, np.float64))[0]
    a, inv = y, np.ones((rows, d))
    w = np.ones(d)
    if norm_w is not None:
        w = np.resize(np.asarray(norm_w, np.float64), d)
        r = 1.0 / np.sqrt((y.reshape(rows, -1, n) ** 2).mean(-1) + eps)
        inv = np.repeat(r, n, 1)
        a = y * inv * w
    gated = a if z is None or gate_first else a * _gate(np.asarray(z, np.float64))[0]
    t = gated if scale is None else gated * np.asarray(scale, np.float64)
    t = t if residual is None else t + np.asarray(residual, np.float64)
    oi = 1.0 / np.sqrt((t * t).mean(-1, keepdims=True) + eps)
    out = t if out_norm_w is None else t * oi * np.asarray(out_norm_w, np.float64)
    if parts is not None:
        parts.update(y=y, inv=inv, w=w, gated=gated, a=a, t=t, oi=oi, n=n)
    return out, t


def block_norm_backward(x, *, dout=None, dt=None, norm_w=None, z=None, gate_first=False, residual=None, scale=None,
                        out_norm_w=None, group_size=None, eps=1e-6):
    p = {}
    x = np.asarray(x, np.float64)
    block_norm(x, norm_w=norm_w, z=z, gate_first=gate_first, residual=residual, scale=scale, out_norm_w=out_norm_w,
               group_size=group_size, eps=eps, parts=p)
    rows, d = x.shape
    g = {}
    D = np.zeros(x.shape) if dt is None else np.asarray(dt, np.float64).copy()
    if dout is not None:
        do = np.asarray(dout, np.float64)
        if out_norm_w is None:
            D += do
        else:
            g["out_norm_w"] = (do * p["t"] * p["oi"]).sum(0)
            e = do * np.asarray(out_norm_w, np.float64)
            D += p["oi"] * (e - p["t"] * p["oi"] ** 2 * (e * p["t"]).mean(-1, keepdims=True))
    elif out_norm_w is not None:
        g["out_norm_w"] = np.zeros(d)
    if residual is not None:
        g["residual"] = D
    if scale is not None:
        g["scale"] = (D * p["gated"]).sum(0)
        D = D * np.asarray(scale, np.float64)
    gate, sig = _gate(np.asarray(z, np.float64)) if z is not None else (np.ones(x.shape), None)
    da = D if gate_first else D * gate
    dy = da
    if norm_w is not None:
        nrm = p["y"] * p["inv"]
        dw = (da * nrm).sum(0)
        g["norm_w"] = dw.reshape(-1, np.asarray(norm_w).size).sum(0)
        e = (da * p["w"]).reshape(rows, -1, p["n"])
        m = np.repeat((e * nrm.reshape(e.shape)).mean(-1), p["n"], 1)
        dy = p["inv"] * (e.reshape(rows, d) - nrm * m)
    g["x"] = dy * gate if gate_first else dy
    if z is not None:
        dgate = dy * x if gate_first else D * p["a"]
        g["z"] = dgate * sig * (1.0 + np.asarray(z, np.float64) * (1.0 - sig))
    return g
