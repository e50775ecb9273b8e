"""Plain 64-bit references of the sequence operators, on numpy arrays (test side).

The gated delta rule token by token, its gradients by the formulas, and the
acceptance of drafted tokens.  Shapes as in include/stq.h: packed tokens q, k
[N,H,d_k], v [N,H,d_v], a [N,H] or [N,H,d_k], beta [N,H]; states [B,H,d_k,d_v].
"""
from __future__ import annotations

import numpy as np


def _gate(a):
    return a[..., None] if a.ndim == 2 else a[..., None, None]


def forward(cu, q, k, v, a, beta, S0, commit=None):
    """Outputs [N,H,d_v] (NaN where no sequence has the token), last states,
    and the states after `commit` tokens of each sequence."""
    q, k, v, a, beta = (np.asarray(x, np.float64) for x in (q, k, v, a, beta))
    last = np.array(S0, np.float64)
    kept = last.copy()
    o = np.full(v.shape, np.nan)
    for b in range(len(cu) - 1):
        S = last[b]
        for t in range(cu[b], cu[b + 1]):
            D = _gate(a[t]) * S
            u = beta[t][:, None] * (v[t] - np.einsum("hij,hi->hj", D, k[t]))
            S = D + k[t][:, :, None] * u[:, None, :]
            o[t] = np.einsum("hij,hi->hj", S, q[t])
            if commit is not None and t - cu[b] + 1 == commit[b]:
                kept[b] = S
        last[b] = S
    return o, last, kept


def backward(cu, q, k, v, a, beta, S0, do, dlast):
    """Gradients of sum(o * do) + sum(last * dlast) with respect to q, k, v, a,
    beta and the initial states, token by token from the end."""
    q, k, v, a, beta, do = (np.asarray(x, np.float64) for x in (q, k, v, a, beta, do))
    g = {n: np.zeros(x.shape) for n, x in (("q", q), ("k", k), ("v", v), ("a", a), ("beta", beta))}
    dS0 = np.array(dlast, np.float64)
    for b in range(len(cu) - 1):
        S, seen = np.array(S0[b], np.float64), []
        for t in range(cu[b], cu[b + 1]):
            D = _gate(a[t]) * S
            e = v[t] - np.einsum("hij,hi->hj", D, k[t])
            u = beta[t][:, None] * e
            S1 = D + k[t][:, :, None] * u[:, None, :]
            seen.append((t, S, D, e, u, S1))
            S = S1
        G = dS0[b]
        for t, S, D, e, u, S1 in reversed(seen):
            g["q"][t] = np.einsum("hij,hj->hi", S1, do[t])
            G = G + q[t][:, :, None] * do[t][:, None, :]
            du = np.einsum("hij,hi->hj", G, k[t])
            de = beta[t][:, None] * du
            g["beta"][t] = (du * e).sum(-1)
            g["v"][t] = de
            g["k"][t] = np.einsum("hij,hj->hi", G, u) - np.einsum("hij,hj->hi", D, de)
            G = G - k[t][:, :, None] * de[:, None, :]
            da = (G * S).sum(-1)
            g["a"][t] = da if a.ndim == 3 else da.sum(-1)
            G = _gate(a[t]) * G
        dS0[b] = G
    return dict(g, state=dS0)


def verify(tokens, lens, p, q, r):
    """(accepted, next): exact products, running sums in 64 bits."""
    B, T = tokens.shape
    p, q, r = (np.asarray(x, np.float64) for x in (p, q, r))
    V = p.shape[2]
    acc, nxt = np.zeros(B, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        n = int(min(max(lens[b], 0), T)) if lens is not None else T
        t = 0
        while t < n:
            x = int(tokens[b, t])
            if not (0 <= x < V and r[b, t] * q[b, t, x] < p[b, t, x]):
                break
            t += 1
        full = np.where(p[b, t] > 0, p[b, t], 0.0)
        w = full
        if t < n:
            rest = np.where(p[b, t] > q[b, t], p[b, t] - q[b, t], 0.0)
            w = rest if rest.sum() > 0 else full
        c = np.cumsum(w)
        past = np.nonzero(c > min(max(r[b, T], 0.0), 1.0) * c[-1])[0]
        acc[b] = t
        nxt[b] = -1 if c[-1] == 0 else past[0] if len(past) else np.nonzero(w > 0)[0][-1]
    return acc, nxt
