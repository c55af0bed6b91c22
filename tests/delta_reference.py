"""The gated delta rule and its gradients token by token in 64 bits, from the recurrence alone.

    D = exp(g) S;  u = beta (v - k^T D);  S = D + k u^T;  o = scale q^T S

for one sequence: q, k [T, Hk, K], v [T, Hv, V], g, beta [T, Hv], state [Hv, K, V].  Used by the tests only; shares no
code with the kernels.
"""
from __future__ import annotations

import torch


def _wide(x, hv):
    return x.double().repeat_interleave(hv // x.shape[1], 1)


def sequence(q, k, v, g, beta, scale, h0=None, do=None, dht=None):
    """{"o", "state"} and, with ``do``, {"dq", "dk", "dv", "dg", "dbeta", "dh0"}."""
    hk, hv, T = q.shape[1], v.shape[1], q.shape[0]
    Q, K, Vv, G, B = _wide(q, hv), _wide(k, hv), v.double(), g.double(), beta.double()
    S = torch.zeros(hv, q.shape[2], v.shape[2], dtype=torch.float64, device=q.device) if h0 is None else h0.double()
    o, kept = torch.zeros(T, hv, v.shape[2], dtype=torch.float64, device=q.device), []
    for t in range(T):
        # a forgotten state is gone, whatever it held
        D = torch.where((G[t] == -torch.inf)[:, None, None], 0.0, S * G[t].exp()[:, None, None])
        miss = Vv[t] - (K[t][:, :, None] * D).sum(1)
        N = D + K[t][:, :, None] * (B[t][:, None] * miss)[:, None, :]
        o[t] = scale * (Q[t][:, :, None] * N).sum(1)
        kept.append((D, miss, N))
        S = N
    out = {"o": o, "state": S}
    if do is None:
        return out
    dS = torch.zeros_like(S) if dht is None else dht.double()
    dq, dk = torch.zeros_like(Q), torch.zeros_like(K)
    dv, dg, db = torch.zeros_like(Vv), torch.zeros_like(G), torch.zeros_like(B)
    for t in range(T - 1, -1, -1):
        D, miss, N = kept[t]
        d_o = do[t].double()
        dS = dS + scale * Q[t][:, :, None] * d_o[:, None, :]
        dq[t] = scale * (N * d_o[:, None, :]).sum(2)
        du = (K[t][:, :, None] * dS).sum(1)
        db[t] = (du * miss).sum(1)
        dv[t] = B[t][:, None] * du
        dk[t] = (dS * (B[t][:, None] * miss)[:, None, :]).sum(2) - (D * dv[t][:, None, :]).sum(2)
        dS = dS - K[t][:, :, None] * dv[t][:, None, :]
        dg[t] = (dS * D).sum((1, 2))
        dS = dS * G[t].exp()[:, None, None]
    shared = lambda x: x.unflatten(1, (hk, hv // hk)).sum(2)  # noqa: E731
    out.update(dq=shared(dq), dk=shared(dk), dv=dv, dg=dg, dbeta=db, dh0=dS)
    return out


def packed(q, k, v, g, beta, scale, lens, h0=None, do=None, dht=None):
    """The same over packed sequences: tokens together, states stacked."""
    at, parts = 0, []
    for i, n in enumerate(lens):
        cut = lambda x: None if x is None else x[at:at + n]  # noqa: E731, B023
        pick = lambda x: None if x is None else x[i]  # noqa: E731, B023
        parts.append(sequence(cut(q), cut(k), cut(v), cut(g), cut(beta), scale, pick(h0), cut(do), pick(dht)))
        at += n
    return {name: (torch.stack if name in ("state", "dh0") else torch.cat)([p[name] for p in parts]) for name in parts[0]}
