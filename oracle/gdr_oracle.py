"""fp64 oracle of the gated delta rule (include/gdr.h): the recurrence token by
token and its reverse scan, in plain numpy. Test infrastructure only; it shares
no code or chunk algebra with the kernels.

    u_t = v_t - e^{g_t} S k_t,  S <- e^{g_t} S + beta_t u_t k_t^T,  o_t = scale S q_t

q, k [B][T][Hk][K]; v, o [B][T][Hv][V]; g, beta [B][T][Hv]; states [B][Hv][V][K].
"""
from __future__ import annotations

import numpy as np

EPS = 1e-6


def _heads(x, group):
    return np.repeat(x, group, axis=2)


def _norms(x, l2norm):
    return np.sqrt((x * x).sum(-1, keepdims=True) + EPS) if l2norm else np.ones_like(x[..., :1])


def forward(q, k, v, g, beta, s_init=None, *, scale=None, l2norm=False, history=False):
    """(o, s_final), and with history the state before each token and u."""
    B, T, Hk, K = q.shape
    Hv, V = v.shape[2:]
    scale = K ** -0.5 if scale is None else scale
    q, k = (_heads(x / _norms(x, l2norm), Hv // Hk) for x in (q, k))
    S = np.zeros((B, Hv, V, K)) if s_init is None else s_init.astype(np.float64).copy()
    o, u = np.zeros((B, T, Hv, V)), np.zeros((B, T, Hv, V))
    before = np.zeros((T, B, Hv, V, K)) if history else None
    for t in range(T):
        if history:
            before[t] = S
        S = np.exp(g[:, t])[..., None, None] * S
        u[:, t] = v[:, t] - np.einsum("bhvk,bhk->bhv", S, k[:, t])
        S = S + (beta[:, t][..., None] * u[:, t])[..., None] * k[:, t][:, :, None, :]
        o[:, t] = scale * np.einsum("bhvk,bhk->bhv", S, q[:, t])
    return (o, S, before, u) if history else (o, S)


def backward(q, k, v, g, beta, do, s_init=None, dS_final=None, *, scale=None, l2norm=False):
    """Gradients of sum <do, o> + <dS_final, s_final>: dict dq, dk, dv, dg, dbeta, dS_init."""
    B, T, Hk, K = q.shape
    Hv, V = v.shape[2:]
    group = Hv // Hk
    scale = K ** -0.5 if scale is None else scale
    _, _, before, u = forward(q, k, v, g, beta, s_init, scale=scale, l2norm=l2norm, history=True)
    nq, nk = _norms(q, l2norm), _norms(k, l2norm)
    qh, kh = _heads(q / nq, group), _heads(k / nk, group)
    D = np.zeros((B, Hv, V, K)) if dS_final is None else dS_final.astype(np.float64).copy()
    dq, dk = np.zeros_like(qh), np.zeros_like(kh)
    dv, dg, db = np.zeros((B, T, Hv, V)), np.zeros((B, T, Hv)), np.zeros((B, T, Hv))
    for t in reversed(range(T)):
        kt, b = kh[:, t], beta[:, t][..., None]
        decayed = np.exp(g[:, t])[..., None, None] * before[t]
        after = decayed + (b * u[:, t])[..., None] * kt[:, :, None, :]
        dq[:, t] = scale * np.einsum("bhvk,bhv->bhk", after, do[:, t])
        D = D + scale * do[:, t][..., None] * qh[:, t][:, :, None, :]
        du = np.einsum("bhvk,bhk->bhv", D, kt)
        db[:, t] = (du * u[:, t]).sum(-1)
        lam = b * du
        dv[:, t] = lam
        dk[:, t] = np.einsum("bhvk,bhv->bhk", D, b * u[:, t]) - np.einsum("bhvk,bhv->bhk", decayed, lam)
        D = D - lam[..., None] * kt[:, :, None, :]
        dg[:, t] = (D * decayed).sum((-1, -2))
        D = np.exp(g[:, t])[..., None, None] * D

    def joined(d, x, n):
        d = d.reshape(B, T, Hk, group, K).sum(3)
        y = x / n
        return (d - y * (y * d).sum(-1, keepdims=True)) / n if l2norm else d

    return {"dq": joined(dq, q, nq), "dk": joined(dk, k, nk), "dv": dv, "dg": dg, "dbeta": db, "dS_init": D}


def packed(fn, starts, args, state=None, **kw):
    """fn over the sequences starts[s] .. starts[s+1] of the one batch row of args,
    each from state[s]; a list of its results."""
    out = []
    for s, (a, b) in enumerate(zip(starts, starts[1:])):
        st = {n: None if x is None else x[s:s + 1] for n, x in (state or {}).items()}
        out.append(fn(*(x[:, a:b] for x in args), **st, **kw))
    return out
