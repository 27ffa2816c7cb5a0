"""fp64 oracle of linear attention with a decay (include/linattn.h): the recurrence
token by token and its reverse scan, in plain numpy. Test infrastructure only; it
shares no code or chunk algebra with the kernels.

    S <- e^{g_t} S + v_t k_t^T,  o_t = scale S q_t

q, k [B][T][Hk][K]; v, o [B][T][Hv][V]; g [B][T][Hv] or [Hv]; states [B][Hv][V][K].
"""
from __future__ import annotations

import numpy as np


def _heads(x, group):
    return np.repeat(x, group, axis=2)


def _decay(g, v):
    """e^g of every token; log decays below -1e6 (and -inf) empty the state."""
    return np.exp(np.broadcast_to(g, v.shape[:3]))


def forward(q, k, v, g, s_init=None, *, scale=None, history=False):
    """(o, s_final), and with history the state before each token."""
    B, T, Hk, K = q.shape
    Hv, V = v.shape[2:]
    scale = K ** -0.5 if scale is None else scale
    q, k, a = _heads(q, Hv // Hk), _heads(k, Hv // Hk), _decay(g, v)
    S = np.zeros((B, Hv, V, K)) if s_init is None else s_init.astype(np.float64).copy()
    o = np.zeros((B, T, Hv, V))
    before = np.zeros((T, B, Hv, V, K)) if history else None
    for t in range(T):
        if history:
            before[t] = S
        S = a[:, t, :, None, None] * S + v[:, t, :, :, None] * k[:, t, :, None, :]
        o[:, t] = scale * np.einsum("bhvk,bhk->bhv", S, q[:, t])
    return (o, S, before) if history else (o, S)


def backward(q, k, v, g, do, s_init=None, dS_final=None, *, scale=None):
    """Gradients of sum <do, o> + <dS_final, s_final>: dict dq, dk, dv, dg, dS_init."""
    B, T, Hk, K = q.shape
    Hv, V = v.shape[2:]
    group = Hv // Hk
    scale = K ** -0.5 if scale is None else scale
    _, _, before = forward(q, k, v, g, s_init, scale=scale, history=True)
    qh, kh, a = _heads(q, group), _heads(k, group), _decay(g, v)
    D = np.zeros((B, Hv, V, K)) if dS_final is None else dS_final.astype(np.float64).copy()
    dq, dk = np.zeros_like(qh), np.zeros_like(kh)
    dv, dg = np.zeros((B, T, Hv, V)), np.zeros((B, T, Hv))
    for t in reversed(range(T)):
        decayed = a[:, t, :, None, None] * before[t]
        after = decayed + v[:, t, :, :, None] * kh[:, t, :, None, :]
        dq[:, t] = scale * np.einsum("bhvk,bhv->bhk", after, do[:, t])
        D = D + scale * do[:, t, :, :, None] * qh[:, t, :, None, :]
        dv[:, t] = np.einsum("bhvk,bhk->bhv", D, kh[:, t])
        dk[:, t] = np.einsum("bhvk,bhv->bhk", D, v[:, t])
        dg[:, t] = (D * decayed).sum((-1, -2))
        D = a[:, t, :, None, None] * D
    dq, dk = (x.reshape(B, T, Hk, group, K).sum(3) for x in (dq, dk))
    return {"dq": dq, "dk": dk, "dv": dv, "dg": dg.sum((0, 1)) if g.ndim == 1 else dg, "dS_init": D}


def packed(fn, starts, args, state=None, **kw):
    """fn over the sequences starts[s] .. starts[s+1] of the one batch row of args (one
    with a single axis is every sequence's), each from state[s]; a list of its results."""
    out = []
    for s, (a, b) in enumerate(zip(starts, starts[1:])):
        st = {n: None if x is None else x[s:s + 1] for n, x in (state or {}).items()}
        out.append(fn(*(x if x.ndim == 1 else x[:, a:b] for x in args), **st, **kw))
    return out
