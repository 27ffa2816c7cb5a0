"""Cases for the gated delta rule (chunked and recurrent) and the norms around its block.

Four operators, each in its plain form and as the call a user makes:

  delta  the gated delta rule over whole sequences (forward, or forward and backward):
             S_t = e^{g_t} S_{t-1} + beta_t (v_t - e^{g_t} S_{t-1} k_t) k_t^T,   o_t = scale S_t q_t
         with S [value][key] in 32 bits, heads shared between query/key and value heads, sequences
         of one length or packed one after the other, and optionally q and k normalised to length one
  step   the same recurrence for a few tokens of many sequences, states updated in place in a pool
  add    the norm before a block: h = residual + scale * x,  n = h / rms(h) * weight
  gated  the norm after it, a head at a time: y = o / rms(o) * weight * silu(z)
"""
import math

import numpy as np
import torch

own = False

CHUNK = 64  # the plain form's chunk
EPS_NORM = 1e-6
EPS_L2 = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------- the cases ---

def _delta(name, B, T, Hk, Hv, K, V, dtype, train, *, packed=0, carry=False, l2norm=False):
    return {"name": name, "op": "delta", "B": B, "T": T, "Hk": Hk, "Hv": Hv, "K": K, "V": V, "dtype": dtype,
            "train": train, "packed": packed, "carry": carry, "l2norm": l2norm}


def listed():
    return [
        # the framework's smallest workload: one short sequence, where the launches count
        _delta("prefill-tiny-fp32", 1, 64, 2, 2, 16, 16, "f32", False),
        # a serving batch's prompts, packed without padding, each going on from the state it has;
        # grouped heads of 128
        _delta("prefill-packed-bf16", 1, 8191, 16, 32, 128, 128, "bf16", False, packed=24, carry=True, l2norm=True),
        # the framework's long workload: one sequence of 65536 tokens with a carried state
        _delta("prefill-long-fp32", 1, 65536, 40, 40, 64, 64, "f32", False, carry=True),
        # a training step on the framework's throughput workload (the 1.5B-shaped layer)
        _delta("train-1.5b-layer-bf16", 4, 4096, 32, 32, 64, 64, "bf16", True),
        # a training step on its 0.1B-shaped layer in 32 bits
        _delta("train-0.1b-layer-fp32", 8, 4096, 12, 12, 64, 64, "f32", True),
        # a training step with grouped heads of 128, q and k normalised inside, an odd length
        _delta("train-grouped-bf16", 2, 4095, 16, 32, 128, 128, "bf16", True, carry=True, l2norm=True),
        # one user's next token
        {"name": "decode-1-bf16", "op": "step", "R": 1, "T": 1, "Hk": 16, "Hv": 32, "K": 128, "V": 128,
         "dtype": "bf16", "l2norm": True, "slots": 4},
        # a full serving batch's next tokens, states anywhere in the pool
        {"name": "decode-256-bf16", "op": "step", "R": 256, "T": 1, "Hk": 16, "Hv": 32, "K": 128, "V": 128,
         "dtype": "bf16", "l2norm": True, "slots": 300},
        # the norm before a block for one token (the 1.5B-shaped width)
        {"name": "norm-before-1-bf16", "op": "add", "rows": 1, "D": 2048, "dtype": "bf16", "residual": "bf16",
         "scaled": True, "train": False},
        # and over a training batch of the throughput workload, residual stream in 32 bits
        {"name": "norm-before-train-bf16", "op": "add", "rows": 16384, "D": 2048, "dtype": "bf16", "residual": "f32",
         "scaled": True, "train": True},
        # the gated norm after a block for one token
        {"name": "norm-after-1-bf16", "op": "gated", "rows": 1, "H": 32, "D": 128, "dtype": "bf16", "train": False},
        # and over a training batch of the throughput workload
        {"name": "norm-after-train-bf16", "op": "gated", "rows": 16384, "H": 32, "D": 64, "dtype": "bf16",
         "train": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta", "step", "add", "gated"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    train = rng.random() < 0.5
    if op in ("delta", "step"):
        Hk = rng.choice([1, 2, 3, 4, 8, 12, 16])
        Hv = Hk * rng.choice([1, 1, 2, 3])
        K = rng.choice([16, 32, 64, 64, 96, 128, 128])
        V = rng.choice([K, K, 64, 128])
        l2norm = rng.random() < 0.5
    if op == "delta":
        tokens = _log(rng, 1, 16384)
        packed = rng.choice([0, 0, 1, 2, 7, 30])
        B = 1 if packed else rng.choice([1, 1, 2, 5, 8])
        T = max(1, tokens // B)
        case = _delta("", B, T, Hk, Hv, K, V, dtype, train, packed=packed, carry=rng.random() < 0.5, l2norm=l2norm)
        del case["name"]
        return case
    if op == "step":
        R = _log(rng, 1, 256)
        return {"op": "step", "R": R, "T": rng.choice([1, 1, 1, 2, 5]), "Hk": Hk, "Hv": Hv, "K": K, "V": V,
                "dtype": dtype, "l2norm": l2norm, "slots": R + rng.randrange(0, 40)}
    if op == "add":
        D = rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 8, 1024), 768, 2048, 2560])
        return {"op": "add", "rows": _log(rng, 1, 16384 * 2048 // D), "D": D, "dtype": dtype,
                "residual": rng.choice([dtype, "f32"]), "scaled": rng.random() < 0.5, "train": train}
    D = rng.choice([16, 32, 64, 64, 96, 128, 128, 256])
    H = rng.choice([1, 2, 8, 12, 32, 40])
    return {"op": "gated", "rows": _log(rng, 1, 16384 * 2048 // (H * D)), "H": H, "D": D, "dtype": dtype,
            "train": train}


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "delta":
        n, nseq = case["B"] * case["T"], case["packed"] or case["B"]
        qk, vo, gb = n * case["Hk"] * case["K"] * e, n * case["Hv"] * case["V"] * e, n * case["Hv"] * 4
        state = nseq * case["Hv"] * case["K"] * case["V"] * 4
        forward = 2 * qk + 2 * vo + 2 * gb + state * (2 if case["carry"] else 1)
        products = 2.0 * n * case["Hv"] * case["K"] * case["V"]  # one product of the state with a vector a token
        if not case["train"]:  # S k, the update, S q
            return {"bytes": forward, "flops": 3 * products}
        # the gradients of each of the three products are two more
        return {"bytes": forward + 4 * qk + 3 * vo + 4 * gb + state * (2 if case["carry"] else 0),
                "flops": 9 * products}
    if op == "step":
        n = case["R"] * case["T"]
        state = case["R"] * case["Hv"] * case["K"] * case["V"] * 4
        small = n * (2 * case["Hk"] * case["K"] + 2 * case["Hv"] * case["V"]) * e + n * case["Hv"] * 8
        return {"bytes": 2 * state + small + 4 * case["R"], "flops": 6.0 * n * case["Hv"] * case["K"] * case["V"]}
    if op == "add":
        m, r = case["rows"] * case["D"], 2 if case["residual"] == "bf16" else 4
        vec = case["D"] * 4 * (2 if case["scaled"] else 1)
        forward = 2 * m * e + 2 * m * r + vec  # x, residual in; n, h out
        if not case["train"]:
            return {"bytes": forward, "flops": 6.0 * m}
        # x, residual, dn, dh in; the residual's gradient and x's out
        return {"bytes": forward + 3 * m * e + 3 * m * r + 2 * vec, "flops": 20.0 * m}
    m = case["rows"] * case["H"] * case["D"]
    if not case["train"]:
        return {"bytes": 3 * m * e + 4 * case["D"], "flops": 8.0 * m}
    return {"bytes": 8 * m * e + 12 * case["D"], "flops": 28.0 * m}


# --------------------------------------------------------------------------- the inputs ---

def _gates(gen, shape, H):
    """Log decays and write strengths as a trained layer has them: a rate and a step size a head, moved by the token."""
    rate = torch.empty(H, device="cuda").uniform_(1, 16, generator=gen)
    step = torch.empty(H, device="cuda").uniform_(math.log(1e-3), math.log(1e-1), generator=gen).exp()
    x = torch.randn(shape, device="cuda", generator=gen)
    g = -rate * torch.nn.functional.softplus(x + step.expm1().log())
    return g.contiguous(), torch.sigmoid(torch.randn(shape, device="cuda", generator=gen))


def _lengths(case, seed):
    """The packed sequences' lengths: shares of very different size, some of them one token or none."""
    rng = np.random.RandomState(seed % (1 << 31))
    n, total = case["packed"], case["B"] * case["T"]
    share = rng.exponential(1.0, n) * (rng.rand(n) > 0.1)
    share = share / share.sum() if share.sum() else np.full(n, 1.0 / n)
    cuts = np.floor(np.cumsum(share) * total + 1e-9).astype(np.int64)
    cuts[-1] = total
    return [0] + [int(c) for c in np.minimum(cuts, total)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    s = {"case": dict(case)}
    op = case["op"]
    if op in ("delta", "step"):
        B, T, Hk, Hv, K, V = case["R" if op == "step" else "B"], case["T"], case["Hk"], case["Hv"], case["K"], case["V"]
        common = 0.3 * normal(B, 1, Hk, K)  # keys of one sequence are related
        q, k = normal(B, T, Hk, K), normal(B, T, Hk, K) + common
        if not case["l2norm"]:
            q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
        s["q"], s["k"], s["v"] = q.to(dt), k.to(dt), normal(B, T, Hv, V).to(dt)
        s["g"], s["beta"] = _gates(gen, (B, T, Hv), Hv)
        s["scale"] = K ** -0.5
        if op == "step":
            s["state"] = 0.1 * normal(case["slots"], Hv, V, K)
            s["slots"] = torch.randperm(case["slots"], device="cuda", generator=gen)[:B].to(torch.int32)
            return s
        nseq = case["packed"] or B
        s["starts"] = None
        if case["packed"]:
            cuts = _lengths(case, seed)
            s["starts"] = torch.tensor(cuts, dtype=torch.int32, device="cuda")
            s["longest"] = max(b - a for a, b in zip(cuts, cuts[1:]))
        s["s_init"] = 0.1 * normal(nseq, Hv, V, K) if case["carry"] else None
        if case["train"]:
            s["do"] = normal(B, T, Hv, V).to(dt)
            s["dS_final"] = 0.1 * normal(nseq, Hv, V, K) if case["carry"] else None
        return s
    if op == "add":
        rows, D, rt = case["rows"], case["D"], DTYPES[case["residual"]]
        s["x"], s["residual"] = normal(rows, D).to(dt), (3 * normal(rows, D)).to(rt)
        s["weight"] = 1 + 0.1 * normal(D)
        s["scale"] = 0.5 + 0.1 * normal(D) if case["scaled"] else None
        if case["train"]:
            s["dn"], s["dh"] = normal(rows, D).to(dt), normal(rows, D).to(rt)
        return s
    rows, H, D = case["rows"], case["H"], case["D"]
    s["o"], s["z"] = (0.2 * normal(rows, H, D)).to(dt), normal(rows, H, D).to(dt)
    s["weight"] = 1 + 0.1 * normal(D)
    if case["train"]:
        s["dy"] = normal(rows, H, D).to(dt)
    return s


# ----------------------------------------------------------------------- the plain forms ---

def _unit_lower_inverse(L):
    """(I + L)^-1 of a strictly lower L [..., C, C], C a power of two: blocks joined two by two."""
    C = L.shape[-1]
    X = torch.eye(C, device=L.device, dtype=L.dtype).expand(L.shape).clone()
    m = 1
    while m < C:
        cut = X.unflatten(-2, (C // (2 * m), 2, m)).unflatten(-1, (C // (2 * m), 2, m))
        low = L.unflatten(-2, (C // (2 * m), 2, m)).unflatten(-1, (C // (2 * m), 2, m))
        top = cut[..., 0, :, :, 0, :].diagonal(dim1=-4, dim2=-2).movedim(-1, -3)
        bottom = cut[..., 1, :, :, 1, :].diagonal(dim1=-4, dim2=-2).movedim(-1, -3)
        left = low[..., 1, :, :, 0, :].diagonal(dim1=-4, dim2=-2).movedim(-1, -3)
        cut[..., 1, :, :, 0, :].diagonal(dim1=-4, dim2=-2).movedim(-1, -3).copy_(-(bottom @ left @ top))
        m *= 2
    return X


def _chunks(x):
    """[B][T][H][D] as [B][H][n][C][D], the last chunk filled up with zeros."""
    B, T, H, D = x.shape
    n = max(1, -(-T // CHUNK))
    x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * CHUNK - T))
    return x.view(B, n, CHUNK, H, D).permute(0, 3, 1, 2, 4).contiguous()


def _whole(x, T):
    B, H, n, C, D = x.shape
    return x.permute(0, 2, 3, 1, 4).reshape(B, n * C, H, D)[:, :T].contiguous()


def _pad_index(starts, longest):
    """For packed sequences: which token each place of [sequence][longest] is, and whether there is one."""
    at = starts[:-1, None].long() + torch.arange(longest, device=starts.device)
    return at, at < starts[1:, None]


def _delta_plain(s):
    case = s["case"]
    q, k, v, g, beta = (s[n].float() for n in ("q", "k", "v", "g", "beta"))
    do = s["do"].float() if case["train"] else None
    if s["starts"] is not None:
        at, there = _pad_index(s["starts"], s["longest"])
        at = torch.where(there, at, 0)
        q, k, v, g, beta, do = (None if x is None else torch.where(there.view(*there.shape, *[1] * (x.dim() - 2)), x[0][at], 0.0)
                                for x in (q, k, v, g, beta, do))
    B, T, Hk, K = q.shape
    Hv, V = v.shape[2:]
    group = Hv // Hk
    if case["l2norm"]:
        rq, rk = (torch.rsqrt(x.square().sum(-1, keepdim=True) + EPS_L2) for x in (q, k))
        q, k = q * rq, k * rk
    qc, kc = (_chunks(x.repeat_interleave(group, dim=2)) for x in (q, k))
    vc, gc, bc = _chunks(v), _chunks(g[..., None])[..., 0], _chunks(beta[..., None])[..., 0]
    scale, n = s["scale"], qc.shape[2]
    G = gc.cumsum(-1)
    i = torch.arange(CHUNK, device=q.device)
    lower = i[:, None] >= i
    ratio = torch.exp(torch.where(lower, G[..., :, None] - G[..., None, :], -math.inf))
    strict = torch.where(i[:, None] > i, ratio, 0.0)
    inverse = _unit_lower_inverse(kc @ kc.mT * strict * bc[..., None, :])
    P = scale * (qc @ kc.mT) * ratio * bc[..., None, :]
    head, tail = G.exp()[..., None], (G[..., -1:] - G).exp()[..., None]
    whole = G[..., -1].exp()[..., None, None]
    write = tail * bc[..., None] * kc
    S = torch.zeros(B, Hv, V, K, device=q.device) if s["s_init"] is None else s["s_init"].float()
    states, us = [], []
    for c in range(n):
        states.append(S)
        u = inverse[:, :, c] @ (vc[:, :, c] - head[:, :, c] * (kc[:, :, c] @ S.mT))
        us.append(u)
        S = whole[:, :, c] * S + u.mT @ write[:, :, c]
    states, u = torch.stack(states, 2), torch.stack(us, 2)
    o = scale * head * (qc @ states.mT) + P @ u
    out = {"o": _whole(o, T), "s_final": S}
    if case["train"]:
        doc = _chunks(do)
        dS = torch.zeros_like(S) if s["dS_final"] is None else s["dS_final"].float()
        dstates, lams = [], []
        for c in reversed(range(n)):
            dstates.append(dS)
            lam = inverse[:, :, c].mT @ (P[:, :, c].mT @ doc[:, :, c] + write[:, :, c] @ dS.mT)
            lams.append(lam)
            dS = whole[:, :, c] * dS + scale * doc[:, :, c].mT @ (head[:, :, c] * qc[:, :, c]) - lam.mT @ (head[:, :, c] * kc[:, :, c])
        dstates, lam = torch.stack(dstates[::-1], 2), torch.stack(lams[::-1], 2)
        F, E = scale * (doc @ u.mT) * strict, (lam @ u.mT) * strict
        # a token's effect on itself does not decay: kept out of the sums whose differences are dg
        self_ = scale * (doc * u).sum(-1, keepdim=True)
        Fb, Eb = F * bc[..., None, :], E * bc[..., None, :]
        dq = scale * head * (doc @ states) + Fb @ kc
        read = -head * (lam @ states) - Eb @ kc
        w = F.mT @ qc - E.mT @ kc + tail * (u @ dstates)
        dG = (qc * dq).sum(-1) + (kc * read).sum(-1) - bc * (kc * w).sum(-1)
        dq, w = dq + self_ * bc[..., None] * kc, w + self_ * qc
        dbeta = (kc * w).sum(-1)
        after = whole * states + u.mT @ write
        dG[..., -1] += (after * dstates).sum((-1, -2))
        dg = dG.flip(-1).cumsum(-1).flip(-1)
        dq, dk = (_whole(x, T).view(B, T, Hk, group, K).sum(3) for x in (dq, read + bc[..., None] * w))
        if case["l2norm"]:
            dq, dk = (r * (d - x * (x * d).sum(-1, keepdim=True)) for r, x, d in ((rq, q, dq), (rk, k, dk)))
        out |= {"dq": dq, "dk": dk, "dv": _whole(lam, T), "dg": _whole(dg[..., None], T)[..., 0],
                "dbeta": _whole(dbeta[..., None], T)[..., 0]}
        if s["s_init"] is not None:
            out["dS_init"] = dS
    if s["starts"] is not None:
        for name in [m for m in out if m not in ("s_final", "dS_init")]:
            out[name] = out[name][there][None]
    for name, like in (("o", "v"), ("dq", "q"), ("dk", "k"), ("dv", "v")):
        if name in out:
            out[name] = out[name].to(s[like].dtype)
    return out


def _step_plain(s):
    q, k, v, g, beta = (s[n].float() for n in ("q", "k", "v", "g", "beta"))
    group = v.shape[2] // q.shape[2]
    if s["case"]["l2norm"]:
        q, k = (x * torch.rsqrt(x.square().sum(-1, keepdim=True) + EPS_L2) for x in (q, k))
    q, k = (x.repeat_interleave(group, dim=2) for x in (q, k))
    at = s["slots"].long()
    S, outs = s["state"][at], []
    for t in range(q.shape[1]):
        S = S * g[:, t].exp()[..., None, None]
        u = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, None]).sum(-1))
        S = S + u[..., None] * k[:, t, :, None]
        outs.append(s["scale"] * (S * q[:, t, :, None]).sum(-1))
    s["state"][at] = S
    return {"o": torch.stack(outs, 1).to(s["v"].dtype), "state": s["state"]}


def _add_plain(s):
    x, w, a = s["x"].float(), s["weight"], s["scale"]
    h = s["residual"].float() + (x if a is None else a * x)
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS_NORM)
    out = {"h": h.to(s["residual"].dtype), "n": (h * r * w).to(s["x"].dtype)}
    if s["case"]["train"]:
        dn, u = s["dn"].float(), h * r
        dh = s["dh"].float() + r * (dn * w - u * (dn * w * u).mean(-1, keepdim=True))
        out |= {"dresidual": dh.to(s["residual"].dtype), "dx": (dh if a is None else a * dh).to(s["x"].dtype),
                "dweight": (dn * u).sum(0)}
        if a is not None:
            out["dscale"] = (dh * x).sum(0)
    return out


def _gated_plain(s):
    o, z, w = s["o"].float(), s["z"].float(), s["weight"]
    r = torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS_NORM)
    sig = 1 / (1 + torch.exp(-z))
    u, gate = o * r, z * sig
    out = {"y": (u * w * gate).to(s["o"].dtype)}
    if s["case"]["train"]:
        dy = s["dy"].float()
        du = dy * w * gate
        out |= {"do": (r * (du - u * (du * u).mean(-1, keepdim=True))).to(s["o"].dtype),
                "dz": (dy * u * w * (sig * (1 + z * (1 - sig)))).to(s["z"].dtype),
                "dweight": (dy * u * gate).sum((0, 1))}
    return out


# ---------------------------------------------------------------------- the framework's ---

def _delta_own(s):
    from linear_rnn_state_gb300 import gdr

    case = s["case"]
    opts = {"scale": s["scale"], "qk_l2norm": case["l2norm"], "seq_starts": s["starts"]}
    ins = [s[n] for n in ("q", "k", "v", "g", "beta")]
    o, s_final, saved = gdr.forward(*ins, s["s_init"], want_saved=case["train"], **opts)
    out = {"o": o, "s_final": s_final}
    if case["train"]:
        grads = gdr.backward(*ins, s["do"], saved, dS_final=s["dS_final"], want_dS_init=case["carry"], **opts)
        out |= {n: x for n, x in grads.items() if x is not None}
    return out


def _step_own(s):
    from linear_rnn_state_gb300 import gdr

    o = gdr.step(*(s[n] for n in ("q", "k", "v", "g", "beta", "state")), slots=s["slots"], scale=s["scale"],
                 qk_l2norm=s["case"]["l2norm"])
    return {"o": o, "state": s["state"]}


def _add_own(s):
    from linear_rnn_state_gb300 import blocknorm

    h, n, rstd = blocknorm.add_forward(s["x"], s["residual"], s["weight"], s["scale"], eps=EPS_NORM)
    out = {"h": h, "n": n}
    if s["case"]["train"]:
        g = blocknorm.add_backward(s["x"], s["residual"], s["weight"], rstd, s["dn"], s["dh"], s["scale"])
        out |= {k: x for k, x in g.items() if x is not None}
    return out


def _gated_own(s):
    from linear_rnn_state_gb300 import blocknorm

    y, rstd = blocknorm.gated_forward(s["o"], s["z"], s["weight"], eps=EPS_NORM)
    out = {"y": y}
    if s["case"]["train"]:
        out |= blocknorm.gated_backward(s["o"], s["z"], s["weight"], rstd, s["dy"])
    return out


PLAIN = {"delta": _delta_plain, "step": _step_plain, "add": _add_plain, "gated": _gated_plain}
OWN = {"delta": _delta_own, "step": _step_own, "add": _add_own, "gated": _gated_own}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------------------ 64 bits ---

def _delta_exact(s):
    """Token by token, and the gradients by the reverse scan of the recurrence itself."""
    case = s["case"]
    q, k, v, g, beta = (s[n].double() for n in ("q", "k", "v", "g", "beta"))
    B, T, Hk, K = q.shape
    Hv, V = v.shape[2:]
    if s["starts"] is not None:
        T = s["longest"]
        at, there = _pad_index(s["starts"], T)
        at = at.clamp(max=q.shape[1] - 1)

        def spread(x):
            x = x[0][at]
            x[~there] = 0
            return x
    else:
        def spread(x):
            return x
    q, k, v, g, beta = map(spread, (q, k, v, g, beta))
    B = q.shape[0]
    if case["train"] and T * B * Hv * V * K * 8 > 80e9:
        return None
    nq, nk = ((x.square().sum(-1, keepdim=True) + EPS_L2).sqrt() if case["l2norm"] else torch.ones_like(x[..., :1])
              for x in (q, k))
    q, k = (q / nq).repeat_interleave(Hv // Hk, 2), (k / nk).repeat_interleave(Hv // Hk, 2)
    S = torch.zeros(B, Hv, V, K, device=q.device, dtype=torch.float64) if s["s_init"] is None else s["s_init"].double()
    a, scale = g.exp(), s["scale"]
    o = torch.empty_like(v)
    u = torch.empty_like(v)
    before = torch.empty((T, B, Hv, V, K), device=q.device, dtype=torch.float64) if case["train"] else None
    for t in range(T):
        if before is not None:
            before[t] = S
        S = a[:, t, :, None, None] * S
        u[:, t] = v[:, t] - torch.einsum("bhvk,bhk->bhv", S, k[:, t])
        S = S + (beta[:, t, :, None] * u[:, t])[..., None] * k[:, t, :, None, :]
        o[:, t] = scale * torch.einsum("bhvk,bhk->bhv", S, q[:, t])
    out = {"o": o, "s_final": S}
    if case["train"]:
        do = spread(s["do"].double())
        D = torch.zeros_like(S) if s["dS_final"] is None else s["dS_final"].double()
        dq, dk, dv, dg, db = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(g), torch.empty_like(g)
        for t in reversed(range(T)):
            kt, bt = k[:, t], beta[:, t, :, None]
            decayed = a[:, t, :, None, None] * before[t]
            after = decayed + (bt * u[:, t])[..., None] * kt[..., None, :]
            dq[:, t] = scale * torch.einsum("bhvk,bhv->bhk", after, do[:, t])
            D = D + scale * do[:, t, :, :, None] * q[:, t, :, None, :]
            du = torch.einsum("bhvk,bhk->bhv", D, kt)  # of beta u
            db[:, t] = (du * u[:, t]).sum(-1)
            lam = bt * du
            dv[:, t] = lam
            dk[:, t] = torch.einsum("bhvk,bhv->bhk", D, bt * u[:, t]) - torch.einsum("bhvk,bhv->bhk", decayed, lam)
            D = D - lam[..., None] * kt[..., None, :]
            dg[:, t] = (D * decayed).sum((-1, -2))
            D = a[:, t, :, None, None] * D
        group = Hv // Hk

        def joined(d, x, norm):
            d = d.unflatten(2, (Hk, group)).sum(3)
            x = x.unflatten(2, (Hk, group))[:, :, :, 0]
            return (d - x * (x * d).sum(-1, keepdim=True)) / norm if case["l2norm"] else d

        out |= {"dq": joined(dq, q, nq), "dk": joined(dk, k, nk), "dv": dv, "dg": dg, "dbeta": db}
        if s["s_init"] is not None:
            out["dS_init"] = D
    if s["starts"] is not None:
        for name in [m for m in out if m not in ("s_final", "dS_init")]:
            out[name] = out[name][there][None]
    return out


def _step_exact(s):
    fake = {"case": {**s["case"], "train": False}, "starts": None, "scale": s["scale"],
            "s_init": s["state"][s["slots"].long()], **{n: s[n] for n in ("q", "k", "v", "g", "beta")}}
    got = _delta_exact(fake)
    pool = s["state"].double()
    pool[s["slots"].long()] = got["s_final"]
    return {"o": got["o"], "state": pool}


def _add_exact(s):
    x, w = s["x"].double(), s["weight"].double()
    a = torch.ones_like(w) if s["scale"] is None else s["scale"].double()
    h = s["residual"].double() + a * x
    rms = (h.square().mean(-1, keepdim=True) + EPS_NORM).sqrt()
    out = {"h": h, "n": h / rms * w}
    if s["case"]["train"]:
        dn = s["dn"].double()
        t = dn * w
        dh = s["dh"].double() + t / rms - h * (t * h).mean(-1, keepdim=True) / rms ** 3
        out |= {"dresidual": dh, "dx": a * dh, "dweight": (dn * h / rms).sum(0)}
        if s["scale"] is not None:
            out["dscale"] = (dh * x).sum(0)
    return out


def _gated_exact(s):
    o, z, w = s["o"].double(), s["z"].double(), s["weight"].double()
    rms = (o.square().mean(-1, keepdim=True) + EPS_NORM).sqrt()
    gate = z * torch.sigmoid(z)
    out = {"y": o / rms * w * gate}
    if s["case"]["train"]:
        dy, sig = s["dy"].double(), torch.sigmoid(z)
        t = dy * gate * w
        out |= {"do": t / rms - o * (t * o).mean(-1, keepdim=True) / rms ** 3,
                "dz": dy * (o / rms) * w * (sig + z * sig * (1 - sig)),
                "dweight": (dy * gate * o / rms).sum((0, 1))}
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"delta": _delta_exact, "step": _step_exact, "add": _add_exact, "gated": _gated_exact}[case["op"]](s)
