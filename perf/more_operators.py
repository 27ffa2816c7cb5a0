"""Cases for linear attention with a decay (chunked and recurrent) and for the norms of queries and keys
with the position rotation.

Three operators, each in its plain form and as the call a user makes:

  lin   linear attention over whole sequences (forward, or forward and backward):
            S_t = e^{g_t} S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t
        with S [value][key] in 32 bits, g one number a token and value head or one fixed number a head, heads
        shared between query/key and value heads, sequences of one length or packed one after the other
  step  the same recurrence for a few tokens of many sequences, states updated in place in a pool
  qk    before it, a head at a time for queries and keys in one pass: y = rot(x / rms(x) * weight, position),
        rot turning the pairs of the first dimensions by position * freq (forward, or forward and backward)
"""
import math

import numpy as np
import torch

own = False

CHUNK = 64  # the plain form's chunk
EPS_NORM = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------- the cases ---

def _lin(name, B, T, Hk, Hv, K, V, dtype, train, *, packed=0, carry=False, fixed=False):
    return {"name": name, "op": "lin", "B": B, "T": T, "Hk": Hk, "Hv": Hv, "K": K, "V": V, "dtype": dtype,
            "train": train, "packed": packed, "carry": carry, "fixed": fixed}


def _qk(name, tokens, Hq, Hk, D, R, dtype, train, *, interleaved=False, far=0):
    return {"name": name, "op": "qk", "tokens": tokens, "Hq": Hq, "Hk": Hk, "D": D, "R": R, "dtype": dtype, "train": train,
            "interleaved": interleaved, "far": far}


def listed():
    return [
        # the framework's smallest workload: one short sequence, where the launches count
        _lin("lin-tiny-fp32", 1, 64, 2, 2, 16, 16, "f32", False),
        # a serving batch's prompts, packed without padding, each going on from the state it has; grouped heads of 128
        _lin("lin-prefill-packed-bf16", 1, 8191, 16, 32, 128, 128, "bf16", False, packed=24, carry=True),
        # the framework's long workload: one sequence of 65536 tokens with a carried state, a fixed decay for each head
        _lin("lin-prefill-long-fp32", 1, 65536, 40, 40, 64, 64, "f32", False, carry=True, fixed=True),
        # a training step on the framework's throughput workload (the 1.5B-shaped layer)
        _lin("lin-train-1.5b-layer-bf16", 4, 4096, 32, 32, 64, 64, "bf16", True),
        # a training step on its 0.1B-shaped layer in 32 bits
        _lin("lin-train-0.1b-layer-fp32", 8, 4096, 12, 12, 64, 64, "f32", True),
        # a training step with grouped heads of 128 and a learned fixed decay for each head, an odd length
        _lin("lin-train-grouped-bf16", 2, 4095, 16, 32, 128, 128, "bf16", True, carry=True, fixed=True),
        # one user's next token
        {"name": "step-1-bf16", "op": "step", "R": 1, "T": 1, "Hk": 16, "Hv": 32, "K": 128, "V": 128, "dtype": "bf16",
         "fixed": False, "slots": 4},
        # a full serving batch's next tokens, states anywhere in the pool
        {"name": "step-256-bf16", "op": "step", "R": 256, "T": 1, "Hk": 16, "Hv": 32, "K": 128, "V": 128, "dtype": "bf16",
         "fixed": True, "slots": 300},
        # queries and keys of one token deep in a long text
        _qk("qk-1-bf16", 1, 16, 16, 128, 128, "bf16", False, far=1 << 20),
        # of a serving batch's packed prompts, half of each head rotated
        _qk("qk-prefill-packed-bf16", 8191, 32, 8, 128, 64, "bf16", False, far=1 << 17),
        # of a training batch of the throughput workload
        _qk("qk-train-1.5b-layer-bf16", 16384, 32, 32, 64, 64, "bf16", True),
        # of a training batch of the 0.1B-shaped layer in 32 bits, neighbouring dimensions as pairs
        _qk("qk-train-0.1b-layer-fp32", 32768, 12, 12, 64, 64, "f32", True, interleaved=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lin", "lin", "lin", "step", "qk", "qk"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    train = rng.random() < 0.5
    fixed = rng.random() < 0.4
    if op in ("lin", "step"):
        Hk = rng.choice([1, 2, 3, 4, 8, 12, 16])
        Hv = Hk * rng.choice([1, 1, 2, 3])
        K = rng.choice([16, 32, 64, 64, 96, 128, 128])
        V = rng.choice([K, K, 64, 128])
    if op == "lin":
        tokens = _log(rng, 1, 16384)
        packed = rng.choice([0, 0, 1, 2, 7, 30])
        B = 1 if packed else rng.choice([1, 1, 2, 5, 8])
        case = _lin("", B, max(1, tokens // B), Hk, Hv, K, V, dtype, train, packed=packed, carry=rng.random() < 0.5, fixed=fixed)
        del case["name"]
        return case
    if op == "step":
        R = _log(rng, 1, 256)
        return {"op": "step", "R": R, "T": rng.choice([1, 1, 1, 2, 5]), "Hk": Hk, "Hv": Hv, "K": K, "V": V, "dtype": dtype,
                "fixed": fixed, "slots": R + rng.randrange(0, 40)}
    D = rng.choice([16, 32, 64, 64, 96, 128, 128, 192, 256])
    Hk = rng.choice([1, 2, 4, 8, 12])
    Hq = Hk * rng.choice([1, 1, 2, 4])
    R = rng.choice([D, D, D // 2, 2 * rng.randrange(1, D // 2 + 1)])
    case = _qk("", _log(rng, 1, 16384 * 4096 // ((Hq + Hk) * D)), Hq, Hk, D, R, dtype, train,
               interleaved=rng.random() < 0.3, far=rng.choice([0, 0, 1 << 17, 1 << 20]))
    del case["name"]
    return case


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "qk":
        m, vec = case["tokens"] * (case["Hq"] + case["Hk"]) * case["D"], 8 * case["D"] + 4 * case["R"] + 4 * case["tokens"]
        if not case["train"]:
            return {"bytes": 2 * m * e + vec, "flops": 9.0 * m}
        return {"bytes": 4 * m * e + vec + 8 * case["D"], "flops": 30.0 * m}
    n = (case["R"] if op == "step" else case["B"]) * case["T"]
    qk, vo = n * case["Hk"] * case["K"] * e, n * case["Hv"] * case["V"] * e
    g = case["Hv"] * 4 * (1 if case["fixed"] else n)
    products = 2.0 * n * case["Hv"] * case["K"] * case["V"]  # one product of the state with a vector a token
    if op == "step":
        state = case["R"] * case["Hv"] * case["K"] * case["V"] * 4
        return {"bytes": 2 * state + 2 * qk + 2 * vo + g + 4 * case["R"], "flops": 2 * products}
    state = (case["packed"] or case["B"]) * case["Hv"] * case["K"] * case["V"] * 4
    forward = 2 * qk + 2 * vo + g + state * (2 if case["carry"] else 1)
    if not case["train"]:  # the update and S q
        return {"bytes": forward, "flops": 2 * products}
    # the gradients of each of the two products are two more
    return {"bytes": forward + 2 * qk + 2 * vo + g + state * (2 if case["carry"] else 0), "flops": 6 * products}


# --------------------------------------------------------------------------- the inputs ---

def _decays(gen, shape, H):
    """Log decays as a trained layer has them: a rate and a step size a head, moved by the token."""
    rate = torch.empty(H, device="cuda").uniform_(1, 16, generator=gen)
    step = torch.empty(H, device="cuda").uniform_(math.log(1e-3), math.log(1e-1), generator=gen).exp()
    x = torch.randn(shape, device="cuda", generator=gen)
    return (-rate * torch.nn.functional.softplus(x + step.expm1().log())).contiguous()


def _fixed_decays(gen, H):
    """One log decay a head, from memories of a few tokens to some hundreds, slightly moved by training."""
    at = torch.arange(1, H + 1, device="cuda") / H
    return -torch.exp2(-8 * at) * (1 + 0.1 * torch.rand(H, device="cuda", generator=gen))


def _lengths(n, total, seed):
    """The packed sequences' lengths: shares of very different size, some of them one token or none."""
    rng = np.random.RandomState(seed % (1 << 31))
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
    if case["op"] == "qk":
        n, Hq, Hk, D, R = (case[m] for m in ("tokens", "Hq", "Hk", "D", "R"))
        both = normal(n, Hq + Hk, D) * (0.5 + torch.rand(Hq + Hk, 1, device="cuda", generator=gen))
        both = both.to(dt)
        s["q"], s["k"] = both[:, :Hq], both[:, Hq:]  # slices of one projection
        s["wq"], s["wk"] = 1 + 0.1 * normal(D), 1 + 0.1 * normal(D)
        s["freq"] = 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / max(R, 1))
        if case["far"]:
            s["positions"] = torch.randint(0, case["far"], (n,), device="cuda", generator=gen, dtype=torch.int32)
        else:  # packed sequences, each from 0 on
            cuts = torch.tensor(_lengths(4, n, seed), device="cuda")
            at = torch.arange(n, device="cuda")
            s["positions"] = (at - cuts[torch.searchsorted(cuts, at, right=True) - 1]).to(torch.int32)
        if case["train"]:
            s["dq"], s["dk"] = normal(n, Hq, D).to(dt), normal(n, Hk, D).to(dt)
        return s
    B, T, Hk, Hv, K, V = (case[m] for m in ("R" if case["op"] == "step" else "B", "T", "Hk", "Hv", "K", "V"))
    common = 0.3 * normal(B, 1, Hk, K)  # keys of one sequence are related
    s["q"], s["k"], s["v"] = normal(B, T, Hk, K).to(dt), (normal(B, T, Hk, K) + common).to(dt), normal(B, T, Hv, V).to(dt)
    s["g"] = _fixed_decays(gen, Hv) if case["fixed"] else _decays(gen, (B, T, Hv), Hv)
    s["scale"] = K ** -0.5
    if case["op"] == "step":
        s["state"] = normal(case["slots"], Hv, V, K)
        s["slots"] = torch.randperm(case["slots"], device="cuda", generator=gen)[:B].to(torch.int32)
        return s
    nseq = case["packed"] or B
    s["starts"] = None
    if case["packed"]:
        cuts = _lengths(nseq, B * T, seed)
        s["starts"] = torch.tensor(cuts, dtype=torch.int32, device="cuda")
        s["longest"] = max(b - a for a, b in zip(cuts, cuts[1:]))
    s["s_init"] = normal(nseq, Hv, V, K) if case["carry"] else None
    if case["train"]:
        s["do"] = normal(B, T, Hv, V).to(dt)
        s["dS_final"] = normal(nseq, Hv, V, K) if case["carry"] else None
    return s


# ----------------------------------------------------------------------- the plain forms ---

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


def _g_of(s, dtype):
    """The log decay of every token and value head."""
    g = s["g"].to(dtype)
    return g.expand(*s["v"].shape[:3]) if s["case"]["fixed"] else g


def _lin_plain(s):
    case = s["case"]
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    g = _g_of(s, torch.float32)
    do = s["do"].float() if case["train"] else None
    if s["starts"] is not None:
        at, there = _pad_index(s["starts"], s["longest"])
        at = torch.where(there, at, 0)
        q, k, v, g, do = (None if x is None else torch.where(there.view(*there.shape, *[1] * (x.dim() - 2)), x[0][at], 0.0)
                          for x in (q, k, v, g, do))
    B, T, Hk, K = q.shape
    Hv = v.shape[2]
    group = Hv // Hk
    qc, kc = (_chunks(x.repeat_interleave(group, dim=2)) for x in (q, k))
    vc, gc = _chunks(v), _chunks(g[..., None])[..., 0]
    scale, n = s["scale"], qc.shape[2]
    G = gc.cumsum(-1)
    i = torch.arange(CHUNK, device=q.device)
    ratio = torch.exp(torch.where(i[:, None] >= i, G[..., :, None] - G[..., None, :], -math.inf))
    P = scale * (qc @ kc.mT) * ratio
    head, tail = G.exp()[..., None], (G[..., -1:] - G).exp()[..., None]
    whole = G[..., -1].exp()[..., None, None]
    U = vc.mT @ (tail * kc)
    S = torch.zeros_like(U[:, :, 0]) if s["s_init"] is None else s["s_init"].float()
    states = torch.empty_like(U)
    for c in range(n):
        states[:, :, c] = S
        S = whole[:, :, c] * S + U[:, :, c]
    out = {"o": _whole(P @ vc + scale * head * (qc @ states.mT), T), "s_final": S}
    if case["train"]:
        doc = _chunks(do)
        W = scale * doc.mT @ (head * qc)
        dS = torch.zeros_like(S) if s["dS_final"] is None else s["dS_final"].float()
        dstates = torch.empty_like(W)
        for c in reversed(range(n)):
            dstates[:, :, c] = dS
            dS = whole[:, :, c] * dS + W[:, :, c]
        A = scale * (doc @ vc.mT) * ratio
        dq, dk = scale * head * (doc @ states), tail * (vc @ dstates)  # across chunks, then within
        across = (qc * dq).sum(-1).flip(-1).cumsum(-1).flip(-1)
        before = (kc * dk).sum(-1)
        across = across + before.cumsum(-1) - before + (whole * states * dstates).sum((-1, -2))[..., None]
        # every pair s < t <= i passes the decay of t
        pairs = torch.where(i[:, None] > i, (qc @ kc.mT) * A, 0.0)
        upto = pairs.cumsum(-1) - pairs
        dg = across + torch.where(i[:, None] >= i, upto, 0.0).sum(-2)
        dq, dk = dq + A @ kc, dk + A.mT @ qc
        dv = P.mT @ doc + tail * (kc @ dstates.mT)
        dq, dk = (_whole(x, T).view(B, T, Hk, group, K).sum(3) for x in (dq, dk))
        out |= {"dq": dq, "dk": dk, "dv": _whole(dv, T), "dg": _whole(dg[..., None], T)[..., 0]}
        if s["s_init"] is not None:
            out["dS_init"] = dS
    if s["starts"] is not None:
        for name in [m for m in out if m not in ("s_final", "dS_init")]:
            out[name] = out[name][there][None]
    for name, like in (("o", "v"), ("dq", "q"), ("dk", "k"), ("dv", "v")):
        if name in out:
            out[name] = out[name].to(s[like].dtype)
    if case["train"] and case["fixed"]:
        out["dg"] = out["dg"].double().sum((0, 1)).float()
    return out


def _step_plain(s):
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    g = _g_of(s, torch.float32)
    group = v.shape[2] // q.shape[2]
    q, k = (x.repeat_interleave(group, dim=2) for x in (q, k))
    at = s["slots"].long()
    S, outs = s["state"][at], []
    for t in range(q.shape[1]):
        S = S * g[:, t].exp()[..., None, None] + v[:, t, :, :, None] * k[:, t, :, None]
        outs.append(s["scale"] * (S * q[:, t, :, None]).sum(-1))
    s["state"][at] = S
    return {"o": torch.stack(outs, 1).to(s["v"].dtype), "state": s["state"]}


def _turn(x, cos, sin, interleaved):
    """The pairs of the first dimensions turned; cos and sin [tokens][1][pairs]."""
    half = cos.shape[-1]
    head, rest = x[..., : 2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), rest], -1)
    a, b = head[..., :half], head[..., half:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1)


def _qk_plain(s):
    case = s["case"]
    angle = (s["positions"].double()[:, None] * s["freq"])[:, None]
    cos, sin = angle.cos().float(), angle.sin().float()
    out = {}
    for name in ("q", "k"):
        x, w = s[name].float(), s["w" + name]
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS_NORM)
        out[name] = _turn(x * r * w, cos, sin, case["interleaved"]).to(s[name].dtype)
        if case["train"]:
            d = _turn(s["d" + name].float(), cos, -sin, case["interleaved"])
            u = x * r
            out["d" + name] = (r * (d * w - u * (d * w * u).mean(-1, keepdim=True))).to(s[name].dtype)
            out["dw" + name] = (d * u).sum((0, 1))
    return out


# ---------------------------------------------------------------------- the framework's ---

def _lin_own(s):
    from linear_rnn_state_gb300 import linattn

    case = s["case"]
    opts = {"scale": s["scale"], "seq_starts": s["starts"]}
    ins = [s[n] for n in ("q", "k", "v", "g")]
    o, s_final, saved = linattn.forward(*ins, s["s_init"], want_saved=case["train"], **opts)
    out = {"o": o, "s_final": s_final}
    if case["train"]:
        grads = linattn.backward(*ins, s["do"], saved, dS_final=s["dS_final"], want_dS_init=case["carry"], **opts)
        out |= {n: x for n, x in grads.items() if x is not None}
    return out


def _step_own(s):
    from linear_rnn_state_gb300 import linattn

    o = linattn.step(*(s[n] for n in ("q", "k", "v", "g", "state")), slots=s["slots"], scale=s["scale"])
    return {"o": o, "state": s["state"]}


def _qk_own(s):
    from linear_rnn_state_gb300 import qkrope

    opts = {"positions": s["positions"], "interleaved": s["case"]["interleaved"], "eps": EPS_NORM}
    ins = [s[n] for n in ("q", "k", "wq", "wk", "freq")]
    q, k = qkrope.forward(*ins, **opts)
    out = {"q": q, "k": k}
    if s["case"]["train"]:
        out |= qkrope.backward(*ins, s["dq"], s["dk"], **opts)
    return out


PLAIN = {"lin": _lin_plain, "step": _step_plain, "qk": _qk_plain}
OWN = {"lin": _lin_own, "step": _step_own, "qk": _qk_own}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------------------ 64 bits ---

def _lin_exact(s):
    """Token by token: the recurrence for o and dq, the reverse one for dk and dv. A token's log decay moves
    whatever passes it: what queries from there on read less what they read of keys from there on."""
    case = s["case"]
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    g = _g_of(s, torch.float64)
    there = None
    if s["starts"] is not None:
        at, there = _pad_index(s["starts"], s["longest"])
        at = at.clamp(max=q.shape[1] - 1)

    def spread(x):
        if there is None:
            return x
        x = x[0][at]
        x[~there] = 0
        return x

    q, k, v, g = map(spread, (q, k, v, g))
    B, T, Hk, K = q.shape
    Hv, V = v.shape[2:]
    group, scale = Hv // Hk, s["scale"]
    q, k = q.repeat_interleave(group, 2), k.repeat_interleave(group, 2)
    S = torch.zeros(B, Hv, V, K, device=q.device, dtype=torch.float64) if s["s_init"] is None else s["s_init"].double()
    decay = g.exp()[..., None, None]
    o, dq = torch.empty_like(v), torch.empty_like(q)
    do = spread(s["do"].double()) if case["train"] else None
    for t in range(T):
        S = torch.addcmul(decay[:, t] * S, v[:, t, :, :, None], k[:, t, :, None, :])
        o[:, t] = scale * (S @ q[:, t, :, :, None])[..., 0]
        if case["train"]:
            dq[:, t] = scale * (do[:, t, :, None, :] @ S)[:, :, 0]
    out = {"o": o, "s_final": S}
    if case["train"]:
        D = torch.zeros_like(S) if s["dS_final"] is None else s["dS_final"].double()
        dk, dv = torch.empty_like(k), torch.empty_like(v)
        end = (S * D).sum((-1, -2))
        for t in reversed(range(T)):
            D = torch.addcmul(D, scale * do[:, t, :, :, None], q[:, t, :, None, :])
            dv[:, t] = (D @ k[:, t, :, :, None])[..., 0]
            dk[:, t] = (v[:, t, :, None, :] @ D)[:, :, 0]
            D = decay[:, t] * D
        moved = (q * dq).sum(-1) - (k * dk).sum(-1)
        dg = moved.flip(1).cumsum(1).flip(1) + end[:, None]
        dq, dk = (x.unflatten(2, (Hk, group)).sum(3) for x in (dq, dk))
        out |= {"dq": dq, "dk": dk, "dv": dv, "dg": dg}
        if s["s_init"] is not None:
            out["dS_init"] = D
    if there is not None:
        for name in [m for m in out if m not in ("s_final", "dS_init")]:
            out[name] = out[name][there][None]
    if case["train"] and case["fixed"]:
        out["dg"] = out["dg"].sum((0, 1))
    return out


def _step_exact(s):
    fake = {"case": {**s["case"], "train": False}, "starts": None, "scale": s["scale"],
            "s_init": s["state"][s["slots"].long()], **{n: s[n] for n in ("q", "k", "v", "g")}}
    got = _lin_exact(fake)
    pool = s["state"].double()
    pool[s["slots"].long()] = got["s_final"]
    return {"o": got["o"], "state": pool}


def _qk_exact(s):
    case = s["case"]
    half = s["freq"].shape[0]
    turn = torch.polar(torch.ones((), device="cuda", dtype=torch.float64), s["positions"].double()[:, None] * s["freq"])[:, None]

    def rotate(x, turn):
        head = x[..., : 2 * half]
        pair = head.unflatten(-1, (half, 2)) if case["interleaved"] else head.unflatten(-1, (2, half)).mT
        pair = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        head = pair.flatten(-2) if case["interleaved"] else pair.mT.flatten(-2)
        return torch.cat([head, x[..., 2 * half:]], -1)

    out = {}
    for name in ("q", "k"):
        x, w = s[name].double(), s["w" + name].double()
        rms = (x.square().mean(-1, keepdim=True) + EPS_NORM).sqrt()
        out[name] = rotate(x / rms * w, turn)
        if case["train"]:
            d = rotate(s["d" + name].double(), turn.conj())
            t = d * w
            out["d" + name] = t / rms - x * (t * x).mean(-1, keepdim=True) / rms ** 3
            out["dw" + name] = (d * x / rms).sum((0, 1))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"lin": _lin_exact, "step": _step_exact, "qk": _qk_exact}[case["op"]](s)
