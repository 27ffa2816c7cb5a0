"""GPU tests of the norms of queries and keys with the position rotation
(include/qkrope.h) against the fp64 oracle, and of the operators of a linear attention
layer together.

Bars: fp32 arithmetic over rows of up to 256 and angles within 2^-25 of half a turn
(1e-7 of a pair) give 2e-6 in the 2-norm; the weights' sums run over up to 10^5 terms of both signs
in partial sums of 100 or so: 4e-6. bfloat16 outputs are rounded once: 2.5e-3, or one and a half
times what rounding the reference itself costs, and every element within 2^-8 of |ref| + rms.
"""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F32 = torch.bfloat16, torch.float32


def _load(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, "oracle", name + ".py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.fixture(scope="module")
def env():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_rnn_state_gb300 import _build, qkrope

    _build.build()
    qkrope.load()
    torch.cuda.set_device(0)
    return _load("qkrope_oracle"), qkrope


def _close(name, got, ref):
    bf16 = got.dtype == BF16
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), name
    if ref.size == 0:
        return
    norm, off = np.linalg.norm(ref), np.linalg.norm(got - ref)
    rounding = np.linalg.norm(torch.from_numpy(ref).to(BF16).double().numpy() - ref) if bf16 else 0.0
    if norm == 0:
        assert off == 0, name
        return
    bar = 2.5e-3 if bf16 else 4e-6 if name.startswith("dw") else 2e-6
    assert off <= max(bar * norm, 1.5 * rounding), f"{name}: {off / norm:.2e}"
    if bf16:
        worst = np.max(np.abs(got - ref) / (np.abs(ref) + norm / np.sqrt(ref.size)))
        assert worst <= 2.0 ** -8, f"{name}: element {worst:.2e}"


def _make(tokens, Hq, Hk, D, half, dtype, seed=0, far=1 << 20):
    rng = np.random.default_rng(seed)
    t = lambda a, dt=dtype: torch.from_numpy(np.asarray(a)).to("cuda", dt)
    r = rng.standard_normal
    return {"q": t(2 * r((tokens, Hq, D))), "k": t(0.3 * r((tokens, Hk, D))), "wq": t(1 + 0.2 * r(D), F32), "wk": t(r(D), F32),
            "freq": t(10000.0 ** (-np.arange(half) / max(half, 1)), torch.float64),
            "positions": t(rng.integers(-far, far, tokens), torch.int32), "dq": t(r((tokens, Hq, D))), "dk": t(r((tokens, Hk, D)))}


ARGS = ("q", "k", "wq", "wk", "freq")


def _n(x):
    return x.cpu().numpy() if x.dtype is torch.int32 else x.double().cpu().numpy()


def _check(env, d, *, interleaved=False, eps=1e-6, positions=True):
    orc, qr = env
    opts = {"interleaved": interleaved, "eps": eps}
    pos = d["positions"] if positions else None
    at = _n(d["positions"]) if positions else np.broadcast_to(np.arange(d["q"].shape[-3]), d["q"].shape[:-2])
    q, k = qr.forward(*(d[n] for n in ARGS), pos, **opts)
    g = qr.backward(*(d[n] for n in ARGS), d["dq"], d["dk"], pos, **opts)
    for name, y in (("q", q), ("k", k)):
        x, w, f = _n(d[name]), _n(d["w" + name]), _n(d["freq"])
        _close(name, y, orc.forward(x, w, f, at, **opts))
        dx, dw = orc.backward(x, w, f, at, _n(d["d" + name]), **opts)
        _close("d" + name, g["d" + name], dx), _close("dw" + name, g["dw" + name], dw)
    return q, k, g


BOTH = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])


@BOTH
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("D,half", [(8, 4), (8, 1), (16, 8), (32, 16), (40, 8), (64, 32), (64, 16), (96, 48), (96, 37), (128, 64), (128, 3), (192, 96), (256, 128),
                                    (256, 0), (248, 124)])
def test_sizes(env, D, half, interleaved, dtype):
    _check(env, _make(37, 3, 2, D, half, dtype, D + half), interleaved=interleaved)


@BOTH
@pytest.mark.parametrize("tokens,Hq,Hk", [(1, 1, 1), (1, 32, 8), (2, 5, 1), (3, 64, 64), (700, 1, 1), (300, 7, 3), (5000, 8, 8), (600, 32, 8), (2500, 6, 2)])
def test_tokens_and_heads(env, tokens, Hq, Hk, dtype):
    """From one row to more units than blocks, and heads that do not fill a unit."""
    _check(env, _make(tokens, Hq, Hk, 64, 32, dtype, tokens))


@pytest.mark.parametrize("Hq,Hk", [(0, 2), (3, 0)])
def test_queries_or_keys_alone(env, Hq, Hk):
    _, _, g = _check(env, _make(50, Hq, Hk, 64, 32, BF16, Hq))
    assert torch.count_nonzero(g["dwq" if Hq == 0 else "dwk"]) == 0


@BOTH
def test_positions_along_a_batch(env, dtype):
    d = _make(2 * 50, 4, 2, 64, 32, dtype, 3)
    for n in ("q", "k", "dq", "dk"):
        d[n] = d[n].unflatten(0, (2, 50))
    _check(env, d, positions=False)
    d["positions"] = d["positions"].view(2, 50)
    _check(env, d)


def test_far_positions(env):
    """To the ends of 32 bits: the angles are as exact as near 0."""
    orc, qr = env
    d = _make(6, 2, 2, 128, 64, F32, 4)
    d["positions"][:] = torch.tensor([0, 1, -1, (1 << 31) - 1, -(1 << 31), 123456789])
    q, k = qr.forward(*(d[n] for n in ARGS), d["positions"])
    # fp64 angles of 2^31 are off by 2^-22 (2.4e-7): compared pair by pair within that and the fp32 bar
    ref = orc.forward(_n(d["q"]), _n(d["wq"]), _n(d["freq"]), _n(d["positions"]))
    rms = np.sqrt((ref ** 2).mean())
    assert np.abs(q.double().cpu().numpy() - ref).max() <= 4e-6 * max(rms, np.abs(ref).max())
    # a whole turn: positions whose angle is a multiple of 2 pi leave the values alone
    d["freq"][:] = 2 * np.pi
    y, _ = qr.forward(*(d[n] for n in ARGS), torch.full_like(d["positions"], 4096))
    z, _ = qr.forward(*(d[n] for n in ARGS), torch.zeros_like(d["positions"]))
    assert (y - z).abs().max() <= 2e-6 * z.abs().max()  # (2 pi to 2^-53, 4096 times: 1e-12; the sine's own error)


@BOTH
def test_rows_of_zeros_and_of_any_size(env, dtype):
    d = _make(40, 2, 2, 64, 32, dtype, 5)
    d["q"][:10] = 0
    d["q"][10:20] *= 1e-12
    d["k"][10:20] *= 1e12
    _check(env, d, eps=1e-6)


@BOTH
def test_slices_of_a_wider_tensor(env, dtype):
    _, qr = env
    d = _make(300, 4, 2, 64, 24, dtype, 6)
    wide = torch.full((300, 6 * 64 + 128), float("nan"), dtype=dtype, device="cuda")
    q, k = wide[:, 64:320].unflatten(-1, (4, 64)), wide[:, 320:448].unflatten(-1, (2, 64))
    q.copy_(d["q"]), k.copy_(d["k"])
    want, got = (qr.forward(x, y, *(d[n] for n in ARGS[2:]), d["positions"]) for x, y in ((d["q"], d["k"]), (q, k)))
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    a, b = (qr.backward(x, y, *(d[n] for n in ARGS[2:]), d["dq"], d["dk"], d["positions"]) for x, y in ((d["q"], d["k"]), (q, k)))
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_offsets_past_32_bits(env):
    _, qr = env
    d = _make(66, 1, 1, 64, 32, BF16, 7)
    far = 1 << 25
    buf = torch.empty(65 * far + 128, dtype=BF16, device="cuda")
    q, k = (buf.as_strided((66, 1, 64), (far, 64, 1), 64 * i) for i in range(2))
    q.copy_(d["q"]), k.copy_(d["k"])
    want, got = (qr.forward(x, y, *(d[n] for n in ARGS[2:]), d["positions"]) for x, y in ((d["q"], d["k"]), (q, k)))
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_nothing(env):
    _, qr = env
    d = _make(0, 2, 2, 64, 32, F32, 8)
    q, k = qr.forward(*(d[n] for n in ARGS), d["positions"])
    assert q.shape == (0, 2, 64) and k.shape == (0, 2, 64)
    g = qr.backward(*(d[n] for n in ARGS), d["dq"], d["dk"], d["positions"])
    assert torch.count_nonzero(g["dwq"]) == 0 and torch.count_nonzero(g["dwk"]) == 0


@BOTH
def test_another_stream_a_graph_and_the_same_bits(env, dtype):
    _, qr = env
    d = _make(3000, 8, 4, 128, 64, dtype, 9)
    run = lambda **kw: (*qr.forward(*(d[n] for n in ARGS), d["positions"], **kw),
                        *qr.backward(*(d[n] for n in ARGS), d["dq"], d["dk"], d["positions"], **kw).values())
    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = run()
    for x in again:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, again))


@BOTH
def test_values_that_are_not_numbers_stay_in_their_row(env, dtype):
    _, qr = env
    d = _make(500, 6, 3, 64, 32, dtype, 11)
    run = lambda: (*qr.forward(*(d[n] for n in ARGS), d["positions"]),
                   *(qr.backward(*(d[n] for n in ARGS), d["dq"], d["dk"], d["positions"])[n] for n in ("dq", "dk")))
    want = run()
    keep = torch.ones(500, 6, dtype=torch.bool, device="cuda")
    for t, h in ((0, 0), (17, 5), (499, 2)):
        d["q"][t, h, 5], keep[t, h] = float("nan"), False
    d["dq"][250, 1, 60], keep[250, 1] = float("inf"), False
    got = run()
    assert all(torch.equal(x[keep] if x.shape[1] == 6 else x, y[keep] if y.shape[1] == 6 else y) for x, y in zip(want, got))


def test_refusals(env):
    _, qr = env
    d = _make(8, 4, 2, 64, 32, BF16, 10)
    ins = [d[n] for n in ARGS]

    def bad(i, x, exc):
        with pytest.raises(exc):
            qr.forward(*ins[:i], x, *ins[i + 1:], d["positions"])

    bad(0, d["q"].half(), TypeError)
    bad(1, d["k"].float(), TypeError)
    bad(1, d["k"][:4], ValueError)
    bad(1, d["k"].cpu(), ValueError)
    bad(2, d["wq"][:32], ValueError)
    bad(3, d["wk"].bfloat16(), TypeError)
    bad(4, d["freq"].float(), TypeError)
    bad(4, torch.ones(33, dtype=torch.float64, device="cuda"), qr.wkv7.Wkv7Error)
    bad(0, d["q"].transpose(1, 2), ValueError)
    with pytest.raises(TypeError):
        qr.forward(*ins, d["positions"].long())
    with pytest.raises(ValueError):
        qr.forward(*ins, d["positions"][:4])
    with pytest.raises(qr.wkv7.Wkv7Error):
        qr.forward(d["q"][..., :60].contiguous(), d["k"][..., :60].contiguous(), d["wq"][:60].contiguous(), d["wk"][:60].contiguous(), d["freq"][:8])
    with pytest.raises(ValueError):
        qr.backward(*ins, d["dq"][:4], d["dk"], d["positions"])


@BOTH
@pytest.mark.parametrize("eps", [0.0, 1e-2])
@pytest.mark.parametrize("tokens,Hq,Hk,D", [(5, 3, 2, 64), (37, 3, 2, 24), (600, 33, 9, 64), (2500, 6, 2, 128), (1, 1, 1, 256)])
def test_other_eps(env, tokens, Hq, Hk, D, eps, dtype):
    """Also none at all: places of a block without a head, and heads that do not fill a unit, add nothing to the weights'
    gradients (rows of zeros there have no norm where eps is 0)."""
    _check(env, _make(tokens, Hq, Hk, D, D // 4, dtype, tokens + D), eps=eps)


@BOTH
@pytest.mark.parametrize("interleaved,half", [(False, 32), (False, 13), (True, 20)])
def test_rows_whose_squares_leave_fp32(env, interleaved, half, dtype):
    """Rows of 1e25 and 1e30, and (without an eps) of 1e-25, beside others: each by itself as exact as they are, and the others' bits stay."""
    orc, qr = env
    d = _make(70, 7, 3, 64, half, dtype, 14)
    opts = {"interleaved": interleaved, "eps": 0.0}
    run = lambda: (*qr.forward(*(d[n] for n in ARGS), d["positions"], **opts),
                   *qr.backward(*(d[n] for n in ARGS), d["dq"], d["dk"], d["positions"], **opts).values())
    want = run()
    for t, h, size in ((0, 0, 1e25), (3, 6, 1e30), (40, 2, 1e-25), (69, 5, 1e25)):
        d["q"][t, h] *= size
    d["k"][::9, 1] *= 1e30
    d["k"][5, 2] *= 1e-25
    got = run()
    for i, (name, x) in enumerate((("q", "q"), ("k", "k"), ("q", "dq"), ("k", "dk"))):
        a, w, f, at = _n(d[name]), _n(d["w" + name]), _n(d["freq"]), _n(d["positions"])
        ref = orc.forward(a, w, f, at, **opts) if i < 2 else orc.backward(a, w, f, at, _n(d["d" + name]), **opts)[0]
        y = got[i].double().cpu().numpy()
        off = np.linalg.norm(y - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
        # (one row's 64 roundings to bfloat16: 2^-8 of each at most)
        assert off.max() <= (2.0 ** -8 if dtype is BF16 else 4e-6), (x, off.max())
        moved = torch.ones(70, got[i].shape[1], dtype=torch.bool, device="cuda")
        if name == "q":
            for t, h in ((0, 0), (3, 6), (40, 2), (69, 5)):
                moved[t, h] = False
        else:
            moved[::9, 1] = moved[5, 2] = False
        assert torch.equal(got[i][moved], want[i][moved])
    for i, name in ((4, "q"), (5, "k")):
        ref = orc.backward(_n(d[name]), _n(d["w" + name]), _n(d["freq"]), _n(d["positions"]), _n(d["d" + name]), **opts)[1]
        _close("dw" + name, got[i], ref)


# ------------------------------------------------------------- a layer of them all ---


class _Rope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, freq, positions):
        from linear_rnn_state_gb300 import qkrope

        ctx.save_for_backward(q, k, wq, wk, freq, positions)
        return qkrope.forward(q, k, wq, wk, freq, positions)

    @staticmethod
    def backward(ctx, dq, dk):
        from linear_rnn_state_gb300 import qkrope

        q, k, wq, wk, freq, positions = ctx.saved_tensors
        g = qkrope.backward(q, k, wq, wk, freq, dq.contiguous(), dk.contiguous(), positions)
        return g["dq"], g["dk"], g["dwq"], g["dwk"], None, None


class _Attend(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, starts):
        from linear_rnn_state_gb300 import linattn

        o, s, saved = linattn.forward(q, k, v, g, seq_starts=starts)
        ctx.save_for_backward(q, k, v, g, saved)
        ctx.starts = starts
        return o, s

    @staticmethod
    def backward(ctx, do, ds):
        from linear_rnn_state_gb300 import linattn

        q, k, v, g, saved = ctx.saved_tensors
        d = linattn.backward(q, k, v, g, do.contiguous(), saved, dS_final=ds.contiguous(), want_dS_init=False, seq_starts=ctx.starts)
        return d["dq"], d["dk"], d["dv"], d["dg"], None


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, o, z, weight):
        from linear_rnn_state_gb300 import blocknorm

        y, rstd = blocknorm.gated_forward(o, z, weight)
        ctx.save_for_backward(o, z, weight, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        from linear_rnn_state_gb300 import blocknorm

        o, z, weight, rstd = ctx.saved_tensors
        g = blocknorm.gated_backward(o, z, weight, rstd, dy.contiguous())
        return g["do"], g["dz"], g["dweight"]


def _layer(p, x, positions, starts):
    """x [T][width] of packed sequences -> (the layer's output, the final states): a projection, the norms with
    the rotation, linear attention with a learned decay a head, the gated norm, a projection."""
    q, k, v, z = (x @ p["w_in"]).split([2 * 64, 2 * 64, 4 * 32, 4 * 32], -1)
    q, k = _Rope.apply(q.unflatten(-1, (2, 64)), k.unflatten(-1, (2, 64)), p["wq"], p["wk"], p["freq"], positions)
    o, s = _Attend.apply(q[None], k[None], v.unflatten(-1, (4, 32))[None], -p["rate"].exp(), starts)
    return _Norm.apply(o[0], z.unflatten(-1, (4, 32)), p["norm"]).flatten(-2) @ p["w_out"], s


def _parameters(dtype):
    gen = torch.Generator("cuda").manual_seed(0)
    n = lambda *s: torch.randn(s, device="cuda", generator=gen)
    p = {"w_in": (n(96, 512) * 96 ** -0.5).to(dtype), "w_out": (n(128, 96) * 128 ** -0.5).to(dtype), "wq": 1 + 0.1 * n(64), "wk": 1 + 0.1 * n(64),
         "norm": 1 + 0.1 * n(32), "rate": torch.linspace(-4.0, 0.0, 4, device="cuda")}
    p = {m: x.requires_grad_() for m, x in p.items()}
    p["freq"] = 10000.0 ** (-torch.arange(32, device="cuda", dtype=torch.float64) / 32)
    return p


STARTS = [0, 150, 151, 420]


@pytest.fixture(scope="module")
def packed_input(env):
    x = torch.randn(420, 96, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    at = torch.cat([torch.arange(b - a) for a, b in zip(STARTS, STARTS[1:])]).to("cuda", torch.int32)
    return x, at, torch.tensor(STARTS, dtype=torch.int32, device="cuda")


def test_a_layer_s_slope_against_differences(packed_input):
    """The loss's slope along random directions of all parameters, by central differences of steps of 1e-2
    times a direction of unit length a parameter: fp32 losses of order 100 (rounding 1e-5, over 2e-2: 1e-3) and a third
    derivative's term of about 1e-4 of a slope of order 10: 1 %."""
    x, at, starts = packed_input
    p = _parameters(F32)
    gen = torch.Generator("cuda").manual_seed(2)
    target = torch.randn(420, 96, device="cuda", generator=gen)

    def loss():
        y, s = _layer(p, x, at, starts)
        return (y.double() * target).sum() + 0.01 * (s.double() ** 2).sum()

    loss().backward()
    names = [m for m in p if m != "freq"]
    for trial in range(3):
        way = {m: torch.randn(p[m].shape, device="cuda", generator=gen) for m in names}
        way = {m: w / w.norm() for m, w in way.items()}
        slope = sum((p[m].grad.double() * way[m]).sum() for m in names)
        with torch.no_grad():
            ends = []
            for sign in (1e-2, -1e-2):
                for m in names:
                    p[m] += sign * way[m]
                ends.append(loss())
                for m in names:
                    p[m] -= sign * way[m]
        numeric = (ends[0] - ends[1]) / 2e-2
        scale = sum(float((p[m].grad.double().norm())) for m in names)
        assert abs(numeric - slope) <= 1e-2 * max(abs(float(slope)), 0.05 * scale), (trial, float(slope), float(numeric))


@pytest.mark.parametrize("dtype,bar", [(F32, 2e-5), (BF16, 4e-2)], ids=["f32", "bf16"])
def test_a_layer_decodes_as_it_prefills(packed_input, dtype, bar):
    """The next tokens of prefilled sequences, one at a time from a pool of states, are those of the whole sequences.
    fp32: ten fp32 sums of some hundred terms. bfloat16: four roundings (2^-9 each in the mean) on each way, the
    gated norm's row of 32 divided by its own length: 1 % in the mean, 4 % at most."""
    from linear_rnn_state_gb300 import blocknorm, linattn, qkrope

    x, at, starts = packed_input
    x = x.to(dtype)
    p = {m: w.detach() for m, w in _parameters(dtype).items()}
    with torch.no_grad():
        whole, _ = _layer(p, x, at, starts)
        # of each sequence all but the last five tokens (the second has one)
        cuts = [(a, b - 5 if b - a > 5 else b) for a, b in zip(STARTS, STARTS[1:])]
        rows = torch.cat([torch.arange(a, b) for a, b in cuts]).cuda()
        sub = torch.tensor([0, 145, 146, 410], dtype=torch.int32, device="cuda")
        _, states = _layer(p, x[rows], at[rows], sub)
        pool = torch.zeros(5, 4, 32, 64, device="cuda")
        slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
        pool[3], pool[1] = states[0], states[2]
        for i in range(5):
            now = torch.tensor([145 + i, 415 + i], device="cuda")
            q, k, v, z = (x[now] @ p["w_in"]).split([128, 128, 128, 128], -1)
            q, k = qkrope.forward(q.unflatten(-1, (2, 64))[:, None], k.unflatten(-1, (2, 64))[:, None], p["wq"], p["wk"], p["freq"], at[now][:, None])
            o = linattn.step(q, k, v.unflatten(-1, (4, 32))[:, None], -p["rate"].exp(), pool, slots=slots)
            y = blocknorm.gated_forward(o[:, 0], z.unflatten(-1, (4, 32)), p["norm"])[0].flatten(-2) @ p["w_out"]
            want = whole[now].double()
            assert (y.double() - want).norm() <= bar * want.norm(), i
