"""GPU tests of the gated delta rule (include/gdr.h) against the fp64 oracle.

Bars, from the kernels' arithmetic. bfloat16 outputs are rounded once (relative
error up to 2^-8 an element, 1.7e-3 in the 2-norm of many) from fp32 results, o
from products whose operands have 11 bits or more: relative 2-norm 2.5e-3 or one
and a half times what rounding the reference itself costs, and every element
within 2^-8 of |ref| + the output's rms. fp32 outputs come from products
of 22-bit operands summed in fp32: each product is within about 2^-22 and a
64-term fp32 sum within 8 * 2^-24 of its terms, some ten of them in a row: 4e-6 in
the 2-norm. dg and dbeta are sums whose terms cancel to a tenth or so: 2e-5.
"""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def env():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_rnn_state_gb300 import _build, gdr

    _build.build()
    gdr.load()
    spec = importlib.util.spec_from_file_location("gdr_oracle", os.path.join(ROOT, "oracle", "gdr_oracle.py"))
    orc = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(orc)
    torch.cuda.set_device(0)
    return orc, gdr


def _close(name, got, ref):
    bf16 = got.dtype == BF16
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), f"{name}: non-finite"
    if ref.size == 0:
        return
    norm, off = np.linalg.norm(ref), np.linalg.norm(got - ref)
    rounding = np.linalg.norm(torch.from_numpy(ref).to(BF16).double().numpy() - ref) if bf16 else 0.0
    if norm == 0:
        assert off == 0, name
        return
    bar = 2.5e-3 if bf16 else 2e-5 if name in ("dg", "dbeta") else 4e-6
    assert off <= max(bar * norm, 1.5 * rounding), f"{name}: relative error {off / norm:.2e} (bar {bar})"
    if bf16:
        rms = norm / np.sqrt(ref.size)
        worst = np.max(np.abs(got - ref) / (np.abs(ref) + rms))
        assert worst <= 2.0 ** -8, f"{name}: element error {worst:.2e}"


def _make(B, T, Hk, Hv, K, V, dtype, seed=0, *, states=None, l2norm=False, rate=1.0, related=0.3):
    """Inputs on the GPU in `dtype`, and the same values in fp64."""
    rng = np.random.default_rng(seed)
    r = rng.standard_normal
    q, k = r((B, T, Hk, K)), r((B, T, Hk, K)) + related * r((B, 1, Hk, K))
    if not l2norm:
        q, k = (x / np.maximum(np.linalg.norm(x, axis=-1, keepdims=True), 1e-9) for x in (q, k))
    x = {"q": q, "k": k, "v": r((B, T, Hv, V)), "do": r((B, T, Hv, V))}
    d = {n: torch.from_numpy(a).to("cuda", dtype) for n, a in x.items()}
    n = B if states is None else states
    x = {"g": -rate * np.abs(r((B, T, Hv))), "beta": rng.random((B, T, Hv)), "s_init": 0.3 * r((n, Hv, V, K)),
         "dS_final": 0.3 * r((n, Hv, V, K))}
    d.update({m: torch.from_numpy(a).to("cuda", F32) for m, a in x.items()})
    return d


def _np(d):
    return {n: x.double().cpu().numpy() for n, x in d.items()}


INS = ("q", "k", "v", "g", "beta")


def _check(env, d, *, carry=True, **opts):
    """Forward and backward of the inputs d against the oracle's."""
    orc, gdr = env
    s0, dS = (d["s_init"], d["dS_final"]) if carry else (None, None)
    o, s, saved = gdr.forward(*(d[n] for n in INS), s0, **opts)
    grads = gdr.backward(*(d[n] for n in INS), d["do"], saved, dS_final=dS, **opts)
    gdr.wkv7.status()
    h = _np(d)
    kw = {"scale": opts.get("scale"), "l2norm": opts.get("qk_l2norm", False)}
    h0, hD = (h["s_init"], h["dS_final"]) if carry else (None, None)
    o_ref, s_ref = orc.forward(*(h[n] for n in INS), h0, **kw)
    _close("o", o, o_ref), _close("s_final", s, s_ref)
    ref = orc.backward(*(h[n] for n in INS), h["do"], h0, hD, **kw)
    for n in ("dq", "dk", "dv", "dg", "dbeta", "dS_init"):
        _close(n, grads[n], ref[n])
    # without what the backward needs: the same results
    o2, s2, none = gdr.forward(*(d[n] for n in INS), s0, want_saved=False, **opts)
    assert none is None
    _close("o", o2, o_ref)
    assert torch.equal(s2, s)
    return o, s, grads


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 63, 64, 65, 127, 128, 200, 449])
def test_lengths(env, T, dtype):
    _check(env, _make(2, T, 1, 2, 64, 64, dtype, T))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("K,V", [(8, 8), (16, 16), (32, 16), (40, 24), (64, 128), (72, 64), (96, 56), (128, 128), (128, 8), (8, 128)])
def test_head_sizes(env, K, V, dtype):
    _check(env, _make(1, 150, 2, 2, K, V, dtype, K + V))


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (1, 5), (2, 4), (3, 9), (7, 7)])
def test_heads(env, Hk, Hv):
    _check(env, _make(3, 100, Hk, Hv, 64, 32, BF16, Hv, l2norm=True), qk_l2norm=True, scale=0.3)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_normalised_heads_of_128(env, dtype):
    _check(env, _make(1, 260, 1, 2, 128, 128, dtype, 5, l2norm=True), qk_l2norm=True)


@pytest.mark.parametrize("B,Hv", [(1, 40), (2, 80)])
def test_more_and_fewer_heads_than_sms(env, B, Hv):
    # the chains' blocks take two or four tiles of value columns
    _check(env, _make(B, 70, Hv, Hv, 16, 64, F32, B), carry=False)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,T", [(2, 8191), (1, 8193), (1, 12345)])
def test_long_sequences_of_few_heads(env, B, T, dtype):
    # 128 chunks, 129 and 193: the forward goes in segments of its own accord
    orc, gdr = env
    d = _make(B, T, 1, 2, 16, 24, dtype, T, rate=0.1)
    o, s, _ = _check(env, d)
    o2, none, _ = gdr.forward(*(d[n] for n in INS), d["s_init"], want_s_final=False)
    assert none is None and torch.equal(o2, o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, s3, _ = gdr.forward(*(d[n] for n in INS), d["s_init"], want_saved=False)
    o3.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(s3, s)
    _close("o", o3, o.double().cpu().numpy())


@pytest.mark.parametrize("Hk,Hv,K,dtype", [(2, 2, 64, F32), (1, 3, 128, BF16), (3, 3, 72, BF16)])
def test_long_sequences_backward_in_segments(env, Hk, Hv, K, dtype):
    orc, gdr = env
    d = _make(1, 8300, Hk, Hv, K, 16, dtype, K, rate=0.1)
    _check(env, d)
    o, s, saved = gdr.forward(*(d[n] for n in INS))
    first = gdr.backward(*(d[n] for n in INS), d["do"], saved, dS_final=d["dS_final"])
    again = gdr.backward(*(d[n] for n in INS), d["do"], saved, dS_final=d["dS_final"], want_dS_init=False)
    assert again["dS_init"] is None
    assert all(torch.equal(first[n], again[n]) for n in ("dq", "dk", "dv", "dg", "dbeta"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = gdr.backward(*(d[n] for n in INS), d["do"], saved, dS_final=d["dS_final"])
    for x in third.values():
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(first[n], third[n]) for n in third)


def test_one_token_from_nothing_has_no_decay_gradient(env):
    _, _, g = _check(env, _make(3, 1, 2, 2, 64, 64, BF16), carry=False)
    assert torch.count_nonzero(g["dg"]) == 0


@pytest.mark.parametrize("rate", [0.0, 1e-4, 0.3, 3.0, 40.0])
def test_decays(env, rate):
    # 3.0 and 40.0: a chunk's decay spans more than the factored form's 60
    _check(env, _make(1, 180, 2, 2, 64, 64, F32, 7, rate=rate))


def test_resets(env):
    """g = -inf empties the state, and lets no gradient through."""
    orc, gdr = env
    d = _make(1, 150, 1, 2, 64, 64, F32, 8)
    for t in (0, 40, 64, 65, 149):
        d["g"][:, t] = -torch.inf
    o, s, saved = gdr.forward(*(d[n] for n in INS), d["s_init"])
    grads = gdr.backward(*(d[n] for n in INS), d["do"], saved, dS_final=d["dS_final"])
    h = _np(d)
    o_ref, s_ref = orc.forward(*(h[n] for n in INS), h["s_init"])
    _close("o", o, o_ref), _close("s_final", s, s_ref)
    h["g"][np.isinf(h["g"])] = -1e3  # the oracle's e^g S: the same, without inf * 0
    ref = orc.backward(*(h[n] for n in INS), h["do"], h["s_init"], h["dS_final"])
    for n in ("dq", "dk", "dv", "dg", "dbeta", "dS_init"):
        _close(n, grads[n], ref[n])
    assert torch.count_nonzero(grads["dS_init"]) == 0 and torch.count_nonzero(grads["dg"][:, 40]) == 0


def test_write_strengths(env):
    """Nothing written, all of it, and the reflections of beta = 2."""
    d = _make(1, 140, 1, 3, 64, 64, F32, 9)
    d["beta"][..., 0], d["beta"][..., 1], d["beta"][..., 2] = 0, 1, 2
    _check(env, d)


def test_the_same_key_every_time(env):
    # L is full: T = (I + L)^-1 by its blocks, without the help of near-orthogonal keys
    d = _make(1, 192, 1, 2, 64, 64, F32, 10)
    d["k"][:] = d["k"][:, :1]
    d["beta"][:] = 1
    d["g"][:] = 0
    _check(env, d)


def test_zero_vectors(env):
    d = _make(1, 100, 2, 2, 64, 64, BF16, 11, l2norm=True)
    d["k"][:, 10:30] = 0
    d["q"][:, 20:40] = 0
    d["v"][:, 64:80] = 0
    _check(env, d, qk_l2norm=True)
    d["do"][:] = 0
    d["dS_final"][:] = 0
    _, _, g = _check(env, d, qk_l2norm=True)
    assert all(torch.count_nonzero(x) == 0 for x in g.values())


def test_states_that_die_away(env):
    """Nothing is written in the last 36 tokens and the state falls to 1e-12 of what
    it was: what the operands' floor (2^-39 of a tile's largest value) leaves is far
    below the state that was, though not below what is left of it."""
    orc, gdr = env
    d = _make(1, 100, 2, 2, 64, 64, BF16, 11, l2norm=True)
    d["v"][:, 64:] = 0
    o, s, _ = gdr.forward(*(d[m] for m in INS), d["s_init"], qk_l2norm=True)
    h = _np(d)
    o_ref, s_ref = orc.forward(*(h[m] for m in INS), h["s_init"], l2norm=True)
    _close("o", o, o_ref)
    largest = max(np.abs(h["v"]).max(), np.abs(h["s_init"]).max())
    assert np.abs(s.double().cpu().numpy() - s_ref).max() <= 2.0 ** -36 * largest


@pytest.mark.parametrize("size", [1e-12, 1e12])
def test_magnitudes(env, size):
    """The fp16 pairs' scales follow the values, row by row and tile by tile."""
    d = _make(1, 130, 1, 2, 64, 64, F32, 12, l2norm=True)
    d["v"] *= size
    d["s_init"] *= size
    d["dS_final"] /= size  # the two parts of the loss are of one size
    d["k"][:, ::3] *= 1e6  # normalised inside; with others of length eight
    d["q"][:, ::5] *= 1e5
    _check(env, d, qk_l2norm=True)


def test_rows_of_different_magnitude(env):
    d = _make(1, 130, 1, 1, 64, 64, F32, 13)
    d["v"] *= torch.logspace(-3, 3, 64, device="cuda")
    _check(env, d)


def test_growing_states(env):
    """g > 0: decays above 1 within a chunk."""
    d = _make(1, 100, 1, 2, 64, 64, F32, 14)
    d["g"] = 0.05 * torch.rand_like(d["g"])
    _check(env, d)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("starts", [[0, 7], [0, 64, 64, 129, 130, 300], [0, 0, 0, 1, 63, 190, 190]], ids=["one", "mixed", "empty"])
def test_packed_sequences(env, starts, dtype):
    orc, gdr = env
    n = len(starts) - 1
    d = _make(1, starts[-1], 2, 4, 64, 64, dtype, 15, states=n)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    o, s, saved = gdr.forward(*(d[m] for m in INS), d["s_init"], seq_starts=st)
    grads = gdr.backward(*(d[m] for m in INS), d["do"], saved, dS_final=d["dS_final"], seq_starts=st)
    h = _np(d)
    fwd = orc.packed(orc.forward, starts, [h[m] for m in INS], {"s_init": h["s_init"]})
    _close("o", o, np.concatenate([x[0] for x in fwd], 1)), _close("s_final", s, np.concatenate([x[1] for x in fwd]))
    bwd = orc.packed(orc.backward, starts, [h[m] for m in INS + ("do",)], {"s_init": h["s_init"], "dS_final": h["dS_final"]})
    for m in ("dq", "dk", "dv", "dg", "dbeta"):
        _close(m, grads[m], np.concatenate([x[m] for x in bwd], 1))
    _close("dS_init", grads["dS_init"], np.concatenate([x["dS_init"] for x in bwd]))


def test_packed_starts_outside_the_tokens_stay_in_bounds(env):
    _, gdr = env
    d = _make(1, 100, 1, 1, 64, 64, BF16, 16, states=3)
    st = torch.tensor([-5, 40, 1000, 90], dtype=torch.int32, device="cuda")  # clamped: 0, 40, 100, 90 (empty)
    o, s, _ = gdr.forward(*(d[m] for m in INS), d["s_init"], seq_starts=st)
    good = torch.tensor([0, 40, 100, 100], dtype=torch.int32, device="cuda")
    o2, s2, _ = gdr.forward(*(d[m] for m in INS), d["s_init"], seq_starts=good)
    gdr.wkv7.status()
    assert torch.equal(o, o2) and torch.equal(s, s2)


def test_empty_calls(env):
    _, gdr = env
    d = _make(2, 0, 1, 2, 64, 64, BF16, 17)
    o, s, saved = gdr.forward(*(d[m] for m in INS), d["s_init"])
    assert o.shape == (2, 0, 2, 64) and torch.equal(s, d["s_init"])
    g = gdr.backward(*(d[m] for m in INS), d["do"], saved, dS_final=d["dS_final"])
    assert torch.equal(g["dS_init"], d["dS_final"])
    assert torch.count_nonzero(gdr.forward(*(d[m] for m in INS))[1]) == 0
    d = _make(0, 5, 1, 2, 64, 64, F32, 17)
    gdr.backward(*(d[m] for m in INS), d["do"], gdr.forward(*(d[m] for m in INS))[2])


def test_slices_of_a_wider_tensor(env):
    """q, k, v of one projection's output, and tokens farther apart than 2^31 elements in all."""
    orc, gdr = env
    d = _make(2, 130, 2, 4, 64, 32, BF16, 18)
    wide = torch.empty((2, 130, 2 * 128 + 128 + 8), dtype=BF16, device="cuda")
    parts = (wide[..., :128], wide[..., 128:256], wide[..., 264:392])
    views = [p.unflatten(-1, (h, -1)) for p, h in zip(parts, (2, 2, 4))]
    for view, n in zip(views, ("q", "k", "v")):
        view.copy_(d[n])
    dense = gdr.forward(*(d[m] for m in INS))
    apart = gdr.forward(*views, d["g"], d["beta"])
    assert torch.equal(dense[0], apart[0]) and torch.equal(dense[1], apart[1])
    a, b = (gdr.backward(*x, d["g"], d["beta"], d["do"], s[2]) for x, s in (((d["q"], d["k"], d["v"]), dense), (views, apart)))
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_offsets_past_32_bits(env):
    orc, gdr = env
    d = _make(1, 66, 1, 1, 64, 64, BF16, 19)
    far = 1 << 25  # 65 of these: 2^31 + 2^25 elements
    buf = torch.empty(65 * far + 192, dtype=BF16, device="cuda")
    views = [buf.as_strided((1, 66, 1, 64), (0, far, 64, 1), 64 * i) for i in range(3)]
    for view, n in zip(views, ("q", "k", "v")):
        view.copy_(d[n])
    o, s, _ = gdr.forward(*views, d["g"], d["beta"])
    o2, s2, _ = gdr.forward(*(d[m] for m in INS))
    assert torch.equal(o, o2) and torch.equal(s, s2)


def test_the_same_bits_every_time(env):
    _, gdr = env
    d = _make(2, 333, 2, 6, 128, 64, BF16, 20)

    def run():
        o, s, saved = gdr.forward(*(d[m] for m in INS), d["s_init"])
        return [o, s, *gdr.backward(*(d[m] for m in INS), d["do"], saved, dS_final=d["dS_final"]).values()]

    first = run()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, run()))


def test_another_stream_and_a_graph(env):
    _, gdr = env
    d = _make(1, 100, 1, 2, 64, 64, BF16, 21)
    want = gdr.forward(*(d[m] for m in INS), d["s_init"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gdr.forward(*(d[m] for m in INS), d["s_init"], stream=side)
    grads = gdr.backward(*(d[m] for m in INS), d["do"], got[2], stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with torch.cuda.stream(side):  # warm, then recorded
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            o, s, saved = gdr.forward(*(d[m] for m in INS), d["s_init"])
            g2 = gdr.backward(*(d[m] for m in INS), d["do"], saved)
    o.zero_(), g2["dg"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(g2["dg"], grads["dg"]) and torch.equal(g2["dq"], grads["dq"])


def test_a_sequence_cut_in_two(env):
    """States and their gradients carry a long sequence over calls."""
    _, gdr = env
    d = _make(1, 200, 1, 2, 64, 64, F32, 22)
    whole = gdr.forward(*(d[m] for m in INS), d["s_init"])
    gw = gdr.backward(*(d[m] for m in INS), d["do"], whole[2], dS_final=d["dS_final"])
    a, b = ({m: d[m][:, s].contiguous() for m in INS + ("do",)} for s in (slice(0, 70), slice(70, 200)))
    fa = gdr.forward(*(a[m] for m in INS), d["s_init"])
    fb = gdr.forward(*(b[m] for m in INS), fa[1])
    gb = gdr.backward(*(b[m] for m in INS), b["do"], fb[2], dS_final=d["dS_final"])
    ga = gdr.backward(*(a[m] for m in INS), a["do"], fa[2], dS_final=gb["dS_init"])
    for name, x, y in [("s_final", fb[1], whole[1]), ("o", torch.cat((fa[0], fb[0]), 1), whole[0])] + [
            (m, torch.cat((ga[m], gb[m]), 1), gw[m]) for m in ("dq", "dk", "dv", "dg", "dbeta")] + [("dS_init", ga["dS_init"], gw["dS_init"])]:
        _close(name, x, y.double().cpu().numpy())


# ------------------------------------------------ roundings, gates, magnitudes ---


def _close_rounded(name, got, ref):
    """A bfloat16 output against its reference rounded to bfloat16. An fp32 result
    that is off by e is rounded to another neighbour with a probability of 2 |e| / ulp
    and then differs by one ulp, at most 2^-7 |x|: the squares sum up to 2^-6 sum |e x|,
    at most 2^-6 |e| |x| in 2-norms. With fp32's bar, 4e-6: 2.5e-4 of the norm."""
    want = torch.from_numpy(ref).to(BF16).double().numpy()
    off = np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)
    assert off <= 2.5e-4, f"{name}: {off:.2e} from the rounded reference"


@pytest.mark.parametrize("K,V", [(64, 64), (128, 128), (40, 24)])
def test_bfloat16_outputs_are_fp32_results_rounded_once(env, K, V):
    orc, gdr = env
    d = _make(2, 300, 2, 4, K, V, BF16, 30, l2norm=True, rate=0.3)
    o, s, saved = gdr.forward(*(d[n] for n in INS), d["s_init"], qk_l2norm=True)
    o2, _, _ = gdr.forward(*(d[n] for n in INS), d["s_init"], qk_l2norm=True, want_saved=False)
    g = gdr.backward(*(d[n] for n in INS), d["do"], saved, dS_final=d["dS_final"], qk_l2norm=True)
    h = _np(d)
    o_ref, _ = orc.forward(*(h[n] for n in INS), h["s_init"], l2norm=True)
    ref = orc.backward(*(h[n] for n in INS), h["do"], h["s_init"], h["dS_final"], l2norm=True)
    _close_rounded("o", o, o_ref), _close_rounded("o without saved", o2, o_ref)
    for n in ("dq", "dk", "dv"):
        _close_rounded(n, g[n], ref[n])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("up", [1e-3, 0.5])
@pytest.mark.parametrize("rate", [0.3, 0.5, 3.0])
def test_growth_among_decays(env, rate, up, dtype):
    """Single tokens with g > 0: what grows from a token to a later one, not the
    chunk's whole span of decays, bounds the gradients' factors."""
    d = _make(1, 150, 1, 2, 64, 64, dtype, 31, rate=rate)
    d["g"][:, ::13] = up
    _check(env, d)


@pytest.mark.parametrize("size", [0.5, 1.0])
@pytest.mark.parametrize("Hk,Hv,K,dtype", [(1, 2, 64, BF16), (2, 2, 128, F32)])
def test_gates_of_both_signs(env, Hk, Hv, K, dtype, size):
    d = _make(1, 150, Hk, Hv, K, 64, dtype, 32)
    d["g"] = size * torch.randn(d["g"].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(32))
    _check(env, d)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_large_gradients_before_large_values(env, dtype):
    """Of a chunk's tokens the first have large gradients and the last large values, which never meet."""
    d = _make(1, 128, 1, 2, 64, 64, dtype, 40, rate=0.1)
    d["do"][:, :32] *= 1e4
    d["v"][:, 32:64] *= 1e4
    _check(env, d)


def test_a_reset_beside_growth(env):
    orc, gdr = env
    d = _make(1, 100, 1, 2, 64, 64, F32, 33, rate=0.1)
    d["g"][:, 20], d["g"][:, 30], d["g"][:, 70] = -torch.inf, 0.01, 0.01
    o, s, saved = gdr.forward(*(d[n] for n in INS), d["s_init"])
    grads = gdr.backward(*(d[n] for n in INS), d["do"], saved, dS_final=d["dS_final"])
    h = _np(d)
    h["g"][np.isinf(h["g"])] = -1e3
    o_ref, s_ref = orc.forward(*(h[n] for n in INS), h["s_init"])
    _close("o", o, o_ref), _close("s_final", s, s_ref)
    ref = orc.backward(*(h[n] for n in INS), h["do"], h["s_init"], h["dS_final"])
    for n in ("dq", "dk", "dv", "dg", "dbeta", "dS_init"):
        _close(n, grads[n], ref[n])


@pytest.mark.parametrize("T", [1, 90])
def test_nothing_to_learn_from_large_queries(env, T):
    """No values, no state and no gradient beside queries of 1e9: all gradients are 0."""
    orc, gdr = env
    d = _make(1, T, 1, 2, 64, 64, F32, 34)
    d["q"] *= 1e9
    d["v"][:], d["do"][:] = 0, 0
    o, s, saved = gdr.forward(*(d[n] for n in INS))
    grads = gdr.backward(*(d[n] for n in INS), d["do"], saved)
    assert torch.count_nonzero(o) == 0 and torch.count_nonzero(s) == 0
    assert all(torch.count_nonzero(x) == 0 for x in grads.values())


@pytest.mark.parametrize("Hk", [1, 2])
@pytest.mark.parametrize("K", [24, 64, 128])
def test_normalised_vectors_whose_squares_pass_fp32(env, K, Hk):
    """Queries and keys of length 1e21, some of their rows: divided by their lengths all the same."""
    orc, gdr = env
    d = _make(2, 130, Hk, 2, K, 64, F32, 35, l2norm=True)
    d["q"][:, ::3] *= 1e20
    d["k"][:, ::5] *= 1e20
    o, s, saved = gdr.forward(*(d[n] for n in INS), d["s_init"], qk_l2norm=True)
    g = gdr.backward(*(d[n] for n in INS), d["do"], saved, dS_final=d["dS_final"], qk_l2norm=True)
    h = _np(d)
    o_ref, s_ref = orc.forward(*(h[n] for n in INS), h["s_init"], l2norm=True)
    ref = orc.backward(*(h[n] for n in INS), h["do"], h["s_init"], h["dS_final"], l2norm=True)
    _close("o", o, o_ref), _close("s_final", s, s_ref)
    for n in ("dv", "dg", "dbeta", "dS_init"):
        _close(n, g[n], ref[n])
    for n, x, step in (("dq", "q", 3), ("dk", "k", 5)):  # a row's gradient is 1e20 smaller where the row is larger
        far = np.zeros(130, bool)
        far[::step] = True
        for rows in (far, ~far):
            _close(n, g[n][:, torch.from_numpy(rows).cuda()], ref[n][:, rows])
    pool = d["s_init"].clone()
    o1 = gdr.step(*(d[n][:, :1].contiguous() for n in INS), pool, qk_l2norm=True)
    o_ref, s_ref = orc.forward(*(h[n][:, :1] for n in INS), h["s_init"], l2norm=True)
    _close("o", o1, o_ref), _close("s_final", pool, s_ref)


# ---------------------------------------------- shared heads, segments, starts ---


@pytest.mark.parametrize("Hk,Hv,K,V,T,l2norm,starts", [
    (16, 32, 128, 128, 640, True, None),
    (16, 48, 96, 16, 640, False, None),
    (20, 40, 128, 24, 500, True, [0, 1, 1, 130, 300, 500]),
], ids=["128", "96", "packed"])
def test_shared_heads_summed_in_the_block(env, Hk, Hv, K, V, T, l2norm, starts):
    """bfloat16, keys wider than 64 and at least 152 chunks of key heads."""
    orc, gdr = env
    n = len(starts) - 1 if starts else 1
    d = _make(1, T, Hk, Hv, K, V, BF16, 36, states=n, l2norm=l2norm, rate=0.3)
    if not starts:
        _check(env, d, qk_l2norm=l2norm)
    kw = {"qk_l2norm": l2norm, "seq_starts": torch.tensor(starts, dtype=torch.int32, device="cuda") if starts else None}

    def run():
        o, s, saved = gdr.forward(*(d[m] for m in INS), d["s_init"], **kw)
        return o, s, gdr.backward(*(d[m] for m in INS), d["do"], saved, dS_final=d["dS_final"], **kw)

    o, s, g = run()
    if starts:
        h = _np(d)
        fwd = orc.packed(orc.forward, starts, [h[m] for m in INS], {"s_init": h["s_init"]}, l2norm=l2norm)
        _close("o", o, np.concatenate([x[0] for x in fwd], 1)), _close("s_final", s, np.concatenate([x[1] for x in fwd]))
        bwd = orc.packed(orc.backward, starts, [h[m] for m in INS + ("do",)], {"s_init": h["s_init"], "dS_final": h["dS_final"]}, l2norm=l2norm)
        for m in ("dq", "dk", "dv", "dg", "dbeta"):
            _close(m, g[m], np.concatenate([x[m] for x in bwd], 1))
        _close("dS_init", g["dS_init"], np.concatenate([x["dS_init"] for x in bwd]))
    for _ in range(3):
        again = run()
        assert torch.equal(o, again[0]) and all(torch.equal(g[m], again[2][m]) for m in g)


def test_shared_heads_summed_in_the_block_by_segments(env):
    _check(env, _make(1, 8300, 2, 4, 128, 16, BF16, 37, rate=0.1, l2norm=True), qk_l2norm=True)


@pytest.mark.parametrize("T,Hk,Hv,dtype", [(4096, 16, 16, F32), (4159, 9, 18, BF16), (8191, 8, 16, F32)])
def test_two_segments_of_many_heads(env, T, Hk, Hv, dtype):
    """64 to 128 chunks and at least 16 chains: two segments, forwards and backwards."""
    _check(env, _make(1, T, Hk, Hv, 16, 16, dtype, 38, rate=0.1))


@pytest.mark.parametrize("B,Hv,V", [(1, 40, 16), (1, 40, 64), (1, 40, 80), (2, 80, 128)])
def test_fewer_and_more_chains_than_sms(env, B, Hv, V):
    """A chain's block has 64 value columns: 40, 40, 80 and 320 of them, whole ones and with columns left over."""
    _check(env, _make(B, 70, Hv, Hv, 16, V, F32, B), carry=False)

@pytest.mark.parametrize("starts", [[0, 0], [30, 30, 30], [100, 100, 100, 100]])
def test_packed_sequences_without_a_token(env, starts):
    """Tokens there are, but the sequences have none: states and their gradients pass through,
    and are there for what follows on the stream."""
    _, gdr = env
    n = len(starts) - 1
    d = _make(1, 100, 1, 2, 64, 64, BF16, 41, states=n)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    for _ in range(5):
        o, s, saved = gdr.forward(*(d[m] for m in INS), d["s_init"], seq_starts=st)
        grads = gdr.backward(*(d[m] for m in INS), d["do"], saved, dS_final=d["dS_final"], seq_starts=st)
        after = s + 1, grads["dS_init"] + 1
        assert torch.equal(after[0], d["s_init"] + 1) and torch.equal(after[1], d["dS_final"] + 1)
    gdr.wkv7.status()


@pytest.mark.parametrize("dtype,Hk,Hv,K,T,starts", [
    (BF16, 1, 2, 64, 100, [0, 40, 70]),
    (F32, 2, 2, 72, 333, [10, 40, 40, 70]),
    (BF16, 2, 4, 128, 6000, [70, 5100]),  # 80 chunks of two key heads: summed in the block
    (F32, 2, 4, 64, 200, [3, 3, 130, 199]),
    (BF16, 1, 2, 64, 90, [50]),  # no sequence at all
    (BF16, 1, 3, 64, 90, [50, 50]),
])
def test_tokens_of_no_sequence(env, dtype, Hk, Hv, K, T, starts):
    """Before the first start and from the last on: o and the gradients are 0 there,
    whatever the buffers held, and the others' are those of the tokens alone."""
    _, gdr = env
    n, V = len(starts) - 1, 80
    d = _make(1, T, Hk, Hv, K, V, dtype, 39, states=n, l2norm=True)
    out = _raw(gdr, d, starts)
    a, b = starts[0], starts[-1]
    cut = {m: x if m in ("s_init", "dS_final") else x[:, a:b].contiguous() for m, x in d.items()}
    want = _raw(gdr, cut, [x - a for x in starts])
    for m, x in out.items():
        if m in ("s_final", "dS_init"):
            assert torch.equal(x, want[m]), m
        else:
            assert torch.equal(x[:, a:b], want[m]), m
            assert torch.count_nonzero(x[:, :a]) == 0 and torch.count_nonzero(x[:, b:]) == 0, m


def _raw(gdr, d, starts):
    """Forward and backward by the C functions, into buffers that hold NaN before."""
    lib = gdr.load()
    q, v = d["q"], d["v"]
    (B, T, Hk, K), (Hv, V), n, bf16 = q.shape, v.shape[2:], len(starts) - 1, q.dtype == BF16
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")

    def nan(*shape, dtype=F32):
        return torch.full(shape, float("nan"), dtype=dtype, device="cuda")

    def junk(size):
        return torch.full((size,), 255, dtype=torch.uint8, device="cuda")

    dims = (B, T, Hk, Hv, K, V, n)
    saved, work = junk(gdr.saved_bytes(*dims, bf16=bf16, for_backward=True)), junk(lib.gdr_backward_bytes(*dims, bf16))
    out = {"o": nan(B, T, Hv, V, dtype=q.dtype), "s_final": nan(n, Hv, V, K)}
    stream, tail = torch.cuda.current_stream().cuda_stream, (None, 0.25, 1)
    p = lambda *xs: [x.data_ptr() for x in xs]
    fn, back = (lib.gdr_forward_bf16, lib.gdr_backward_bf16) if bf16 else (lib.gdr_forward, lib.gdr_backward)
    ins = p(*(d[m] for m in INS))
    assert fn(*ins, *p(d["s_init"], st, out["o"], out["s_final"], saved), *tail, 1, *dims, stream) == 0
    g = {"dq": nan(*q.shape, dtype=q.dtype), "dk": nan(*q.shape, dtype=q.dtype), "dv": nan(*v.shape, dtype=q.dtype),
         "dg": nan(B, T, Hv), "dbeta": nan(B, T, Hv), "dS_init": nan(n, Hv, V, K)}
    assert back(*ins, *p(d["do"], d["dS_final"], st, saved, work, *g.values()), *tail, *dims, stream) == 0
    gdr.wkv7.status()
    return {**out, **g}


# ------------------------------------------------------------------------- step ---


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("K,V,Hk,Hv,T", [(128, 128, 2, 4, 1), (64, 64, 1, 1, 3), (32, 40, 2, 6, 1), (8, 8, 1, 2, 2), (96, 72, 3, 3, 1), (16, 128, 1, 3, 5)])
def test_step(env, K, V, Hk, Hv, T, dtype):
    orc, gdr = env
    d = _make(6, T, Hk, Hv, K, V, dtype, K, states=9, l2norm=True)
    slots = torch.tensor([4, 0, -1, 8, 2, 9], dtype=torch.int32, device="cuda")  # -1 and 9: no state
    pool = d["s_init"].clone()
    o = gdr.step(*(d[m] for m in INS), pool, slots=slots, qk_l2norm=True)
    h = _np(d)
    at = [0, 1, 3, 4]
    idx = [4, 0, 8, 2]
    o_ref, s_ref = orc.forward(*(h[m][at] for m in INS), h["s_init"][idx], l2norm=True)
    want = h["s_init"].copy()
    want[idx] = s_ref
    _close("o", o[at], o_ref), _close("s_final", pool, want)
    assert torch.count_nonzero(o[[2, 5]]) == 0
    keep = [i for i in range(9) if i not in idx]
    assert torch.equal(pool[keep], d["s_init"][keep])


def test_steps_continue_a_prefill(env):
    _, gdr = env
    d = _make(2, 40, 2, 4, 64, 64, F32, 23)
    o, s, _ = gdr.forward(*(d[m] for m in INS), d["s_init"], want_saved=False)
    _, state, _ = gdr.forward(*(d[m][:, :30].contiguous() for m in INS), d["s_init"], want_saved=False)
    outs = []
    for t in range(30, 40):
        outs.append(gdr.step(*(d[m][:, t:t + 1] if m in "qkv" else d[m][:, t:t + 1].contiguous() for m in INS), state))
    _close("o", torch.cat(outs, 1), o[:, 30:].double().cpu().numpy())
    _close("s_final", state, s.double().cpu().numpy())


def test_step_with_a_pool_past_32_bits(env):
    orc, gdr = env
    d = _make(2, 1, 1, 1, 128, 128, BF16, 24)
    n = (1 << 32) // (128 * 128) + 2  # elements past 2^32
    pool = torch.empty((n, 1, 128, 128), device="cuda")
    pool[n - 1], pool[1] = d["s_init"][0], d["s_init"][1]
    o = gdr.step(*(d[m] for m in INS), pool, slots=torch.tensor([n - 1, 1], dtype=torch.int32, device="cuda"))
    h = _np(d)
    o_ref, s_ref = orc.forward(*(h[m] for m in INS), h["s_init"])
    _close("o", o, o_ref)
    _close("s_final", pool[[n - 1, 1]], s_ref)


def test_step_resets(env):
    orc, gdr = env
    d = _make(2, 1, 1, 1, 64, 64, F32, 25)
    d["g"][0] = -torch.inf
    pool = d["s_init"].clone()
    o = gdr.step(*(d[m] for m in INS), pool)
    h = _np(d)
    o_ref, s_ref = orc.forward(*(h[m] for m in INS), h["s_init"])
    _close("o", o, o_ref), _close("s_final", pool, s_ref)


def test_empty_step(env):
    _, gdr = env
    d = _make(0, 1, 1, 1, 64, 64, F32, 26)
    assert gdr.step(*(d[m] for m in INS), torch.zeros(3, 1, 64, 64, device="cuda")).shape == (0, 1, 1, 64)


# -------------------------------------------------------------------- refusals ---


def test_refusals(env):
    _, gdr = env
    d = _make(1, 8, 1, 2, 64, 64, BF16, 27)
    ins = [d[m] for m in INS]

    def bad(i, x, exc):
        with pytest.raises(exc):
            gdr.forward(*ins[:i], x, *ins[i + 1:])

    bad(0, d["q"].half(), TypeError)
    bad(1, d["k"][:, :4], ValueError)
    bad(1, d["k"].float(), TypeError)
    bad(2, d["v"].cpu(), ValueError)
    bad(3, d["g"].bfloat16(), TypeError)
    bad(4, d["beta"].transpose(1, 2), ValueError)
    bad(2, d["v"].transpose(2, 3), ValueError)
    with pytest.raises(gdr.wkv7.Wkv7Error):
        gdr.forward(d["q"][..., :60], d["k"][..., :60], *ins[2:])
    with pytest.raises(ValueError):
        gdr.forward(*ins, d["s_init"][:, :1])
    with pytest.raises(ValueError):
        gdr.backward(*ins, d["do"], None)
    with pytest.raises(ValueError):
        gdr.backward(*ins, d["do"], gdr.forward(*ins, want_saved=True)[2][:-1])
    with pytest.raises(TypeError):
        gdr.step(*ins, d["s_init"].bfloat16())
    with pytest.raises(TypeError):
        gdr.step(*ins, d["s_init"], slots=torch.zeros(1, device="cuda"))
    two = _make(2, 8, 1, 2, 64, 64, BF16, 27)
    with pytest.raises(gdr.wkv7.Wkv7Error):
        gdr.forward(*(two[m] for m in INS), seq_starts=torch.tensor([0, 8], dtype=torch.int32, device="cuda"))
