"""GPU tests of linear attention with a decay (include/linattn.h) against the fp64 oracle.

Bars, from the kernels' arithmetic. bfloat16 outputs are rounded once (relative error
up to 2^-8 an element, 1.7e-3 in the 2-norm of many) from products whose operands have
16 bits or more (2^-18 of a value each): relative 2-norm 2.5e-3 or one and a half times what
rounding the reference itself costs, and every element within 2^-8 of |ref| + the output's
rms. fp32 outputs come from products of 24-bit operands summed in fp32: a product is within
2^-23 and a sum of 128 terms, cut at each of its steps, within 8 * 2^-23 of its terms, some ten of
them in a row: 4e-6 in the 2-norm. dg is a sum over the pairs that pass a token, whose terms
cancel to a tenth or so: 2e-5.
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
    from linear_rnn_state_gb300 import _build, linattn

    _build.build()
    linattn.load()
    spec = importlib.util.spec_from_file_location("linattn_oracle", os.path.join(ROOT, "oracle", "linattn_oracle.py"))
    orc = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(orc)
    torch.cuda.set_device(0)
    return orc, linattn


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
    bar = 2.5e-3 if bf16 else 2e-5 if name == "dg" else 4e-6
    assert off <= max(bar * norm, 1.5 * rounding), f"{name}: relative error {off / norm:.2e} (bar {bar})"
    if bf16:
        worst = np.max(np.abs(got - ref) / (np.abs(ref) + norm / np.sqrt(ref.size)))
        assert worst <= 2.0 ** -8, f"{name}: element error {worst:.2e}"


INS = ("q", "k", "v", "g")
GRADS = ("dq", "dk", "dv", "dg", "dS_init")


def _make(B, T, Hk, Hv, K, V, dtype, seed=0, *, states=None, rate=0.3, fixed=False):
    """Inputs on the GPU in `dtype` (states and decays fp32)."""
    rng = np.random.default_rng(seed)
    r = rng.standard_normal
    x = {"q": r((B, T, Hk, K)), "k": r((B, T, Hk, K)), "v": r((B, T, Hv, V)), "do": r((B, T, Hv, V))}
    d = {n: torch.from_numpy(a).to("cuda", dtype) for n, a in x.items()}
    n = B if states is None else states
    x = {"g": -rate * np.abs(r((Hv,) if fixed else (B, T, Hv))), "s_init": r((n, Hv, V, K)), "dS_final": r((n, Hv, V, K))}
    d.update({m: torch.from_numpy(a).to("cuda", F32) for m, a in x.items()})
    return d


def _np(d):
    return {n: x.double().cpu().numpy() for n, x in d.items()}


def _check(env, d, *, carry=True, **opts):
    """Forward and backward of the inputs d against the oracle's."""
    orc, la = env
    s0, dS = (d["s_init"], d["dS_final"]) if carry else (None, None)
    o, s, saved = la.forward(*(d[n] for n in INS), s0, **opts)
    grads = la.backward(*(d[n] for n in INS), d["do"], saved, dS_final=dS, **opts)
    la.wkv7.status()
    h = _np(d)
    h0, hD = (h["s_init"], h["dS_final"]) if carry else (None, None)
    o_ref, s_ref = orc.forward(*(h[n] for n in INS), h0, **opts)
    _close("o", o, o_ref), _close("s_final", s, s_ref)
    ref = orc.backward(*(h[n] for n in INS), h["do"], h0, hD, **opts)
    for n in GRADS:
        _close(n, grads[n], ref[n])
    # without what the backward needs: the same results
    o2, s2, none = la.forward(*(d[n] for n in INS), s0, want_saved=False, **opts)
    assert none is None and torch.equal(o2, o) and torch.equal(s2, s)
    return o, s, grads


BOTH = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])


@BOTH
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 127, 128, 129, 255, 257, 449])
def test_lengths(env, T, dtype):
    _check(env, _make(2, T, 1, 2, 64, 64, dtype, T))


@BOTH
@pytest.mark.parametrize("K,V", [(8, 8), (16, 16), (32, 16), (40, 24), (64, 128), (72, 64), (96, 56), (128, 128), (128, 8), (8, 128), (128, 96)])
def test_head_sizes(env, K, V, dtype):
    _check(env, _make(1, 150, 2, 2, K, V, dtype, K + V))


@BOTH
@pytest.mark.parametrize("Hk,Hv,K,V", [(1, 1, 64, 32), (1, 5, 64, 64), (2, 4, 128, 128), (3, 9, 40, 72), (7, 7, 16, 64)])
def test_heads(env, Hk, Hv, K, V, dtype):
    _check(env, _make(3, 140, Hk, Hv, K, V, dtype, Hv), scale=0.3)


@BOTH
@pytest.mark.parametrize("Hk,Hv,K", [(2, 2, 64), (2, 6, 128), (300, 300, 8)])
def test_fixed_decays(env, Hk, Hv, K, dtype):
    """One decay a head for all tokens, and the sums of its gradients."""
    _check(env, _make(2, 130, Hk, Hv, K, 16, dtype, 3, fixed=True))


def test_fixed_decays_are_those_of_every_token(env):
    _, la = env
    d = _make(2, 200, 1, 2, 64, 64, BF16, 4, fixed=True)
    o, s, saved = la.forward(*(d[m] for m in INS), d["s_init"])
    each = d["g"].expand(2, 200, 2).contiguous()
    o2, s2, saved2 = la.forward(d["q"], d["k"], d["v"], each, d["s_init"])
    assert torch.equal(o, o2) and torch.equal(s, s2)
    a = la.backward(*(d[m] for m in INS), d["do"], saved)
    b = la.backward(d["q"], d["k"], d["v"], each, d["do"], saved2)
    assert all(torch.equal(a[m], b[m]) for m in ("dq", "dk", "dv"))
    _close("dg", a["dg"], b["dg"].double().sum((0, 1)).cpu().numpy())


@BOTH
def test_gradients_that_are_not_wanted(env, dtype):
    _, la = env
    for fixed in (False, True):
        d = _make(1, 140, 1, 2, 64, 64, dtype, 5, fixed=fixed)
        saved = la.forward(*(d[m] for m in INS), d["s_init"])[2]
        full = la.backward(*(d[m] for m in INS), d["do"], saved)
        some = la.backward(*(d[m] for m in INS), d["do"], saved, want_dg=False, want_dS_init=False)
        assert some["dg"] is None and some["dS_init"] is None
        assert all(torch.equal(some[m], full[m]) for m in ("dq", "dk", "dv"))


@BOTH
@pytest.mark.parametrize("rate", [0.0, 1e-4, 3.0, 40.0])
def test_decays(env, rate, dtype):
    # 3.0 and 40.0: 32 tokens' decays span more than the factored form's 60
    _check(env, _make(1, 280, 1, 2, 64, 64, dtype, 7, rate=rate))


@BOTH
@pytest.mark.parametrize("K", [64, 128])
def test_resets(env, K, dtype):
    """g = -inf empties the state, and lets no gradient through."""
    orc, la = env
    d = _make(1, 290, 1, 2, K, 64, dtype, 8)
    for t in (0, 40, 127, 128, 129, 289):
        d["g"][:, t] = -torch.inf
    o, s, saved = la.forward(*(d[n] for n in INS), d["s_init"])
    grads = la.backward(*(d[n] for n in INS), d["do"], saved, dS_final=d["dS_final"])
    h = _np(d)
    o_ref, s_ref = orc.forward(*(h[n] for n in INS), h["s_init"])
    _close("o", o, o_ref), _close("s_final", s, s_ref)
    ref = orc.backward(*(h[n] for n in INS), h["do"], h["s_init"], h["dS_final"])
    for n in GRADS:
        _close(n, grads[n], ref[n])
    assert torch.count_nonzero(grads["dS_init"]) == 0 and torch.count_nonzero(grads["dg"][:, [0, 40, 127, 128, 129, 289]]) == 0


@BOTH
@pytest.mark.parametrize("size", [0.02, 0.5])
def test_gates_of_both_signs(env, size, dtype):
    d = _make(1, 150, 1, 2, 64, 64, dtype, 9)
    d["g"] = size * torch.randn(d["g"].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(9))
    _check(env, d)


@BOTH
def test_a_reset_beside_growth(env, dtype):
    orc, la = env
    d = _make(1, 160, 1, 2, 64, 64, dtype, 10, rate=0.1)
    d["g"][:, 20], d["g"][:, 30], d["g"][:, 140] = -torch.inf, 0.5, 2.0
    o, s, saved = la.forward(*(d[n] for n in INS), d["s_init"])
    grads = la.backward(*(d[n] for n in INS), d["do"], saved, dS_final=d["dS_final"])
    h = _np(d)
    o_ref, s_ref = orc.forward(*(h[n] for n in INS), h["s_init"])
    _close("o", o, o_ref), _close("s_final", s, s_ref)
    ref = orc.backward(*(h[n] for n in INS), h["do"], h["s_init"], h["dS_final"])
    for n in GRADS:
        _close(n, grads[n], ref[n])


@BOTH
@pytest.mark.parametrize("size", [1e-18, 1e15])
def test_magnitudes(env, size, dtype):
    """Parts have fp32's exponents: small values beside large ones, and gradients of any size."""
    d = _make(1, 200, 1, 2, 64, 64, dtype, 11)
    d["v"] *= size
    d["s_init"] *= size
    d["do"] /= size
    d["dS_final"] /= size
    d["v"][:, ::7] *= 1e3
    d["q"][:, ::5] *= 1e-3
    _check(env, d)


@BOTH
def test_small_outputs_beside_large_ones(env, dtype):
    """A head dimension 1e12 below its neighbours is as exact as they are."""
    orc, la = env
    d = _make(1, 200, 1, 1, 64, 64, dtype, 12)
    d["v"][..., 1::2] *= 1e-12
    o, s, _ = la.forward(*(d[n] for n in INS))
    h = _np(d)
    o_ref, s_ref = orc.forward(*(h[n] for n in INS))
    _close("o", o[..., 1::2], o_ref[..., 1::2])
    _close("s_final", s[:, :, 1::2], s_ref[:, :, 1::2])


def _close_rounded(name, got, ref):
    """A bfloat16 output against its reference rounded to bfloat16. A result that is off by e is
    rounded to another neighbour with a probability of 2 |e| / ulp and then differs by one ulp, at most
    2^-7 |x|: the squares sum up to 2^-6 sum |e x|, at most 2^-6 |e| |x| in 2-norms. With
    operands of 16 bits, two of them in a product (1.4 * 2^-18 each way, 8e-6): 3.5e-4 of the norm."""
    want = torch.from_numpy(ref).to(BF16).double().numpy()
    off = np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)
    assert off <= 3.5e-4, f"{name}: {off:.2e} from the rounded reference"


@pytest.mark.parametrize("K,V", [(64, 64), (128, 128), (40, 24)])
def test_bfloat16_outputs_are_results_rounded_once(env, K, V):
    orc, la = env
    d = _make(2, 300, 2, 4, K, V, BF16, 30)
    o, s, saved = la.forward(*(d[n] for n in INS), d["s_init"])
    g = la.backward(*(d[n] for n in INS), d["do"], saved, dS_final=d["dS_final"])
    h = _np(d)
    o_ref, _ = orc.forward(*(h[n] for n in INS), h["s_init"])
    ref = orc.backward(*(h[n] for n in INS), h["do"], h["s_init"], h["dS_final"])
    _close_rounded("o", o, o_ref)
    for n in ("dq", "dk", "dv"):
        _close_rounded(n, g[n], ref[n])


@BOTH
def test_values_that_are_not_numbers_stay_in_their_sequence_and_head(env, dtype):
    """A NaN or an infinity makes its chunk and those after it non-finite in its head, and nothing else."""
    _, la = env
    d = _make(1, 400, 2, 2, 64, 64, dtype, 13, states=2)
    st = torch.tensor([0, 260, 400], dtype=torch.int32, device="cuda")
    want = la.forward(*(d[m] for m in INS), d["s_init"], seq_starts=st)
    gw = la.backward(*(d[m] for m in INS), d["do"], want[2], seq_starts=st)
    d["v"][0, 300, 1, 3], d["k"][0, 270, 1, 5], d["do"][0, 265, 1, 0] = torch.nan, torch.inf, -torch.inf
    got = la.forward(*(d[m] for m in INS), d["s_init"], seq_starts=st)
    gg = la.backward(*(d[m] for m in INS), d["do"], got[2], seq_starts=st)
    la.wkv7.status()
    assert torch.equal(got[0][:, :260], want[0][:, :260]) and torch.equal(got[0][:, :, 0], want[0][:, :, 0])
    assert torch.equal(got[1][0], want[1][0]) and torch.equal(got[1][1, 0], want[1][1, 0])
    for m in ("dq", "dk", "dv", "dg"):
        assert torch.equal(gg[m][:, :260], gw[m][:, :260]) and torch.equal(gg[m][:, :, 0], gw[m][:, :, 0])
    assert not torch.isfinite(got[0][0, 300, 1]).all() and torch.isnan(got[1][1, 1]).any()


def test_zero_vectors(env):
    d = _make(1, 200, 2, 2, 64, 64, BF16, 14)
    d["k"][:, 10:30] = 0
    d["q"][:, 20:40] = 0
    d["v"][:, 64:180] = 0
    _check(env, d)
    d["do"][:] = 0
    d["dS_final"][:] = 0
    _, _, g = _check(env, d)
    assert all(torch.count_nonzero(x) == 0 for x in g.values())


@BOTH
def test_one_token_from_nothing_has_no_decay_gradient(env, dtype):
    _, _, g = _check(env, _make(3, 1, 2, 2, 64, 64, dtype), carry=False)
    assert torch.count_nonzero(g["dg"]) == 0


# ------------------------------------------------------- long sequences, segments ---


@BOTH
@pytest.mark.parametrize("B,T,Hk,Hv,K,V,fixed", [(1, 1024, 1, 1, 64, 64, False), (1, 4097, 1, 2, 64, 64, False), (2, 3000, 1, 2, 16, 24, True),
                                                 (1, 2100, 1, 2, 128, 72, False)])
def test_few_long_sequences(env, B, T, Hk, Hv, K, V, fixed, dtype):
    """In segments, from states made before (fp32 with heads above 64: chunk by chunk)."""
    _, la = env
    d = _make(B, T, Hk, Hv, K, V, dtype, T, rate=0.02, fixed=fixed)
    o, s, _ = _check(env, d)
    _check(env, d, carry=False)
    o2, none, _ = la.forward(*(d[n] for n in INS), d["s_init"], want_s_final=False)
    assert none is None and torch.equal(o2, o)


@pytest.mark.parametrize("B,Hv,T,dtype", [(5, 40, 200, BF16), (4, 77, 150, F32), (2, 38, 700, BF16)])
def test_more_chains_than_sms(env, B, Hv, T, dtype):
    _check(env, _make(B, T, Hv, Hv, 16, 64, dtype, B), carry=False)


@BOTH
def test_a_sequence_cut_in_two(env, dtype):
    """States and their gradients carry a long sequence over calls."""
    _, la = env
    d = _make(1, 300, 1, 2, 64, 64, dtype, 22)
    whole = la.forward(*(d[m] for m in INS), d["s_init"])
    gw = la.backward(*(d[m] for m in INS), d["do"], whole[2], dS_final=d["dS_final"])
    a, b = ({m: d[m][:, s].contiguous() for m in INS + ("do",)} for s in (slice(0, 70), slice(70, 300)))
    fa = la.forward(*(a[m] for m in INS), d["s_init"])
    fb = la.forward(*(b[m] for m in INS), fa[1])
    gb = la.backward(*(b[m] for m in INS), b["do"], fb[2], dS_final=d["dS_final"])
    ga = la.backward(*(a[m] for m in INS), a["do"], fa[2], dS_final=gb["dS_init"])
    # two results of the same bars, each from the exact ones
    bar = lambda x: 5e-3 if x.dtype == BF16 else 4e-5
    for x, y in [(fb[1], whole[1]), (torch.cat((fa[0], fb[0]), 1), whole[0])] + [
            (torch.cat((ga[m], gb[m]), 1), gw[m]) for m in ("dq", "dk", "dv", "dg")] + [(ga["dS_init"], gw["dS_init"])]:
        assert (x.double() - y.double()).norm() <= bar(x) * y.double().norm()


# ------------------------------------------------------------------ packed sequences ---


def _raw(la, d, starts):
    """Forward and backward by the C functions, into buffers that hold NaN before."""
    lib = la.load()
    q, v = d["q"], d["v"]
    (B, T, Hk, K), (Hv, V), n, bf16 = q.shape, v.shape[2:], len(starts) - 1, int(q.dtype == BF16)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    fixed = int(d["g"].dim() == 1)

    def nan(*shape, dtype=F32):
        return torch.full(shape, float("nan"), dtype=dtype, device="cuda")

    def junk(size):
        return torch.full((size,), 255, dtype=torch.uint8, device="cuda")

    dims = (B, T, Hk, Hv, K, V, n)
    saved, work = junk(la.saved_bytes(*dims, bf16=bf16, for_backward=True)), junk(lib.linattn_backward_bytes(*dims, fixed, bf16))
    out = {"o": nan(B, T, Hv, V, dtype=q.dtype), "s_final": nan(n, Hv, V, K)}
    stream = torch.cuda.current_stream().cuda_stream
    p = lambda *xs: [x.data_ptr() for x in xs]
    ins = p(*(d[m] for m in INS))
    assert lib.linattn_forward(*ins, *p(d["s_init"], st, out["o"], out["s_final"], saved), None, 0.25, fixed, 1, *dims, bf16, stream) == 0
    g = {"dq": nan(*q.shape, dtype=q.dtype), "dk": nan(*q.shape, dtype=q.dtype), "dv": nan(*v.shape, dtype=q.dtype),
         "dg": nan(*d["g"].shape), "dS_init": nan(n, Hv, V, K)}
    assert lib.linattn_backward(*ins, *p(d["do"], d["dS_final"], st, saved, work, *g.values()), None, 0.25, fixed, *dims, bf16, stream) == 0
    la.wkv7.status()
    return {**out, **g}


@BOTH
@pytest.mark.parametrize("starts", [[0, 7], [0, 128, 128, 257, 258, 500], [0, 0, 0, 1, 63, 190, 190]], ids=["one", "mixed", "empty"])
@pytest.mark.parametrize("Hk,Hv,K,V", [(2, 4, 64, 64), (1, 1, 128, 72)])
def test_packed_sequences(env, starts, Hk, Hv, K, V, dtype):
    orc, la = env
    d = _make(1, starts[-1], Hk, Hv, K, V, dtype, 15, states=len(starts) - 1)
    out = _raw(la, d, starts)
    h = _np(d)
    fwd = orc.packed(orc.forward, starts, [h[m] for m in INS], {"s_init": h["s_init"]}, scale=0.25)
    _close("o", out["o"], np.concatenate([x[0] for x in fwd], 1)), _close("s_final", out["s_final"], np.concatenate([x[1] for x in fwd]))
    bwd = orc.packed(orc.backward, starts, [h[m] for m in INS + ("do",)], {"s_init": h["s_init"], "dS_final": h["dS_final"]}, scale=0.25)
    for m in ("dq", "dk", "dv", "dg"):
        _close(m, out[m], np.concatenate([x[m] for x in bwd], 1))
    _close("dS_init", out["dS_init"], np.concatenate([x["dS_init"] for x in bwd]))


@pytest.mark.parametrize("dtype,K,V,Hk,Hv", [(BF16, 64, 72, 2, 4), (BF16, 128, 64, 1, 5), (BF16, 16, 64, 3, 3), (F32, 64, 64, 2, 4)])
def test_many_short_packed_sequences(env, dtype, K, V, Hk, Hv):
    """More chains than the GPU has SMs, of lengths from none to a few chunks in any order, from and to states of their own."""
    orc, la = env
    lengths = [0, 1, 130, 0, 0, 64, 7, 257, 128, 2] * 6 + [0]
    starts = np.concatenate(([0], np.cumsum(lengths))).tolist()
    d = _make(1, starts[-1], Hk, Hv, K, V, dtype, 23, states=len(lengths))
    out = _raw(la, d, starts)
    h = _np(d)
    fwd = orc.packed(orc.forward, starts, [h[m] for m in INS], {"s_init": h["s_init"]}, scale=0.25)
    _close("o", out["o"], np.concatenate([x[0] for x in fwd], 1)), _close("s_final", out["s_final"], np.concatenate([x[1] for x in fwd]))
    bwd = orc.packed(orc.backward, starts, [h[m] for m in INS + ("do",)], {"s_init": h["s_init"], "dS_final": h["dS_final"]}, scale=0.25)
    for m in ("dq", "dk", "dv", "dg"):
        _close(m, out[m], np.concatenate([x[m] for x in bwd], 1))
    _close("dS_init", out["dS_init"], np.concatenate([x["dS_init"] for x in bwd]))


@pytest.mark.parametrize("dtype,K,Hv", [(BF16, 64, 4), (BF16, 128, 5), (F32, 64, 4)])
def test_many_short_sequences_do_not_meet(env, dtype, K, Hv):
    """Which block takes which sequence changes no bit, and what is not a number stays in its sequence and head."""
    _, la = env
    lengths = [3, 140, 0, 129, 60] * 13
    starts = np.concatenate(([0], np.cumsum(lengths))).tolist()
    d = _make(1, starts[-1], 1, Hv, K, 64, dtype, 24, states=len(lengths))
    want = _raw(la, d, starts)
    again = _raw(la, d, starts)
    assert all(torch.equal(want[m], again[m]) for m in want)
    bad = [(1, 0), (10, 2), (35, 1), (61, 3)]  # sequences (of any length above 0) and heads
    for s, h in bad:
        assert lengths[s] > 0
        d["v"][0, starts[s], h] = float("nan") if s % 2 else float("inf")
        d["do"][0, starts[s], h] = float("nan")
    got = _raw(la, d, starts)
    for m in ("o", "dv", "s_final", "dS_init", "dg"):
        keep = torch.ones(want[m].shape[:2] if m in ("s_final", "dS_init") else want[m].shape[1:3], dtype=torch.bool, device="cuda")
        for s, h in bad:
            keep[s if m in ("s_final", "dS_init") else slice(starts[s], starts[s + 1]), h] = False
        x, y = (t if m in ("s_final", "dS_init") else t[0] for t in (want[m], got[m]))
        assert torch.equal(x[keep], y[keep]), m


@pytest.mark.parametrize("dtype,Hk,Hv,K,T,starts,fixed", [
    (BF16, 1, 2, 64, 100, [0, 40, 70], False),
    (F32, 2, 2, 72, 333, [10, 40, 40, 70], False),
    (F32, 1, 2, 64, 400, [10, 40, 40, 370], True),
    (BF16, 2, 4, 128, 6000, [70, 5100], False),
    (F32, 2, 4, 64, 2200, [3, 3, 1130, 2199], False),
    (BF16, 1, 2, 64, 90, [50], False),  # no sequence at all
    (BF16, 1, 3, 64, 90, [50, 50], True),
])
def test_tokens_of_no_sequence(env, dtype, Hk, Hv, K, T, starts, fixed):
    """Before the first start and from the last on: o and the gradients are 0 there,
    whatever the buffers held, and the others' are those of the tokens alone."""
    _, la = env
    n, V = len(starts) - 1, 64
    d = _make(1, T, Hk, Hv, K, V, dtype, 39, states=n, fixed=fixed)
    a, b = starts[0], starts[-1]
    for m in ("q", "k", "v", "do"):  # what stands there may be anything
        d[m][:, :a], d[m][:, b:] = float("nan"), float("inf")
    out = _raw(la, d, starts)
    orc = env[0]
    h = _np(d)
    fwd = orc.packed(orc.forward, starts, [h[m] for m in INS], {"s_init": h["s_init"]}, scale=0.25)
    bwd = orc.packed(orc.backward, starts, [h[m] for m in INS + ("do",)], {"s_init": h["s_init"], "dS_final": h["dS_final"]}, scale=0.25)
    for m, x in out.items():
        if m in ("s_final", "dS_init") or (m == "dg" and fixed):
            continue
        assert torch.count_nonzero(x[:, :a]) == 0 and torch.count_nonzero(x[:, b:]) == 0, m
    if not n:
        assert all(torch.count_nonzero(x) == 0 for x in out.values())
        return
    _close("o", out["o"][:, a:b], np.concatenate([x[0] for x in fwd], 1))
    _close("s_final", out["s_final"], np.concatenate([x[1] for x in fwd]))
    for m in ("dq", "dk", "dv") + (() if fixed else ("dg",)):
        _close(m, out[m][:, a:b], np.concatenate([x[m] for x in bwd], 1))
    if fixed:
        _close("dg", out["dg"], np.sum([x["dg"] for x in bwd], 0))
    _close("dS_init", out["dS_init"], np.concatenate([x["dS_init"] for x in bwd]))


@BOTH
def test_packed_starts_outside_the_tokens_stay_in_bounds(env, dtype):
    _, la = env
    d = _make(1, 100, 1, 1, 64, 64, dtype, 16, states=3)
    st = torch.tensor([-5, 40, 1000, 90], dtype=torch.int32, device="cuda")  # clamped: 0, 40, 100, 90 (empty)
    o, s, _ = la.forward(*(d[m] for m in INS), d["s_init"], seq_starts=st)
    good = torch.tensor([0, 40, 100, 100], dtype=torch.int32, device="cuda")
    o2, s2, _ = la.forward(*(d[m] for m in INS), d["s_init"], seq_starts=good)
    la.wkv7.status()
    assert torch.equal(o, o2) and torch.equal(s, s2)


@BOTH
def test_empty_calls(env, dtype):
    _, la = env
    for fixed in (False, True):
        d = _make(2, 0, 1, 2, 64, 64, dtype, 17, fixed=fixed)
        o, s, saved = la.forward(*(d[m] for m in INS), d["s_init"])
        assert o.shape == (2, 0, 2, 64) and torch.equal(s, d["s_init"])
        g = la.backward(*(d[m] for m in INS), d["do"], saved, dS_final=d["dS_final"])
        assert torch.equal(g["dS_init"], d["dS_final"]) and torch.count_nonzero(g["dg"]) == 0
        assert torch.count_nonzero(la.forward(*(d[m] for m in INS))[1]) == 0
        d = _make(0, 5, 1, 2, 64, 64, dtype, 17, fixed=fixed)
        assert torch.count_nonzero(la.backward(*(d[m] for m in INS), d["do"], la.forward(*(d[m] for m in INS))[2])["dg"]) == 0


# ------------------------------------------------- strides, streams, graphs, bits ---


@BOTH
def test_slices_of_a_wider_tensor(env, dtype):
    """q, k, v of one projection's output, one batch row for all, and rows that overlap."""
    _, la = env
    d = _make(2, 130, 2, 4, 64, 32, dtype, 18)
    wide = torch.empty((2, 130, 2 * 128 + 128 + 8), dtype=dtype, device="cuda")
    parts = (wide[..., :128], wide[..., 128:256], wide[..., 264:392])
    views = [p.unflatten(-1, (h, -1)) for p, h in zip(parts, (2, 2, 4))]
    for view, n in zip(views, ("q", "k", "v")):
        view.copy_(d[n])
    dense = la.forward(*(d[m] for m in INS))
    apart = la.forward(*views, d["g"])
    assert torch.equal(dense[0], apart[0]) and torch.equal(dense[1], apart[1])
    a, b = (la.backward(*x, d["g"], d["do"], s[2]) for x, s in (((d["q"], d["k"], d["v"]), dense), (views, apart)))
    assert all(torch.equal(a[n], b[n]) for n in a)
    for one in (d["q"][:1].expand(2, -1, -1, -1), d["q"].as_strided((2, 60, 2, 64), (5 * 128, 128, 64, 1))):
        T = one.shape[1]
        x = [d[m][:, :T].contiguous() for m in ("k", "v", "g")]
        want = la.forward(one.contiguous(), *x)
        got = la.forward(one, *x)
        assert torch.equal(got[0], want[0])
        a, b = (la.backward(y, *x, d["do"][:, :T].contiguous(), z[2]) for y, z in ((one.contiguous(), want), (one, got)))
        assert all(torch.equal(a[n], b[n]) for n in a)


@BOTH
def test_offsets_past_32_bits(env, dtype):
    _, la = env
    d = _make(1, 66, 1, 1, 64, 64, dtype, 19)
    far = 1 << 25  # 65 of these: 2^31 + 2^25 elements
    buf = torch.empty(65 * far + 192, dtype=dtype, device="cuda")
    views = [buf.as_strided((1, 66, 1, 64), (0, far, 64, 1), 64 * i) for i in range(3)]
    for view, n in zip(views, ("q", "k", "v")):
        view.copy_(d[n])
    o, s, _ = la.forward(*views, d["g"])
    o2, s2, _ = la.forward(*(d[m] for m in INS))
    assert torch.equal(o, o2) and torch.equal(s, s2)


@pytest.mark.parametrize("T,Hk,Hv,K,V,dtype,fixed", [(333, 2, 6, 128, 64, BF16, False), (333, 2, 2, 64, 64, F32, True), (2000, 1, 2, 64, 64, BF16, True),
                                                   (333, 1, 3, 72, 64, F32, False)])
def test_the_same_bits_every_time(env, T, Hk, Hv, K, V, dtype, fixed):
    _, la = env
    d = _make(2, T, Hk, Hv, K, V, dtype, 20, fixed=fixed)

    def run():
        o, s, saved = la.forward(*(d[m] for m in INS), d["s_init"])
        return [o, s, *la.backward(*(d[m] for m in INS), d["do"], saved, dS_final=d["dS_final"]).values()]

    first = run()
    for _ in range(8):
        assert all(torch.equal(a, b) for a, b in zip(first, run()))


@pytest.mark.parametrize("T,dtype", [(100, BF16), (100, F32), (1500, BF16), (1500, F32)])
def test_another_stream_and_a_graph(env, T, dtype):
    _, la = env
    d = _make(1, T, 1, 2, 64, 64, dtype, 21)
    want = la.forward(*(d[m] for m in INS), d["s_init"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = la.forward(*(d[m] for m in INS), d["s_init"], stream=side)
    grads = la.backward(*(d[m] for m in INS), d["do"], got[2], stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with torch.cuda.stream(side):  # warm, then recorded
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            o, s, saved = la.forward(*(d[m] for m in INS), d["s_init"])
            g2 = la.backward(*(d[m] for m in INS), d["do"], saved)
    o.zero_(), g2["dg"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(g2["dg"], grads["dg"]) and torch.equal(g2["dq"], grads["dq"])


def test_calls_on_two_streams_at_once(env):
    _, la = env
    ds = [_make(2, 700, 4, 8, 64, 64, BF16, 50 + i) for i in range(2)]
    want = [la.forward(*(d[m] for m in INS), d["s_init"])[:2] for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    got = [[la.forward(*(d[m] for m in INS), d["s_init"], stream=s) for _ in range(10)] for d, s in zip(ds, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(x[0], w[0]) and torch.equal(x[1], w[1]) for xs, w in zip(got, want) for x in xs)


# ------------------------------------------------------------------------- step ---


@BOTH
@pytest.mark.parametrize("K,V,Hk,Hv,T,fixed", [(128, 128, 2, 4, 1, False), (64, 64, 1, 1, 3, True), (32, 40, 2, 6, 1, False), (8, 8, 1, 2, 2, False),
                                              (96, 72, 3, 3, 1, True), (16, 128, 1, 3, 5, False)])
def test_step(env, K, V, Hk, Hv, T, fixed, dtype):
    orc, la = env
    d = _make(6, T, Hk, Hv, K, V, dtype, K, states=9, fixed=fixed)
    slots = torch.tensor([4, 0, -1, 8, 2, 9], dtype=torch.int32, device="cuda")  # -1 and 9: no state
    pool = d["s_init"].clone()
    o = la.step(*(d[m] for m in INS), pool, slots=slots)
    h = _np(d)
    at, idx = [0, 1, 3, 4], [4, 0, 8, 2]
    o_ref, s_ref = orc.forward(*(h[m] if h[m].ndim == 1 else h[m][at] for m in INS), h["s_init"][idx])
    want = h["s_init"].copy()
    want[idx] = s_ref
    _close("o", o[at], o_ref), _close("s_final", pool, want)
    assert torch.count_nonzero(o[[2, 5]]) == 0
    keep = [i for i in range(9) if i not in idx]
    assert torch.equal(pool[keep], d["s_init"][keep])


def test_steps_continue_a_prefill(env):
    _, la = env
    d = _make(2, 40, 2, 4, 64, 64, F32, 23)
    o, s, _ = la.forward(*(d[m] for m in INS), d["s_init"], want_saved=False)
    _, state, _ = la.forward(*(d[m][:, :30].contiguous() for m in INS), d["s_init"], want_saved=False)
    outs = []
    for t in range(30, 40):
        outs.append(la.step(*(d[m][:, t:t + 1] if m in "qkv" else d[m][:, t:t + 1].contiguous() for m in INS), state))
    _close("o", torch.cat(outs, 1), o[:, 30:].double().cpu().numpy())
    _close("s_final", state, s.double().cpu().numpy())


def test_step_with_a_pool_past_32_bits(env):
    orc, la = env
    d = _make(2, 1, 1, 1, 128, 128, BF16, 24)
    n = (1 << 32) // (128 * 128) + 2  # elements past 2^32
    pool = torch.empty((n, 1, 128, 128), device="cuda")
    pool[n - 1], pool[1] = d["s_init"][0], d["s_init"][1]
    o = la.step(*(d[m] for m in INS), pool, slots=torch.tensor([n - 1, 1], dtype=torch.int32, device="cuda"))
    h = _np(d)
    o_ref, s_ref = orc.forward(*(h[m] for m in INS), h["s_init"])
    _close("o", o, o_ref)
    _close("s_final", pool[[n - 1, 1]], s_ref)


def test_step_resets_and_an_empty_step(env):
    orc, la = env
    d = _make(2, 1, 1, 1, 64, 64, F32, 25)
    d["g"][0] = -torch.inf
    pool = d["s_init"].clone()
    o = la.step(*(d[m] for m in INS), pool)
    h = _np(d)
    o_ref, s_ref = orc.forward(*(h[m] for m in INS), h["s_init"])
    _close("o", o, o_ref), _close("s_final", pool, s_ref)
    d = _make(0, 1, 1, 1, 64, 64, F32, 26)
    assert la.step(*(d[m] for m in INS), torch.zeros(3, 1, 64, 64, device="cuda")).shape == (0, 1, 1, 64)


def test_steps_in_a_graph(env):
    _, la = env
    d = _make(3, 1, 2, 4, 128, 128, BF16, 27)
    want = d["s_init"].clone()
    outs = [la.step(*(d[m] for m in INS), want) for _ in range(3)]
    pool = d["s_init"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = la.step(*(d[m] for m in INS), pool)
    pool.copy_(d["s_init"])
    for x in outs:
        graph.replay()
        assert torch.equal(o, x)
    assert torch.equal(pool, want)


# -------------------------------------------------------------------- refusals ---


def test_refusals(env):
    _, la = env
    d = _make(1, 8, 1, 2, 64, 64, BF16, 28)
    ins = [d[m] for m in INS]

    def bad(i, x, exc):
        with pytest.raises(exc):
            la.forward(*ins[:i], x, *ins[i + 1:])

    bad(0, d["q"].half(), TypeError)
    bad(1, d["k"][:, :4], ValueError)
    bad(1, d["k"].float(), TypeError)
    bad(2, d["v"].cpu(), ValueError)
    bad(3, d["g"].bfloat16(), TypeError)
    bad(3, d["g"].transpose(1, 2), ValueError)
    bad(3, d["g"][0, 0, :1], ValueError)
    bad(2, d["v"].transpose(2, 3), ValueError)
    with pytest.raises(la.wkv7.Wkv7Error):
        la.forward(d["q"][..., :60], d["k"][..., :60], *ins[2:])
    with pytest.raises(ValueError):
        la.forward(*ins, d["s_init"][:, :1])
    with pytest.raises(ValueError):
        la.backward(*ins, d["do"], None)
    with pytest.raises(ValueError):
        la.backward(*ins, d["do"], la.forward(*ins, want_saved=True)[2][:-1])
    with pytest.raises(TypeError):
        la.step(*ins, d["s_init"].bfloat16())
    with pytest.raises(TypeError):
        la.step(*ins, d["s_init"], slots=torch.zeros(1, device="cuda"))
    two = _make(2, 8, 1, 2, 64, 64, BF16, 28)
    with pytest.raises(la.wkv7.Wkv7Error):
        la.forward(*(two[m] for m in INS), seq_starts=torch.tensor([0, 8], dtype=torch.int32, device="cuda"))
