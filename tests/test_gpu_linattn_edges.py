"""GPU tests of linear attention at its edges: decays, states and gradients that are not numbers, more packed sequences
than are ordered by length, one packed sequence in segments. Bars: as tests/test_gpu_linattn.py derives them.
"""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F32 = torch.bfloat16, torch.float32
INS = ("q", "k", "v", "g")
BOTH = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])


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


def _make(B, T, Hk, Hv, K, V, dtype, seed, states=None):
    gen = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, device="cuda", generator=gen)
    d = {"q": n(B, T, Hk, K).to(dtype), "k": n(B, T, Hk, K).to(dtype), "v": n(B, T, Hv, V).to(dtype), "do": n(B, T, Hv, V).to(dtype)}
    m = B if states is None else states
    return {**d, "g": -0.2 * n(B, T, Hv).abs(), "s_init": n(m, Hv, V, K), "dS_final": n(m, Hv, V, K)}


def _run(la, d, starts=None):
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    o, s, saved = la.forward(*(d[m] for m in INS), d["s_init"], seq_starts=st)
    out = {"o": o, "s_final": s, **la.backward(*(d[m] for m in INS), d["do"], saved, dS_final=d["dS_final"], seq_starts=st)}
    la.wkv7.status()
    return out


def _close(name, got, ref):
    got, bf16 = got.double().cpu().numpy(), got.dtype == BF16
    bar = 2.5e-3 if bf16 else 2e-5 if name == "dg" else 4e-6
    assert np.linalg.norm(got - ref) <= bar * np.linalg.norm(ref), name


# (K, V; tokens: long enough for segments where there are few heads)
SIZES = pytest.mark.parametrize("K,V,T", [(64, 64, 300), (128, 64, 300), (64, 64, 1500)])


@BOTH
@SIZES
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_decay_that_is_not_a_number(env, K, V, T, bad, dtype):
    """From its token on its head is not finite, no other head and batch row is touched, nor what its own did in the chunks before."""
    _, la = env
    d = _make(2, T, 3, 3, K, V, dtype, T + K)
    want = _run(la, d)
    t = T // 2 + 5
    d["g"][1, t, 1] = bad
    got = _run(la, d)
    first = t // 128 * 128
    for m in ("o", "dq", "dk", "dv", "dg"):
        assert torch.equal(got[m][0], want[m][0]) and torch.equal(got[m][1][:, [0, 2]], want[m][1][:, [0, 2]]), m
    assert torch.equal(got["o"][1, :first], want["o"][1, :first])
    assert not torch.isfinite(got["o"][1, t:, 1]).any() and not torch.isfinite(got["s_final"][1, 1]).any()
    assert torch.equal(got["s_final"][0], want["s_final"][0]) and torch.equal(got["s_final"][1, [0, 2]], want["s_final"][1, [0, 2]])
    # gradients: what passes the token on its way back
    assert not torch.isfinite(got["dv"][1, :t, 1]).any() and not torch.isfinite(got["dS_init"][1, 1]).any()
    last = min(T, first + 128)
    assert torch.equal(got["dv"][1, last:], want["dv"][1, last:])


@BOTH
@SIZES
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_state_that_is_not_a_number(env, K, V, T, bad, dtype):
    """An initial state's number, and one of the last state's gradient: their value's outputs, their head's gradients, nothing else."""
    _, la = env
    d = _make(2, T, 3, 3, K, V, dtype, T + K + 1)
    want = _run(la, d)
    d["s_init"][0, 2, 5, 3] = bad
    d["dS_final"][1, 0, 7, 2] = bad
    got = _run(la, d)
    keep = torch.ones(2, 3, dtype=torch.bool, device="cuda")
    keep[0, 2] = keep[1, 0] = False
    for m in ("dq", "dk", "dv", "dg"):
        x, y = (a[m].transpose(1, 2)[keep] for a in (got, want))
        assert torch.equal(x, y), m
    assert torch.equal(got["dS_init"][keep], want["dS_init"][keep])
    x, y = got["o"].clone(), want["o"].clone()
    assert not torch.isfinite(x[0, :, 2, 5]).any()
    x[0, :, 2, 5] = y[0, :, 2, 5] = 0
    assert torch.equal(x, y)
    x, y = got["s_final"].clone(), want["s_final"].clone()
    assert not torch.isfinite(x[0, 2, 5, 3])
    x[0, 2, 5] = y[0, 2, 5] = 0
    assert torch.equal(x, y)
    assert not torch.isfinite(got["dv"][1, :, 0, 7]).any() and not torch.isfinite(got["dS_init"][1, 0, 7, 2])


@BOTH
def test_steps_that_are_not_numbers(env, dtype):
    _, la = env
    d = _make(4, 2, 2, 2, 64, 64, dtype, 3)
    pool = d["s_init"].clone()
    want = la.step(*(d[m] for m in INS), pool)
    d["g"][1, 0, 0] = float("nan")
    d["v"][2, 1, 1, 9] = float("inf")
    again = d["s_init"].clone()
    again[3, 1, 4, 4] = float("nan")
    got = la.step(*(d[m] for m in INS), again)
    off = torch.zeros_like(want, dtype=torch.bool)
    off[1, :, 0], off[2, 1, 1, 9], off[3, :, 1, 4] = True, True, True
    assert torch.equal(got[~off], want[~off]) and not torch.isfinite(got[off]).any()
    off = torch.zeros_like(pool, dtype=torch.bool)
    off[1, 0], off[2, 1, 9], off[3, 1, 4] = True, True, True
    assert torch.equal(again[~off], pool[~off])


@BOTH
@pytest.mark.parametrize("count", [256, 257, 700])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 64)])
def test_hundreds_of_packed_sequences(env, K, V, count, dtype):
    """Up to 256 are taken by length, more as they come."""
    orc, la = env
    rng = np.random.default_rng(count)
    lengths = rng.choice([0, 1, 3, 17, 40, 129], count, p=[0.2, 0.3, 0.2, 0.2, 0.08, 0.02])
    starts = np.concatenate(([0], np.cumsum(lengths))).tolist()
    d = _make(1, starts[-1], 1, 2, K, V, dtype, count, states=count)
    out = _run(la, d, starts)
    h = {m: x.double().cpu().numpy() for m, x in d.items()}
    fwd = orc.packed(orc.forward, starts, [h[m] for m in INS], {"s_init": h["s_init"]})
    bwd = orc.packed(orc.backward, starts, [h[m] for m in INS + ("do",)], {"s_init": h["s_init"], "dS_final": h["dS_final"]})
    _close("o", out["o"], np.concatenate([x[0] for x in fwd], 1))
    _close("s_final", out["s_final"], np.concatenate([x[1] for x in fwd]))
    for m in ("dq", "dk", "dv", "dg"):
        _close(m, out[m], np.concatenate([x[m] for x in bwd], 1))
    _close("dS_init", out["dS_init"], np.concatenate([x["dS_init"] for x in bwd]))
    empty = torch.from_numpy(lengths == 0).cuda()
    assert torch.equal(out["s_final"][empty], d["s_init"][empty]) and torch.equal(out["dS_init"][empty], d["dS_final"][empty])


@pytest.mark.parametrize("dtype,K,heads", [(BF16, 64, 40), (BF16, 128, 16), (F32, 64, 40)])
def test_one_packed_sequence_of_many_heads_in_segments(env, dtype, K, heads):
    """In a padded batch; the segments begin at the sequence's first token, so the numbers are those of the tokens alone."""
    _, la = env
    T, a, b = 4200, 37, 4133
    assert la.saved_bytes(1, T, heads, heads, K, 64, 1, bf16=dtype is BF16, for_backward=False) > 0
    d = _make(1, T, heads, heads, K, 64, dtype, heads)
    for m in ("q", "k", "v", "do"):
        d[m][:, :a], d[m][:, b:] = float("nan"), float("inf")
    got = _run(la, d, [a, b])
    alone = {m: x[:, a:b].contiguous() if m in INS + ("do",) else x for m, x in d.items()}
    want = _run(la, alone, [0, b - a])
    bar = lambda x: 5e-3 if x.dtype == BF16 else 4e-5
    for m in want:
        x = got[m] if m in ("s_final", "dS_init") else got[m][:, a:b]
        assert (x.double() - want[m].double()).norm() <= bar(x) * want[m].double().norm(), m
        if m not in ("s_final", "dS_init"):
            assert torch.count_nonzero(got[m][:, :a]) == 0 and torch.count_nonzero(got[m][:, b:]) == 0
