"""Pins of the fp64 oracles of linear attention with a decay and of the norms of
queries and keys with the rotation: central differences of every input, closed
forms, and the chunk form's algebra that the kernels rest on, written out in numpy
against the recurrence."""
import importlib.util
import os

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _load(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, "oracle", name + ".py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


lin, rope = _load("linattn_oracle"), _load("qkrope_oracle")


def _differences(f, x, h=1e-6):
    """Central differences of a scalar function of x, entry by entry."""
    out = np.zeros_like(x)
    flat, grad = x.reshape(-1), out.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + h
        up = f()
        flat[i] = keep - h
        down = f()
        flat[i] = keep
        grad[i] = (up - down) / (2 * h)
    return out


def _inputs(rng, B=2, T=5, Hk=1, Hv=2, K=4, V=3, fixed=False):
    r = rng.standard_normal
    return {"q": r((B, T, Hk, K)), "k": r((B, T, Hk, K)), "v": r((B, T, Hv, V)),
            "g": -np.abs(r((Hv,) if fixed else (B, T, Hv))), "s_init": r((B, Hv, V, K))}


@pytest.mark.parametrize("fixed", [False, True])
def test_gradients_match_differences(fixed):
    rng = np.random.default_rng(0)
    x = _inputs(rng, fixed=fixed)
    do, dS = rng.standard_normal((2, 5, 2, 3)), rng.standard_normal((2, 2, 3, 4))

    def loss():
        o, s = lin.forward(*(x[n] for n in ("q", "k", "v", "g", "s_init")), scale=0.7)
        return (o * do).sum() + (s * dS).sum()

    got = lin.backward(x["q"], x["k"], x["v"], x["g"], do, x["s_init"], dS, scale=0.7)
    for name, arg in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"), ("dS_init", "s_init")):
        # truncation h^2 and rounding 1e-16 / h of a loss of order 100
        np.testing.assert_allclose(got[name], _differences(loss, x[arg]), rtol=1e-6, atol=1e-7, err_msg=name)


def test_closed_forms():
    rng = np.random.default_rng(1)
    x = _inputs(rng, T=4)
    # no decay: the state is the sum of all, o_t reads the sum so far
    x["g"][:] = 0
    o, s = lin.forward(x["q"], x["k"], x["v"], x["g"], scale=1.0)
    k, q = np.repeat(x["k"], 2, 2), np.repeat(x["q"], 2, 2)
    np.testing.assert_allclose(s, np.einsum("bthv,bthk->bhvk", x["v"], k))
    causal = np.tril(np.ones((4, 4)))
    np.testing.assert_allclose(o, np.einsum("bthk,bshk,ts,bshv->bthv", q, k, causal, x["v"]))
    # -inf before the third token: nothing of the first two is left
    x["g"][:, 2] = -np.inf
    o, s = lin.forward(x["q"], x["k"], x["v"], x["g"], x["s_init"])
    cut = {n: x[n][:, 2:] for n in ("q", "k", "v", "g")}
    o2, s2 = lin.forward(*cut.values())
    np.testing.assert_allclose(o[:, 2:], o2), np.testing.assert_allclose(s, s2)


@pytest.mark.parametrize("T", [1, 7, 16])
def test_the_chunk_form(T):
    """o, dq, dk, dv, dg and the states of one chunk as the kernels form them."""
    rng = np.random.default_rng(T)
    x = _inputs(rng, B=1, T=T, Hk=1, Hv=1)
    do, D = rng.standard_normal((1, T, 1, 3)), rng.standard_normal((1, 1, 3, 4))
    want = lin.backward(x["q"], x["k"], x["v"], x["g"], do, x["s_init"], D, scale=0.6)
    o_ref, s_ref = lin.forward(x["q"], x["k"], x["v"], x["g"], x["s_init"], scale=0.6)
    q, k, v, g, d = (y[0, :, 0] for y in (x["q"], x["k"], x["v"], x["g"], do))
    S, D, sc = x["s_init"][0, 0], D[0, 0], 0.6
    G = np.cumsum(g)
    low = np.tril(np.ones((T, T)))
    ratio = low * np.exp(np.where(low > 0, G[:, None] - G, 0))
    head, tail = sc * np.exp(G)[:, None], np.exp(G[-1] - G)[:, None]
    A = sc * ratio * (d @ v.T)
    np.testing.assert_allclose(sc * ratio * (q @ k.T) @ v + head * (q @ S.T), o_ref[0, :, 0])
    np.testing.assert_allclose(np.exp(G[-1]) * S + (tail * v).T @ k, s_ref[0, 0])
    np.testing.assert_allclose(np.exp(G[-1]) * D + (head * d).T @ q, want["dS_init"][0, 0])
    in_q, in_k = head * (d @ S), tail * (v @ D)
    np.testing.assert_allclose(A @ k + in_q, want["dq"][0, :, 0])
    np.testing.assert_allclose(A.T @ q + in_k, want["dk"][0, :, 0])
    np.testing.assert_allclose((sc * ratio * (q @ k.T)).T @ d + tail * (k @ D.T), want["dv"][0, :, 0])
    X, a, b = A * (q @ k.T), (q * in_q).sum(-1), (k * in_k).sum(-1)
    dg = [sum(X[i, j] for i in range(t, T) for j in range(t)) + a[t:].sum() + b[:t].sum() + np.exp(G[-1]) * (S * D).sum() for t in range(T)]
    np.testing.assert_allclose(dg, want["dg"][0, :, 0])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("half", [0, 1, 3, 4])
def test_rotation_gradients_match_differences(half, interleaved):
    rng = np.random.default_rng(half)
    x, w, dy = rng.standard_normal((3, 2, 8)), rng.standard_normal(8), rng.standard_normal((3, 2, 8))
    freq, pos = rng.random(half), np.array([0, 5, 1000])

    def loss():
        return (rope.forward(x, w, freq, pos, interleaved=interleaved, eps=1e-2) * dy).sum()

    dx, dw = rope.backward(x, w, freq, pos, dy, interleaved=interleaved, eps=1e-2)
    np.testing.assert_allclose(dx, _differences(loss, x), rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(dw, _differences(loss, w), rtol=1e-6, atol=1e-7)


def test_rotation_keeps_products_of_equal_distance():
    rng = np.random.default_rng(3)
    q, k, w, freq = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8)), np.ones(8), rng.random(4)
    at = [(rope.forward(q, w, freq, np.array([7 + p])) * rope.forward(k, w, freq, np.array([p]))).sum() for p in (0, 11, 300)]
    np.testing.assert_allclose(at, at[0])


def test_angles_as_fractions_of_a_turn():
    """freq / (2 pi) in 64 bits by integers, as the kernel forms it (csrc/qkrope.cu), against exact arithmetic."""
    from fractions import Fraction
    import struct

    two_over_pi = 0xA2F9836E4E441529FC2757D1F534DDC0  # 2^128 2 / pi
    mask = (1 << 64) - 1

    def turns(f):
        bits = struct.unpack("<Q", struct.pack("<d", f))[0]
        ex, m = (bits >> 52) & 2047, bits & ((1 << 52) - 1)
        M = ((m | (1 << 52) if ex else m) << 11) & mask
        c, cl = two_over_pi >> 64, two_over_pi & mask
        wide = M * c + ((M * cl) >> 64)
        s = ex - 1088
        t = (wide << s) & mask if s >= 0 else (wide >> -s) & mask
        return -t & mask if bits >> 63 else t

    for f in (1.0, 0.1, 1e-4, 3.0, 1e4, -0.7, 2.0 ** -40, 0.0, 123456.789):
        exact = Fraction(f) * two_over_pi / (4 << 128)
        off = (Fraction(turns(f), 1 << 64) - exact) % 1
        assert min(off, 1 - off) <= max(1, abs(Fraction(f))) / (1 << 63), f
