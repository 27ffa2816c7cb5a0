"""Pins of the gated delta rule's and the block norms' fp64 oracles: central
differences of every input, closed forms, and the chunk form's algebra that the
kernels rest on, written out in numpy against the recurrence."""
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


gdr = _load("gdr_oracle")
norm = _load("blocknorm_oracle")


def _inputs(rng, B=2, T=5, Hk=1, Hv=2, K=4, V=3):
    r = rng.standard_normal
    return {"q": r((B, T, Hk, K)), "k": 0.5 * r((B, T, Hk, K)), "v": r((B, T, Hv, V)), "g": -np.abs(r((B, T, Hv))),
            "beta": rng.random((B, T, Hv)), "s_init": r((B, Hv, V, K))}


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


@pytest.mark.parametrize("l2norm", [False, True])
def test_gdr_gradients_match_differences(l2norm):
    rng = np.random.default_rng(0)
    x = _inputs(rng)
    do, dS = rng.standard_normal((2, 5, 2, 3)), rng.standard_normal((2, 2, 3, 4))

    def loss():
        o, s = gdr.forward(*(x[n] for n in ("q", "k", "v", "g", "beta", "s_init")), scale=0.7, l2norm=l2norm)
        return (o * do).sum() + (s * dS).sum()

    got = gdr.backward(x["q"], x["k"], x["v"], x["g"], x["beta"], do, x["s_init"], dS, scale=0.7, l2norm=l2norm)
    for name, arg in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"), ("dbeta", "beta"), ("dS_init", "s_init")):
        ref = _differences(loss, x[arg])
        # truncation h^2 and rounding 1e-16 / h of a loss of order 100
        np.testing.assert_allclose(got[name], ref, rtol=1e-6, atol=1e-7, err_msg=name)


def test_gdr_closed_forms():
    rng = np.random.default_rng(1)
    x = _inputs(rng, T=1)
    # one token from nothing: S = beta v k^T, o = scale beta v (k.q)
    o, s = gdr.forward(x["q"], x["k"], x["v"], x["g"], x["beta"], scale=1.0)
    k, q = np.repeat(x["k"], 2, 2), np.repeat(x["q"], 2, 2)
    np.testing.assert_allclose(s, (x["beta"][..., None, None] * x["v"][..., None] * k[:, :, :, None, :])[:, 0])
    np.testing.assert_allclose(o, x["beta"][..., None] * x["v"] * (k * q).sum(-1, keepdims=True))
    # beta = 1 and a key of length one: what is written is what is read
    x = _inputs(rng, T=4)
    x["k"] /= np.linalg.norm(x["k"], axis=-1, keepdims=True)
    o, _ = gdr.forward(x["k"], x["k"], x["v"], x["g"], np.ones_like(x["beta"]), x["s_init"], scale=1.0)
    np.testing.assert_allclose(o, x["v"], atol=1e-12)
    # g = -inf empties the state
    x["g"][:, 2] = -np.inf
    o, s = gdr.forward(*(x[n] for n in ("q", "k", "v", "g", "beta", "s_init")))
    o2, s2 = gdr.forward(*(x[n][:, 2:] for n in ("q", "k", "v", "g", "beta")))
    np.testing.assert_allclose(o[:, 2:], o2)
    np.testing.assert_allclose(s, s2)


def test_gdr_packed_is_each_sequence_alone():
    rng = np.random.default_rng(2)
    x = _inputs(rng, B=1, T=9)
    st = rng.standard_normal((3, 2, 3, 4))
    parts = gdr.packed(gdr.forward, [0, 4, 4, 9], [x[n] for n in ("q", "k", "v", "g", "beta")], {"s_init": st})
    assert parts[1][0].shape[1] == 0
    np.testing.assert_array_equal(parts[1][1], st[1:2])
    o, s = gdr.forward(*(x[n][:, 4:] for n in ("q", "k", "v", "g", "beta")), st[2:3])
    np.testing.assert_array_equal(parts[2][0], o)
    np.testing.assert_array_equal(parts[2][1], s)


def test_chunk_form_is_the_recurrence():
    """u = T (v - e^G k S0^T), T = (I + L)^-1, and the gradients' sums over pairs."""
    rng = np.random.default_rng(3)
    T, K, V = 7, 4, 3
    x = _inputs(rng, B=1, T=T, Hk=1, Hv=1, K=K, V=V)
    q, k, v, g, b = (x[n][0, :, 0] for n in ("q", "k", "v", "g", "beta"))
    S0 = x["s_init"][0, 0]
    scale = 0.5
    G = np.cumsum(g)
    r = np.tril(np.exp(G[:, None] - G))
    strict = np.tril(r, -1)
    Ti = np.linalg.inv(np.eye(T) + strict * (k @ k.T) * b)
    u = Ti @ (v - np.exp(G)[:, None] * (k @ S0.T))
    P = scale * r * (q @ k.T) * b
    o = scale * np.exp(G)[:, None] * (q @ S0.T) + P @ u
    S1 = np.exp(G[-1]) * S0 + (u * (b * np.exp(G[-1] - G))[:, None]).T @ k
    o_ref, S_ref = gdr.forward(*(x[n] for n in ("q", "k", "v", "g", "beta", "s_init")), scale=scale)
    np.testing.assert_allclose(o, o_ref[0, :, 0], atol=1e-12)
    np.testing.assert_allclose(S1, S_ref[0, 0], atol=1e-12)
    do, dS1 = rng.standard_normal((T, V)), rng.standard_normal((V, K))
    ref = gdr.backward(x["q"], x["k"], x["v"], x["g"], x["beta"], do[None, :, None], x["s_init"], dS1[None, None], scale=scale)
    tail = np.exp(G[-1] - G)
    lam = Ti.T @ (P.T @ do + (b * tail)[:, None] * (k @ dS1.T))
    dS0 = np.exp(G[-1]) * dS1 + scale * (do * np.exp(G)[:, None]).T @ q - (lam * np.exp(G)[:, None]).T @ k
    F, E, f = scale * strict * (do @ u.T), strict * (lam @ u.T), scale * (do * u).sum(-1)
    dq = scale * np.exp(G)[:, None] * (do @ S0) + (F * b) @ k
    read = -np.exp(G)[:, None] * (lam @ S0) - (E * b) @ k
    w = F.T @ q - E.T @ k + tail[:, None] * (u @ dS1)
    dG = (q * dq).sum(-1) + (k * read).sum(-1) - b * (k * w).sum(-1)
    dG[-1] += (S1 * dS1).sum()
    dq, w = dq + (f * b)[:, None] * k, w + f[:, None] * q
    for name, got in (("dv", lam), ("dq", dq), ("dk", read + b[:, None] * w), ("dbeta", (k * w).sum(-1)),
                      ("dg", np.cumsum(dG[::-1])[::-1]), ("dS_init", dS0)):
        want = ref[name][0, 0] if name == "dS_init" else ref[name][0, :, 0]
        np.testing.assert_allclose(got, want, atol=1e-11, err_msg=name)


@pytest.mark.parametrize("scaled", [False, True])
def test_add_norm_gradients_match_differences(scaled):
    rng = np.random.default_rng(4)
    x, res, w = rng.standard_normal((3, 5)), rng.standard_normal((3, 5)), rng.standard_normal(5)
    a = rng.standard_normal(5) if scaled else None
    dn, dh = rng.standard_normal((3, 5)), rng.standard_normal((3, 5))

    def loss():
        h, n = norm.add(x, res, w, a)
        return (n * dn).sum() + (h * dh).sum()

    got = norm.add_grad(x, res, w, dn, dh, a)
    for name, arg in [("dx", x), ("dresidual", res), ("dweight", w)] + ([("dscale", a)] if scaled else []):
        np.testing.assert_allclose(got[name], _differences(loss, arg), rtol=1e-6, atol=1e-8, err_msg=name)


def test_gated_norm_gradients_match_differences():
    rng = np.random.default_rng(5)
    o, z, w, dy = rng.standard_normal((2, 3, 4)), rng.standard_normal((2, 3, 4)), rng.standard_normal(4), rng.standard_normal((2, 3, 4))
    got = norm.gated_grad(o, z, w, dy)
    for name, arg in (("do", o), ("dz", z), ("dweight", w)):
        ref = _differences(lambda: (norm.gated(o, z, w) * dy).sum(), arg)
        np.testing.assert_allclose(got[name], ref, rtol=1e-6, atol=1e-8, err_msg=name)
