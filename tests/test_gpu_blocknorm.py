"""GPU tests of the norms around a block (include/blocknorm.h) against the fp64
oracle. Bars: fp32 arithmetic over rows of up to 8192 (a tree of sums: 2^-24 times
about 20) gives 2e-6 in the 2-norm; the sums over rows run over up to some 10^5
terms of both signs in partial sums of 100 or so: 4e-6. bfloat16 outputs are
rounded once: 2.5e-3, or one and a half times what rounding the reference itself
costs, and every element within 2^-8 of |ref| + rms.
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
    from linear_rnn_state_gb300 import _build, blocknorm

    _build.build()
    blocknorm.load()
    spec = importlib.util.spec_from_file_location("blocknorm_oracle", os.path.join(ROOT, "oracle", "blocknorm_oracle.py"))
    orc = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(orc)
    torch.cuda.set_device(0)
    return orc, blocknorm


def _close(name, got, ref):
    bf16 = got.dtype == BF16
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), name
    norm, off = np.linalg.norm(ref), np.linalg.norm(got - ref)
    rounding = np.linalg.norm(torch.from_numpy(ref).to(BF16).double().numpy() - ref) if bf16 else 0.0
    if norm == 0:
        assert off == 0, name
        return
    bar = 2.5e-3 if bf16 else 4e-6 if name in ("dweight", "dscale") else 2e-6
    assert off <= max(bar * norm, 1.5 * rounding), f"{name}: {off / norm:.2e}"
    if bf16:
        worst = np.max(np.abs(got - ref) / (np.abs(ref) + norm / np.sqrt(ref.size)))
        assert worst <= 2.0 ** -8, f"{name}: element {worst:.2e}"


def _t(a, dtype):
    return torch.from_numpy(a).to("cuda", dtype)


def _n(t):
    return None if t is None else t.double().cpu().numpy()


def _add(env, rows, D, dt, rt, *, scaled=True, up=True, plain=False, seed=0, size=1.0):
    orc, bn = env
    rng = np.random.default_rng(seed)
    r = rng.standard_normal
    x = None if plain else _t(size * r((rows, D)), dt)
    res, w = _t(size * (3 * r((rows, D)) + 0.5), rt), _t(1 + 0.2 * r(D), F32)
    a = _t(0.5 + r(D), F32) if scaled and not plain else None
    h, n, rstd = bn.add_forward(x, res, w, a)
    dn, dh = _t(r((rows, D)), rt if plain else dt), _t(r((rows, D)), rt) if up else None
    g = bn.add_backward(x, res, w, rstd, dn, dh, a)
    h_ref, n_ref = orc.add(_n(x), _n(res), _n(w), _n(a))
    _close("n", n, n_ref)
    if plain:
        assert h is res and g["dx"] is None
    else:
        _close("h", h, h_ref)
    ref = orc.add_grad(_n(x), _n(res), _n(w), _n(dn), _n(dh), _n(a))
    for name, want in ref.items():
        _close(name, g[name], want)
    return g


@pytest.mark.parametrize("dt,rt", [(BF16, BF16), (BF16, F32), (F32, F32)], ids=["bf16", "bf16_f32", "f32"])
@pytest.mark.parametrize("D", [1, 7, 8, 60, 64, 100, 128, 200, 256, 500, 512, 1000, 1024, 2048, 2056, 4096, 5000, 8192])
def test_add_widths(env, D, dt, rt):
    _add(env, 37, D, dt, rt, seed=D)


@pytest.mark.parametrize("rows", [1, 2, 31, 600, 5000])
@pytest.mark.parametrize("scaled,up,plain", [(True, True, False), (False, True, False), (False, False, False), (False, True, True)])
def test_add_forms(env, rows, scaled, up, plain):
    _add(env, rows, 320, BF16, F32, scaled=scaled, up=up, plain=plain, seed=rows)
    _add(env, rows, 48, BF16, BF16, scaled=scaled, up=up, plain=plain, seed=rows + 1)


def test_add_without_a_scale_of_one_type_shares_the_gradient(env):
    g = _add(env, 5, 64, F32, F32, scaled=False)
    assert g["dx"] is g["dresidual"]


@pytest.mark.parametrize("size", [1e-3, 1e15])
def test_add_magnitudes(env, size):
    # 1e-3: eps counts; 1e15: the squares stay inside fp32
    _add(env, 9, 256, F32, F32, seed=3, size=size)


def test_add_zero_rows_of_values(env):
    orc, bn = env
    x, w = torch.zeros(4, 96, device="cuda"), torch.ones(96, device="cuda")
    h, n, rstd = bn.add_forward(x, x.clone(), w)
    assert torch.count_nonzero(n) == 0
    np.testing.assert_allclose(_n(rstd), 1e3, rtol=1e-6)
    g = bn.add_backward(x, x.clone(), w, rstd, torch.ones_like(x))
    np.testing.assert_allclose(_n(g["dresidual"]), 1e3, rtol=1e-6)


def test_add_of_slices(env):
    orc, bn = env
    rng = np.random.default_rng(4)
    wide, res = _t(rng.standard_normal((6, 5, 256)), BF16), _t(rng.standard_normal((6, 5, 96)), F32)
    w = _t(rng.standard_normal(96), F32)
    x = wide[..., 64:160]
    h, n, rstd = bn.add_forward(x, res, w)
    h2, n2, _ = bn.add_forward(x.contiguous(), res, w)
    assert torch.equal(h, h2) and torch.equal(n, n2)
    with pytest.raises(ValueError):
        bn.add_forward(wide[:, :3, 64:160], res[:, :3], w)  # rows not equally far apart
    dn = torch.randn_like(n)
    a, b = bn.add_backward(x, res, w, rstd, dn), bn.add_backward(x.contiguous(), res, w, rstd, dn)
    assert all(torch.equal(a[m], b[m]) for m in a if a[m] is not None)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tokens,H,D", [(1, 1, 8), (1, 32, 128), (13, 3, 50), (300, 5, 64), (2000, 2, 16), (40, 1, 3000), (7, 2, 256), (3, 40, 96)])
def test_gated(env, tokens, H, D, dt):
    orc, bn = env
    rng = np.random.default_rng(D)
    r = rng.standard_normal
    o, z, dy = (_t(s * r((tokens, H, D)), dt) for s in (0.3, 2.0, 1.0))
    w = _t(1 + 0.2 * r(D), F32)
    y, rstd = bn.gated_forward(o, z, w)
    _close("y", y, orc.gated(_n(o), _n(z), _n(w)))
    g = bn.gated_backward(o, z, w, rstd, dy)
    for name, want in orc.gated_grad(_n(o), _n(z), _n(w), _n(dy)).items():
        _close(name, g[name], want)


PAIRS = pytest.mark.parametrize("dt,rt", [(BF16, BF16), (BF16, F32), (F32, F32)], ids=["bf16", "bf16_f32", "f32"])


@PAIRS
@pytest.mark.parametrize("rows,D", [(37, 513), (37, 1023), (37, 2047), (37, 2049), (37, 4095), (700, 4097), (700, 8191)])
def test_add_wide_odd_widths(env, rows, D, dt, rt):
    """Rows of single values: groups of 128 threads and more, several pieces a thread, more rows than blocks."""
    _add(env, rows, D, dt, rt, seed=D)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tokens,H,D", [(50, 3, 515), (20, 2, 1027), (700, 1, 2047), (9, 2, 4099), (700, 1, 8191)])
def test_gated_wide_odd_widths(env, tokens, H, D, dt):
    test_gated(env, tokens, H, D, dt)


@pytest.mark.parametrize("D", [96, 520, 2048, 5000])
def test_rows_at_odd_strides(env, D):
    """Widths of whole pieces of eight whose rows are not whole pieces apart: by single values."""
    orc, bn = env
    gen = torch.Generator("cuda").manual_seed(D)
    n = lambda *s: torch.randn(s, device="cuda", generator=gen)
    x, r, w, a, dn, dh = n(40, D + 5).bfloat16()[:, :D], n(40, D + 3)[:, :D], n(D), n(D), n(40, D).bfloat16(), n(40, D)
    h, y, rstd = bn.add_forward(x, r, w, a)
    h_ref, n_ref = orc.add(*(_n(t) for t in (x, r, w, a)))
    _close("h", h, h_ref), _close("n", y, n_ref)
    g = bn.add_backward(x, r, w, rstd, dn, dh, a)
    for name, want in orc.add_grad(_n(x), _n(r), _n(w), _n(dn), _n(dh), _n(a)).items():
        _close(name, g[name], want)
    o, z, dy = n(40, 2 * D + 1)[:, :2 * D].unflatten(-1, (2, D)), n(40, 2 * D + 7)[:, :2 * D].unflatten(-1, (2, D)), n(40, 2, D)
    y, rstd = bn.gated_forward(o, z, w)
    _close("y", y, orc.gated(_n(o), _n(z), _n(w)))
    g = bn.gated_backward(o, z, w, rstd, dy)
    for name, want in orc.gated_grad(_n(o), _n(z), _n(w), _n(dy)).items():
        _close(name, g[name], want)


def test_gated_fp32_gates_to_the_last_bits(env):
    """Every element of y, where the sigmoid runs from 1 down to fp32's smallest normal
    numbers: an exponential (2 ulp), a sum, a quotient, the row's sum (16 values: 4 and
    the root's 3) and five products, some sixteen roundings of 2^-24: 1e-6 of the element."""
    orc, bn = env
    z = torch.linspace(-87.0, 30.0, 16 * 400, device="cuda").view(400, 1, 16)
    o = 1 + torch.rand(400, 1, 16, device="cuda", generator=torch.Generator("cuda").manual_seed(7))
    w = torch.ones(16, device="cuda")
    y, _ = bn.gated_forward(o, z, w)
    ref = orc.gated(_n(o), _n(z), _n(w))
    assert np.max(np.abs(_n(y) - ref) / np.maximum(np.abs(ref), 1e-37)) <= 1e-6


def test_gated_gates_far_out(env):
    """z of -200 (its sigmoid is 0 in fp32) and 200."""
    orc, bn = env
    rng = np.random.default_rng(6)
    o, dy, w = _t(rng.standard_normal((4, 2, 64)), F32), _t(rng.standard_normal((4, 2, 64)), F32), torch.ones(64, device="cuda")
    z = torch.where(torch.rand(4, 2, 64, device="cuda") < 0.5, -200.0, 200.0)
    y, rstd = bn.gated_forward(o, z, w)
    _close("y", y, orc.gated(_n(o), _n(z), _n(w)))
    for name, want in orc.gated_grad(_n(o), _n(z), _n(w), _n(dy)).items():
        _close(name, bn.gated_backward(o, z, w, rstd, dy)[name], want)


def test_gated_of_slices(env):
    _, bn = env
    wide = torch.randn(9, 600, device="cuda", dtype=BF16)
    z, o, w = wide[:, 200:328].unflatten(-1, (2, 64)), torch.randn(9, 2, 64, device="cuda", dtype=BF16), torch.ones(64, device="cuda")
    y, rstd = bn.gated_forward(o, z, w)
    assert torch.equal(y, bn.gated_forward(o, z.contiguous(), w)[0])
    a, b = (bn.gated_backward(o, t, w, rstd, torch.ones_like(o)) for t in (z, z.contiguous()))
    assert all(torch.equal(a[m], b[m]) for m in a)


def test_the_same_bits_every_time_and_streams(env):
    _, bn = env
    x, res = torch.randn(3000, 512, device="cuda", dtype=BF16), torch.randn(3000, 512, device="cuda")
    w, a = torch.randn(512, device="cuda"), torch.randn(512, device="cuda")
    side = torch.cuda.Stream()
    first = None
    for stream in (None, side, None):
        if stream:
            side.wait_stream(torch.cuda.current_stream())
        h, n, rstd = bn.add_forward(x, res, w, a, stream=stream)
        g = bn.add_backward(x, res, w, rstd, x, res, a, stream=stream)
        torch.cuda.synchronize()
        got = [h, n, *g.values()]
        first = first or got
        assert all(torch.equal(p, q) for p, q in zip(first, got))


def test_no_rows(env):
    _, bn = env
    x, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    h, n, rstd = bn.add_forward(x, x, w, w)
    g = bn.add_backward(x, x, w, rstd, n, None, w)
    assert n.shape == (0, 64) and torch.count_nonzero(g["dweight"]) == 0 and torch.count_nonzero(g["dscale"]) == 0
    o = torch.empty(0, 2, 64, device="cuda")
    y, r = bn.gated_forward(o, o, w)
    assert torch.count_nonzero(bn.gated_backward(o, o, w, r, y)["dweight"]) == 0


def test_refusals(env):
    _, bn = env
    x, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(TypeError):
        bn.add_forward(x, x.bfloat16(), w)
    with pytest.raises(TypeError):
        bn.add_forward(x.half(), x, w)
    with pytest.raises(ValueError):
        bn.add_forward(x, x[:2], w)
    with pytest.raises(ValueError):
        bn.add_forward(x, x, w[:32])
    with pytest.raises(TypeError):
        bn.add_forward(x, x, w.bfloat16())
    with pytest.raises(ValueError):
        bn.add_forward(x.cpu(), x, w)
    with pytest.raises(ValueError):
        bn.gated_forward(x.view(4, 2, 32), x.view(4, 2, 32), w)
    with pytest.raises(bn.wkv7.Wkv7Error):
        bn.add_forward(torch.randn(2, 9000, device="cuda"), torch.randn(2, 9000, device="cuda"), torch.ones(9000, device="cuda"))
