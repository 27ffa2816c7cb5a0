"""GPU tests of linear attention's gradients where many value heads share a key head of more
than 64 keys: a block goes through them one after the other, and each head's state and its
gradient take the places of the last one's. A thread that waited for a copy whose barrier has
been armed again meanwhile would wait for a copy of another head, or until its patience ends
(which the status reports).

Bars: as tests/test_gpu_linattn.py derives them; the sums of dq and dk over a group are made in fp32 and
rounded once.
"""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.bfloat16
INS = ("q", "k", "v", "g")


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


def _inputs(B, T, Hk, Hv, K, V, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, device="cuda", generator=gen)
    d = {"q": n(B, T, Hk, K).to(BF16), "k": n(B, T, Hk, K).to(BF16), "v": n(B, T, Hv, V).to(BF16), "do": n(B, T, Hv, V).to(BF16)}
    return {**d, "g": -0.2 * n(B, T, Hv).abs(), "s_init": n(B, Hv, V, K), "dS_final": n(B, Hv, V, K)}


@pytest.mark.parametrize("B,T,Hk,Hv,K,V", [(1, 300, 1, 16, 128, 128), (2, 200, 2, 24, 96, 64), (1, 130, 3, 9, 72, 128)])
@pytest.mark.parametrize("want_dg", [True, False])
def test_many_value_heads_of_a_wide_key_head(env, B, T, Hk, Hv, K, V, want_dg):
    orc, la = env
    d = _inputs(B, T, Hk, Hv, K, V, Hv)
    saved = la.forward(*(d[m] for m in INS), d["s_init"])[2]
    got = la.backward(*(d[m] for m in INS), d["do"], saved, dS_final=d["dS_final"], want_dg=want_dg)
    la.wkv7.status()
    h = {m: x.double().cpu().numpy() for m, x in d.items()}
    ref = orc.backward(*(h[m] for m in INS), h["do"], h["s_init"], h["dS_final"])
    for m in ("dq", "dk", "dv", "dS_init") + (("dg",) if want_dg else ()):
        x, r = got[m].double().cpu().numpy(), ref[m]
        bar = 2.5e-3 if got[m].dtype == BF16 else 2e-5 if m == "dg" else 4e-6
        assert np.linalg.norm(x - r) <= bar * np.linalg.norm(r), m


def test_the_same_bits_on_a_full_gpu(env):
    """Blocks of many heads on every SM beside one another, and calls on two streams: no bit moves and no wait runs out."""
    _, la = env
    d = _inputs(2, 2500, 8, 32, 128, 128, 5)
    saved = la.forward(*(d[m] for m in INS), d["s_init"])[2]
    want = la.backward(*(d[m] for m in INS), d["do"], saved)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [la.backward(*(d[m] for m in INS), d["do"], saved, stream=streams[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    la.wkv7.status()
    assert all(torch.equal(g[m], want[m]) for g in got for m in want)
