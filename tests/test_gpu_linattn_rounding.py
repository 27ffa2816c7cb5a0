"""GPU tests that bfloat16 outputs of linear attention are fp32 results rounded once: P, the state and its
gradient enter the products with the bits of fp32.

Bar. A result x that is off by e is rounded to another neighbour than the exact one with a probability of
|e| / ulp, and then differs by one ulp, at most 2^-7 |x|: the squares of the differences sum up to 2^-7 |e| |x| in
2-norms. Operands of 24 bits (three parts) and sums in fp32 are off by 5e-7 of the result at most (two roundings of
2^-25 and 24 steps into an accumulator that cuts at 2^-23 of what it holds, half of that in the mean and of partial sums that
grow to the result: 3 * 2^-23): sqrt(2^-7 * 5e-7) = 6.3e-5. Operands of 16 bits are off by 2^-18 a value, 1.5e-6 in the
mean: 1e-4.
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


@pytest.mark.parametrize("B,T,Hk,Hv,K,V,rate", [
    (2, 700, 2, 2, 64, 64, 0.1),    # two blocks an SM in the gradients, two places for the scores in the chains
    (2, 700, 1, 3, 64, 64, 0.1),    # shared heads
    (1, 700, 2, 2, 48, 128, 0.02),  # wide values
    (2, 700, 2, 4, 128, 128, 0.1),  # wide keys
    (1, 700, 2, 2, 128, 40, 0.5),
    (1, 2300, 1, 2, 64, 64, 0.02),  # segments
    (3, 500, 4, 4, 16, 64, 0.1),
])
def test_outputs_are_the_rounded_exact_ones(env, B, T, Hk, Hv, K, V, rate):
    orc, la = env
    gen = torch.Generator("cuda").manual_seed(T + K + V + Hv)
    n = lambda *s: torch.randn(s, device="cuda", generator=gen)
    d = {"q": n(B, T, Hk, K).to(BF16), "k": n(B, T, Hk, K).to(BF16), "v": n(B, T, Hv, V).to(BF16), "do": n(B, T, Hv, V).to(BF16)}
    d.update(g=-rate * n(B, T, Hv).abs(), s_init=n(B, Hv, V, K), dS_final=n(B, Hv, V, K))
    o, _, saved = la.forward(*(d[m] for m in INS), d["s_init"])
    got = {"o": o, **la.backward(*(d[m] for m in INS), d["do"], saved, dS_final=d["dS_final"])}
    la.wkv7.status()
    h = {m: x.double().cpu().numpy() for m, x in d.items()}
    ref = orc.backward(*(h[m] for m in INS), h["do"], h["s_init"], h["dS_final"])
    ref["o"], _ = orc.forward(*(h[m] for m in INS), h["s_init"])
    off = {}
    for m in ("o", "dv", "dq", "dk"):
        want = torch.from_numpy(ref[m]).to(BF16).double().numpy()
        off[m] = np.linalg.norm(got[m].double().cpu().numpy() - want) / np.linalg.norm(want)
    print({m: f"{x:.2e}" for m, x in off.items()})
    assert all(x <= 6.3e-5 for x in off.values()), off
