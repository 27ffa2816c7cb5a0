"""GPU tests of the decays of linear attention's fp32 kernels, one pair of tokens at a time: with queries, keys and values
of a single 1 an output is the decay between two tokens, and nothing is summed.

Bar, 10 * 2^-23 of the element. A decay is a product of two exponentials (2 units in the last place each, and half a
one for the second float of the exponent) and of three factors more (1.5 in all); it enters the products in three parts (half a unit), which the
tensor cores add up cutting at a unit each (2). Across chunks the state is one such result and the row another.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
T, N = 256, 64


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_rnn_state_gb300 import _build, linattn

    _build.build()
    linattn.load()
    torch.cuda.set_device(0)
    return linattn


RATES = [0.1, 0.2, 0.5, 1.0, 1.8, 2.5, 6.0]  # a token; from 1.9 on 32 tokens span more than the factored form's 60


def _inputs(which, first):
    """`which` of q, k, v, do is a window of 64 tokens' own 1s; the others are the first dimension's."""
    x = {m: torch.zeros(1, T, len(RATES), N) for m in ("q", "k", "v", "do")}
    for m in x:
        if m == which:
            x[m][0, range(first, first + N), :, range(N)] = 1
        else:
            x[m][..., 0] = 1
    rng = np.random.default_rng(first)
    g = -np.array(RATES) * rng.uniform(0.5, 1.5, (T, len(RATES)))
    return {m: t.cuda() for m, t in x.items()}, torch.from_numpy(g[None]).float().cuda()


@pytest.mark.parametrize("first", [0, 32, 50, 96, 128, 192])
@pytest.mark.parametrize("which,output", [("v", "o"), ("do", "dv"), ("k", "dq"), ("q", "dk")])
def test_the_decay_of_every_pair(la, which, output, first):
    x, g = _inputs(which, first)
    o, _, saved = la.forward(x["q"], x["k"], x["v"], g, scale=1.0)
    got = {"o": o, **la.backward(x["q"], x["k"], x["v"], g, x["do"], saved, scale=1.0)}[output]
    la.wkv7.status()
    got = got[0].double().cpu().numpy().transpose(1, 0, 2)  # [head][token][of the window]
    G = np.cumsum(g[0].double().cpu().numpy(), 0).T
    d = G[:, :, None] - G[:, None, first:first + N]
    later = np.arange(T)[:, None] >= np.arange(first, first + N)
    if output in ("dv", "dk"):  # the window's tokens are the later ones
        d, later = -d, np.arange(T)[:, None] <= np.arange(first, first + N)
    want = np.where(later, np.exp(np.where(later, d, 0)), 0)
    assert np.all(got[:, ~later] == 0)
    near = want > 1e-6
    off = np.abs(got - want)[near] / want[near]
    print(f"{off.max():.2e}")
    assert off.max() <= 10 * 2.0 ** -23, off.max()
    assert np.abs(got - want)[~near].max() <= 1e-6 * 10 * 2.0 ** -23 * 8  # (an exponent of tens: some units more)
