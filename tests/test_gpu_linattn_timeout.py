"""Linear attention's chains and gradients when a bounded wait runs out (WKV7_ERR_TIMEOUT), on the GPU without a fault
or a hang.

The debug build (libwkv7_debug.so: 1 ms wait limit) has hooks by which a block leaves out a copy, the arrival of a
product or a question for another block (include/linattn_debug.h). The threads give that wait up after 1 ms, start no
further copy, go through the rest of their work without waiting, whatever the data, wait (some milliseconds at most)
for what is in flight, and end. The tests check that the call returns, that the status is reported once, and that the
same call without the hook then gives the same bits as the product library.
"""
import ctypes

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BF16, F32 = torch.bfloat16, torch.float32
TILES, SCORES, STATE, BACK, CLAIM = range(1, 6)
INS = ("q", "k", "v", "g")


@pytest.fixture(scope="module")
def env():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_rnn_state_gb300 import _build, linattn

    _build.build()
    torch.cuda.set_device(0)
    linattn.load()
    dbg = linattn.load(_build.DEBUG_LIB)
    dbg.linattn_debug_skip.argtypes, dbg.linattn_debug_skip.restype = [ctypes.c_int, ctypes.c_int], ctypes.c_int
    yield linattn, dbg
    dbg.linattn_debug_skip(0, 0)


def _setup(la, dbg, B, T, Hk, Hv, K, V, dtype, starts):
    gen = torch.Generator("cuda").manual_seed(T)
    n = lambda *s: torch.randn(s, device="cuda", generator=gen)
    d = {"q": n(B, T, Hk, K).to(dtype), "k": n(B, T, Hk, K).to(dtype), "v": n(B, T, Hv, V).to(dtype), "g": -0.1 * n(B, T, Hv).abs(),
         "do": n(B, T, Hv, V).to(dtype)}
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    o, s, saved = la.forward(*(d[m] for m in INS), seq_starts=st)
    want = {"o": o, "s": s, **la.backward(*(d[m] for m in INS), d["do"], saved, seq_starts=st)}
    la.wkv7.status()
    bf16, dims = int(dtype is BF16), (B, T, Hk, Hv, K, V, -1 if st is None else len(starts) - 1)
    work = torch.empty(dbg.linattn_backward_bytes(*dims, 0, bf16), dtype=torch.uint8, device="cuda")
    got, kept = {m: torch.empty_like(x) for m, x in want.items()}, torch.empty_like(saved)
    stream = torch.cuda.current_stream().cuda_stream
    p = lambda *xs: [None if x is None else x.data_ptr() for x in xs]

    def forward():
        return dbg.linattn_forward(*p(*(d[m] for m in INS), None, st, got["o"], got["s"], kept), None, K ** -0.5, 0, 1, *dims, bf16, stream)

    def backward():
        return dbg.linattn_backward(*p(*(d[m] for m in INS), d["do"], None, st, saved, work, *list(got.values())[2:]), None, K ** -0.5, 0,
                                    *dims, bf16, stream)

    keep = (d, st, saved, work, kept)
    return forward, backward, want, got, stream, keep


def _run_out(dbg, call, what, n, stream):
    assert dbg.wkv7_status(stream) == 0, dbg.wkv7_last_error().decode()
    assert dbg.linattn_debug_skip(what, n) == 0
    try:
        assert call() == 0
        assert dbg.wkv7_status(stream) == -4  # WKV7_ERR_TIMEOUT
        assert "bounded wait" in dbg.wkv7_last_error().decode()
        assert dbg.wkv7_status(stream) == 0  # the word was cleared
    finally:
        dbg.linattn_debug_skip(0, 0)


# two places for the scores; halves; segments; more sequences than SMs, some of them empty; fp32
CHAINS = {
    "64": (2, 700, 1, 2, 64, 64, BF16, None),
    "128": (1, 700, 1, 2, 128, 72, BF16, None),
    "segments": (1, 4097, 1, 1, 64, 64, BF16, None),
    "packed": (1, 12000, 2, 4, 128, 64, BF16, [0, 0] + [130 * i for i in range(1, 91)] + [12000]),
    "f32": (2, 700, 1, 2, 64, 64, F32, None),
    "f32-segments": (1, 4097, 1, 1, 32, 64, F32, None),
}


NAMES = {TILES: "tiles", SCORES: "scores", STATE: "state", BACK: "back"}


def _cases(of, whats):
    """Those that exist: fp32 tiles are loaded by the threads that use them."""
    return [pytest.param(case, what, n, id=f"{case}-{NAMES[what]}-{n}") for case in of for what, n in whats(of[case])
            if not (what == TILES and of[case][6] is F32)]


@pytest.mark.parametrize("case,what,n", _cases(CHAINS, lambda args: [(w, n) for w in (TILES, SCORES) for n in (1, 2, 3)]))
def test_a_chain_s_wait_that_runs_out_is_reported(env, case, what, n):
    la, dbg = env
    args = CHAINS[case]
    forward, backward, want, got, stream, _keep = _setup(la, dbg, *args)
    _run_out(dbg, forward, what, n, stream)
    _run_out(dbg, backward, what, n, stream)
    assert forward() == 0 and backward() == 0 and dbg.wkv7_status(stream) == 0
    assert all(torch.equal(got[m], want[m]) for m in want)


@pytest.mark.parametrize("n", [1, 2])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128)])
def test_a_block_that_is_not_answered(env, K, V, n):
    """A chain's question for a block that has not begun: its own sequences are done all the same, and the blocks begin."""
    la, dbg = env
    forward, backward, want, got, stream, _keep = _setup(la, dbg, 5, 150, 40, 40, K, V, BF16, None)
    _run_out(dbg, forward, CLAIM, n, stream)
    _run_out(dbg, backward, CLAIM, n, stream)
    assert forward() == 0 and backward() == 0 and dbg.wkv7_status(stream) == 0
    assert all(torch.equal(got[m], want[m]) for m in want)


# two blocks an SM; shared heads of 64 and of 128 keys; wide keys or values alone; fp32, alone and shared
GRADS = {
    "64": (2, 300, 2, 2, 64, 64, BF16, None),
    "64-shared": (1, 300, 1, 3, 64, 64, BF16, None),
    "64-128": (1, 300, 2, 2, 64, 128, BF16, None),
    "128": (1, 300, 2, 2, 128, 128, BF16, None),
    "128-shared": (1, 300, 1, 4, 128, 128, BF16, None),
    "packed": (1, 300, 1, 3, 96, 40, BF16, [0, 5, 5, 140, 290]),
    "f32": (2, 300, 2, 2, 64, 64, F32, None),
    "f32-shared": (1, 300, 1, 3, 64, 64, F32, None),
}


def _of_heads(args):
    """The first, another and the last of a block's value heads, or of their scores."""
    heads = args[3] // args[2]
    return sorted({(w, n) for w in (TILES, STATE, BACK) for n in (1, 2, heads) if n <= heads} | {(SCORES, n) for n in (1, 2, 2 * heads)})


@pytest.mark.parametrize("case,what,n", _cases(GRADS, _of_heads))
def test_the_gradients_wait_that_runs_out_is_reported(env, case, what, n):
    la, dbg = env
    args = GRADS[case]
    forward, backward, want, got, stream, _keep = _setup(la, dbg, *args)
    _run_out(dbg, backward, what, n, stream)
    assert forward() == 0 and backward() == 0 and dbg.wkv7_status(stream) == 0
    assert all(torch.equal(got[m], want[m]) for m in want)


def test_the_hook_is_the_debug_build_alone_s(env):
    la, dbg = env
    assert hasattr(dbg, "linattn_debug_skip") and not hasattr(la.load(), "linattn_debug_skip")
