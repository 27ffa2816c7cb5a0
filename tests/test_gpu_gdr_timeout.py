"""The gradients' kernel of the gated delta rule when a bounded wait runs out
(WKV7_ERR_TIMEOUT), on the GPU without a fault or a hang.

The debug build (libwkv7_debug.so: 1 ms wait limit) has a hook by which the kernel
starts no copy for one of every block's tiles. The threads give that wait up after
1 ms, go through the rest of their work without waiting, whatever the data, wait (a
millisecond a barrier at most) for the copies that are in flight, and end. The test
checks that the call returns, that the status is reported once, and that the same
call without the hook then gives the same bits as the product library.
"""
import ctypes

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def env():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_rnn_state_gb300 import _build, gdr

    _build.build()
    torch.cuda.set_device(0)
    gdr.load()
    dbg = gdr.load(_build.DEBUG_LIB)
    for hook in (dbg.gdr_debug_skip_tile, dbg.gdr_debug_skip_t):
        hook.argtypes, hook.restype = [ctypes.c_int], ctypes.c_int
    yield gdr, dbg
    dbg.gdr_debug_skip_tile(0), dbg.gdr_debug_skip_t(0)


# a head's own gradients, the terms of shared heads, their sum in the block (tiles of two heads), segments
CASES = [(2, 130, 2, 2, 64, 64, F32), (1, 200, 1, 3, 64, 48, BF16), (1, 640, 16, 32, 128, 40, BF16), (1, 8200, 1, 1, 64, 32, F32)]


@pytest.mark.parametrize("tile", ["first", "last"])
@pytest.mark.parametrize("B,T,Hk,Hv,K,V,dtype", CASES, ids=["alone", "terms", "sum", "segments"])
def test_a_wait_that_runs_out_is_reported(env, B, T, Hk, Hv, K, V, dtype, tile):
    gdr, dbg = env
    gen = torch.Generator("cuda").manual_seed(T)
    n = lambda *s: torch.randn(s, device="cuda", generator=gen)
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dtype)
    q, k, v, do = unit(n(B, T, Hk, K)), unit(n(B, T, Hk, K)), n(B, T, Hv, V).to(dtype), n(B, T, Hv, V).to(dtype)
    g, beta = -0.1 * n(B, T, Hv).abs(), torch.sigmoid(n(B, T, Hv))
    _, _, saved = gdr.forward(q, k, v, g, beta)
    want = gdr.backward(q, k, v, g, beta, do, saved)
    gdr.wkv7.status()
    stream, bf16, dims = torch.cuda.current_stream().cuda_stream, dtype is BF16, (B, T, Hk, Hv, K, V, -1)
    work = torch.empty(dbg.gdr_backward_bytes(*dims, bf16), dtype=torch.uint8, device="cuda")
    got = {m: torch.empty_like(x) for m, x in want.items()}

    def run():
        fn = dbg.gdr_backward_bf16 if bf16 else dbg.gdr_backward
        p = lambda *xs: [x.data_ptr() for x in xs]
        return fn(*p(q, k, v, g, beta, do), None, None, *p(saved, work, *got.values()), None, K ** -0.5, 0, *dims, stream)

    assert dbg.wkv7_status(stream) == 0, dbg.wkv7_last_error().decode()
    heads = Hv // Hk if K == 128 else 1
    assert dbg.gdr_debug_skip_tile(1 if tile == "first" else heads * ((V + 15) // 16)) == 0
    try:
        assert run() == 0
        assert dbg.wkv7_status(stream) == -4  # WKV7_ERR_TIMEOUT
        assert "bounded wait" in dbg.wkv7_last_error().decode()
        assert dbg.wkv7_status(stream) == 0  # the word was cleared
    finally:
        dbg.gdr_debug_skip_tile(0)
    assert run() == 0 and dbg.wkv7_status(stream) == 0
    assert all(torch.equal(got[m], want[m]) for m in want)


def test_the_hook_is_the_debug_build_alone_s(env):
    gdr, dbg = env
    assert hasattr(dbg, "gdr_debug_skip_tile") and not hasattr(gdr.load(), "gdr_debug_skip_tile")


@pytest.mark.parametrize("step", [1, 3, 5])
@pytest.mark.parametrize("B,T,Hk,Hv,K,V,dtype", [(2, 300, 1, 2, 64, 64, F32), (1, 300, 1, 2, 128, 80, BF16)], ids=["64", "128"])
def test_a_chain_s_wait_that_runs_out_is_reported(env, B, T, Hk, Hv, K, V, dtype, step):
    """The chains' image of T in one of five steps: their warps go on without it."""
    gdr, dbg = env
    gen = torch.Generator("cuda").manual_seed(step)
    n = lambda *s: torch.randn(s, device="cuda", generator=gen)
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dtype)
    q, k, v, do = unit(n(B, T, Hk, K)), unit(n(B, T, Hk, K)), n(B, T, Hv, V).to(dtype), n(B, T, Hv, V).to(dtype)
    g, beta = -0.1 * n(B, T, Hv).abs(), torch.sigmoid(n(B, T, Hv))
    o, s, saved = gdr.forward(q, k, v, g, beta)
    want = {"o": o, "s": s, **gdr.backward(q, k, v, g, beta, do, saved)}
    gdr.wkv7.status()
    stream, bf16, dims = torch.cuda.current_stream().cuda_stream, dtype is BF16, (B, T, Hk, Hv, K, V, -1)
    work = torch.empty(dbg.gdr_backward_bytes(*dims, bf16), dtype=torch.uint8, device="cuda")
    kept, got = torch.empty_like(saved), {m: torch.empty_like(x) for m, x in want.items()}
    suffix = "_bf16" if bf16 else ""
    p = lambda *xs: [x.data_ptr() for x in xs]
    tail = (None, K ** -0.5, 0)

    def forward():
        return getattr(dbg, "gdr_forward" + suffix)(*p(q, k, v, g, beta), None, None, *p(got["o"], got["s"], kept), *tail, 1, *dims, stream)

    def backward():
        return getattr(dbg, "gdr_backward" + suffix)(*p(q, k, v, g, beta, do), None, None, *p(saved, work),
                                                     *p(*list(got.values())[2:]), *tail, *dims, stream)

    for call in (forward, backward):
        assert dbg.wkv7_status(stream) == 0, dbg.wkv7_last_error().decode()
        assert dbg.gdr_debug_skip_t(step) == 0
        try:
            assert call() == 0
            assert dbg.wkv7_status(stream) == -4  # WKV7_ERR_TIMEOUT
            assert dbg.wkv7_status(stream) == 0
        finally:
            dbg.gdr_debug_skip_t(0)
    assert forward() == 0 and backward() == 0 and dbg.wkv7_status(stream) == 0
    assert all(torch.equal(got[m], want[m]) for m in want)
