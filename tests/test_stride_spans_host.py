"""Strides so large that the bytes a tensor spans pass 64 bits (no GPU needed): a sum cut to 64 bits would be small,
pass for a tensor that fits, and let the call go on to a device with it. Each call must be refused before that."""
import ctypes

import pytest

FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced by these calls
GB = 1 << 30
INVALID = -2


@pytest.fixture(scope="module")
def lib():
    from linear_rnn_state_gb300 import _build, blocknorm, gdr, linattn, qkrope

    _build.build()
    for m in (gdr, blocknorm, linattn, qkrope):
        m.load()
    return linattn.load()


def _at(n):
    return [FAKE + 64 * i * GB for i in range(n)]


# (batch rows, tokens, a batch row's and a token's stride): (B - 1) b + (T - 1) t is 2^64 or a little more, in values or bytes
WRAP = [((1 << 19) + 1, 1, 1 << 45, 0), ((1 << 18) + 1, 1, 1 << 45, 0), (1, (1 << 24) + 1, 0, 1 << 40), (1, (1 << 23) + 1, 0, 1 << 40)]


@pytest.mark.parametrize("which", range(3), ids=["q", "k", "v"])
@pytest.mark.parametrize("bf16", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,T,b,t", WRAP)
def test_strides_of_q_k_and_v(lib, B, T, b, t, bf16, which):
    st = [8 * T, 8] * 3
    st[2 * which:2 * which + 2] = b or 8 * T, t or 8
    st = (ctypes.c_longlong * 6)(*st)
    p = _at(16)
    dims = (B, T, 1, 1, 8, 8)
    assert lib.linattn_forward(*p[:4], None, None, p[4], None, p[5], st, 1.0, 0, 1, *dims, -1, bf16, None) == INVALID
    assert b"too large" in lib.wkv7_last_error()
    assert lib.linattn_backward(*p[:5], None, None, *p[5:11], None, st, 1.0, 0, *dims, -1, bf16, None) == INVALID
    assert lib.linattn_step(*p[:4], p[4], None, p[5], st, 1.0, 0, *dims, B, bf16, None) == INVALID
    assert b"too large" in lib.wkv7_last_error()
    kind = "_bf16" if bf16 else ""
    assert getattr(lib, "gdr_forward" + kind)(*p[:5], None, None, p[5], None, p[6], st, 1.0, 0, 1, *dims, -1, None) == INVALID
    assert b"too large" in lib.wkv7_last_error()
    assert getattr(lib, "gdr_step" + kind)(*p[:5], p[5], None, p[6], st, 1.0, 0, *dims, B, None) == INVALID
    assert b"too large" in lib.wkv7_last_error()


@pytest.mark.parametrize("bf16", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("tokens", [(1 << 25) + 1, (1 << 24) + 1, (1 << 23) + 1])
def test_strides_of_rows(lib, tokens, bf16):
    p = _at(13)
    for far in ((1 << 39, 16), (16, 1 << 39)):
        rope = (*far, tokens, tokens, 2, 2, 8, 4, 0, 1e-6, bf16, None)
        assert lib.qkrope_forward(*p[:5], None, *p[5:7], *rope) == INVALID
        assert b"too large" in lib.wkv7_last_error()
        assert lib.qkrope_backward(*p[:5], None, *p[5:12], *rope) == INVALID
        assert b"too large" in lib.wkv7_last_error()
        assert lib.blocknorm_gated_forward(*p[:5], *far, tokens, 2, 8, 1e-6, bf16, None) == INVALID
        assert b"too large" in lib.wkv7_last_error()


def test_a_stride_that_fits_is_no_fault(lib):
    """The same calls with nothing to do on a device: 0 heads."""
    st = (ctypes.c_longlong * 6)(*([1 << 20, 8] * 3))
    assert lib.linattn_forward(*[None] * 9, st, 1.0, 0, 1, 2, 4, 0, 0, 8, 8, -1, 1, None) == 0
