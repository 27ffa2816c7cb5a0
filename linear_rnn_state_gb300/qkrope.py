"""Python binding of the norms of queries and keys with the position rotation
(include/qkrope.h).

Argument checks and marshalling only: the kernels are those of libwkv7.so. The
functions take torch tensors, allocate outputs and workspaces with torch on the
stream they run on (torch's current stream unless ``stream`` is given) and call
the C functions there. There is no CPU path.

    y = rot(x / rms(x) * weight, position), a head at a time, queries and keys in one pass;
    rot turns the pairs of the first 2 len(freq) values by position * freq
"""
from __future__ import annotations

import ctypes

from . import gdr, wkv7
from .blocknorm import _rows, _vector
from .gdr import _addr, _check_device, _check_tensor, _is_bf16, _on

# C functions declared in include/qkrope.h, with their argument counts.
EXPORTS = {
    "qkrope_forward": 20,
    "qkrope_backward": 25,
    "qkrope_part_bytes": 4,
}

_lib = None


def load(path: str | None = None):
    """The loaded library with the qkrope_* signatures set."""
    global _lib
    lib = wkv7.load(path)
    if path is None:
        _lib = lib
    if gdr._torch is None:
        gdr._setup()
    if not hasattr(lib, "_qkrope_typed"):
        vp, i, n, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
        lib.qkrope_forward.argtypes = [vp] * 8 + [n] * 4 + [i] * 5 + [f, i, vp]
        lib.qkrope_backward.argtypes = [vp] * 13 + [n] * 4 + [i] * 5 + [f, i, vp]
        lib.qkrope_part_bytes.argtypes = [n, i, i, i]
        lib.qkrope_part_bytes.restype = ctypes.c_size_t
        lib.qkrope_forward.restype = lib.qkrope_backward.restype = i
        lib._qkrope_typed = True
    return lib


def _tokens(name, t):
    """(tokens, elements from token to token)."""
    if t.dim() == 3:  # the usual form, checked at less cost
        tokens, _, D = t.shape
        a, b, c = t.stride()
        if c == 1 and b == D:
            return tokens, a
    return _rows(name, t, 2)


def _inputs(q, k, q_weight, k_weight, freq, positions):
    """The inputs checked: bf16, (q's, k's token stride, tokens, T, Hq, Hk, D, half), device."""
    torch = gdr._torch
    bf16 = _is_bf16("q", q)
    qs, ks, dev = q.shape, k.shape, q.device
    if len(qs) < 3 or len(ks) != len(qs):
        raise ValueError("q and k must be [...][T][heads][D]")
    _check_device(dev)
    D = qs[-1]
    if not (k.dtype is q.dtype and k.device == dev and ks[-1] == D and ks[:-2] == qs[:-2]):
        _check_tensor("k", k, (*qs[:-2], ks[-2], D), q.dtype, dev, False)
    _vector("q_weight", q_weight, D, dev)
    _vector("k_weight", k_weight, D, dev)
    half = freq.numel()
    if not (freq.dtype is torch.float64 and freq.dim() == 1 and freq.device == dev and freq.is_contiguous()):
        _check_tensor("freq", freq, (half,), torch.float64, dev)
    if positions is not None and not (positions.shape == qs[:-2] and positions.dtype is torch.int32 and positions.device == dev
                                      and positions.is_contiguous()):
        _check_tensor("positions", positions, qs[:-2], torch.int32, dev)
    (nq, qt), (nk, kt) = _tokens("q", q), _tokens("k", k)
    return bf16, (qt, kt, max(nq, nk), qs[-3], qs[-2], ks[-2], D, half), dev  # (without heads a tensor has no rows)


def forward(q, k, q_weight, k_weight, freq, positions=None, *, interleaved: bool = False, eps: float = 1e-6, stream=None):
    """q [...][T][Hq][D] and k [...][T][Hk][D] (float32 or bfloat16, slices of a wider
    tensor allowed) normed a head at a time and turned by their positions. q_weight,
    k_weight [D] float32; freq [half] float64, radians a position: the pairs are the
    values (j, half + j), or with interleaved (2 j, 2 j + 1), and what follows them is not
    turned. positions [...][T] int32 (None: 0, 1, .. along T). Returns (q, k), new tensors."""
    if stream is not None:
        return _on(stream, forward, q, k, q_weight, k_weight, freq, positions, interleaved=interleaved, eps=eps)
    lib = _lib or load()
    torch = gdr._torch
    bf16, sizes, dev = _inputs(q, k, q_weight, k_weight, freq, positions)
    q_out, k_out = torch.empty(q.shape, dtype=q.dtype, device=dev), torch.empty(k.shape, dtype=q.dtype, device=dev)
    rc = lib.qkrope_forward(q.data_ptr(), k.data_ptr(), q_weight.data_ptr(), k_weight.data_ptr(), freq.data_ptr(), _addr(positions),
                            q_out.data_ptr(), k_out.data_ptr(), *sizes, interleaved, eps, bf16, gdr._raw_stream(dev.index))
    if rc:
        wkv7._check(rc)
    return q_out, k_out


def backward(q, k, q_weight, k_weight, freq, dq_out, dk_out, positions=None, *, interleaved: bool = False, eps: float = 1e-6,
             stream=None):
    """Gradients of sum <dq_out, q'> + <dk_out, k'> of ``forward`` of the same
    inputs. Returns dict dq, dk (q's and k's type, dense), dwq, dwk (the weights')."""
    if stream is not None:
        return _on(stream, backward, q, k, q_weight, k_weight, freq, dq_out, dk_out, positions, interleaved=interleaved, eps=eps)
    lib = _lib or load()
    torch = gdr._torch
    bf16, sizes, dev = _inputs(q, k, q_weight, k_weight, freq, positions)
    _check_tensor("dq_out", dq_out, q.shape, q.dtype, dev)
    _check_tensor("dk_out", dk_out, k.shape, q.dtype, dev)
    _, _, tokens, _, Hq, Hk, D, _ = sizes
    dq, dk = torch.empty(q.shape, dtype=q.dtype, device=dev), torch.empty(k.shape, dtype=q.dtype, device=dev)
    dwq, dwk = (torch.empty(D, dtype=torch.float32, device=dev) for _ in range(2))
    part = torch.empty(lib.qkrope_part_bytes(tokens, Hq, Hk, D), dtype=torch.uint8, device=dev)
    wkv7._check(lib.qkrope_backward(*(_addr(t) for t in (q, k, q_weight, k_weight, freq, positions, dq_out, dk_out, dq, dk, dwq, dwk, part)),
                                    *sizes, interleaved, eps, bf16, gdr._raw_stream(dev.index)))
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
