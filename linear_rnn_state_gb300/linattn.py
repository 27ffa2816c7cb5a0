"""Python binding of linear attention with a decay (include/linattn.h).

Argument checks and marshalling only: the recurrence runs in the CUDA kernels
of libwkv7.so. The raw functions carry the C names and take integer device
addresses; ``forward``, ``backward`` and ``step`` take torch tensors, allocate the
outputs and workspaces with torch on the stream they run on (torch's current
stream unless ``stream`` is given) and call the raw functions there. There is no
CPU path.

    S_t = e^{g_t} S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t

q, k [B][T][Hk][K]; v, o [B][T][Hv][V] (float32 or bfloat16); g [B][T][Hv], or [Hv]
for one fixed decay a head, and states [n][Hv][V][K] float32. q, k, v may be slices
of a wider tensor.
"""
from __future__ import annotations

import ctypes
import functools

from . import gdr, wkv7
from .gdr import _addr, _check_device, _check_tensor, _is_bf16, _on, _sequences, _strides

# C functions declared in include/linattn.h, with their argument counts.
EXPORTS = {
    "linattn_saved_bytes": 9,
    "linattn_backward_bytes": 9,
    "linattn_forward": 22,
    "linattn_backward": 26,
    "linattn_step": 19,
}

_lib = None


def load(path: str | None = None):
    """The loaded library with the linattn_* signatures set."""
    global _lib
    lib = wkv7.load(path)
    if path is None:
        _lib = lib
    if gdr._torch is None:
        gdr._setup()
    if not hasattr(lib, "_linattn_typed"):
        vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        lib.linattn_saved_bytes.argtypes = [i] * 9
        lib.linattn_backward_bytes.argtypes = [i] * 9
        for name in ("linattn_saved_bytes", "linattn_backward_bytes"):
            getattr(lib, name).restype = ctypes.c_size_t
        lib.linattn_forward.argtypes = [vp] * 10 + [f] + [i] * 10 + [vp]
        lib.linattn_backward.argtypes = [vp] * 15 + [f] + [i] * 9 + [vp]
        lib.linattn_step.argtypes = [vp] * 8 + [f] + [i] * 9 + [vp]
        for name in ("linattn_forward", "linattn_backward", "linattn_step"):
            getattr(lib, name).restype = i
        lib._linattn_typed = True
    return lib


def _inputs(q, k, v, g):
    """Checks the inputs against each other; returns bf16, (B, T, Hk, Hv, K, V), whether g is fixed, device."""
    dtype, dev, f32 = q.dtype, q.device, gdr._torch.float32
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v must be [B][T][heads][size]")
    B, T, Hk, K = shape = q.shape
    Hv, V = v.shape[2], v.shape[3]
    fixed = g.dim() == 1
    rows = (Hv,) if fixed else (B, T, Hv)
    if not (dev.type == "cuda" and dev.index == gdr._torch.cuda.current_device() and k.shape == shape
            and v.shape == (B, T, Hv, V) and g.shape == rows and k.dtype is dtype and v.dtype is dtype and g.dtype is f32
            and k.device == dev and v.device == dev and g.device == dev and g.is_contiguous()):  # say which
        _check_device(dev)
        _check_tensor("k", k, shape, dtype, dev, False)
        _check_tensor("v", v, (B, T, Hv, V), dtype, dev, False)
        _check_tensor("g", g, rows, f32, dev)
    return 1 if dtype is gdr._torch.bfloat16 else _is_bf16("q", q), (B, T, Hk, Hv, K, V), fixed, dev


@functools.lru_cache(maxsize=256)
def _saved_bytes(*args):
    return load().linattn_saved_bytes(*args)


@functools.lru_cache(maxsize=256)
def _backward_bytes(*args):
    return load().linattn_backward_bytes(*args)


def saved_bytes(B, T, Hk, Hv, K, V, nseq=-1, *, bf16, for_backward) -> int:
    """Bytes of what ``forward`` keeps for itself and, with for_backward, for ``backward``."""
    return _saved_bytes(B, T, Hk, Hv, K, V, nseq, int(bf16), int(for_backward))


def forward(q, k, v, g, s_init=None, *, scale: float | None = None, seq_starts=None, want_saved: bool = True,
            want_s_final: bool = True, stream=None):
    """The recurrence over whole sequences, in chunks. scale: K ** -0.5 unless
    given. seq_starts (int32, one more than the sequences; B = 1) gives packed
    sequences' starts; tokens before the first and from the last on have outputs
    and gradients of 0. Returns (o, s_final, saved); saved is what ``backward``
    needs (None without want_saved)."""
    if stream is not None:
        return _on(stream, forward, q, k, v, g, s_init, scale=scale, seq_starts=seq_starts, want_saved=want_saved,
                   want_s_final=want_s_final)
    lib = _lib or load()
    torch = gdr._torch
    bf16, dims, fixed, dev = _inputs(q, k, v, g)
    B, T, Hk, Hv, K, V = dims
    n, nseq = _sequences(seq_starts, B, dev)
    if s_init is not None:
        _check_tensor("s_init", s_init, (n, Hv, V, K), torch.float32, dev)
    o = torch.empty((B, T, Hv, V), dtype=q.dtype, device=dev)
    s_final = torch.empty((n, Hv, V, K), dtype=torch.float32, device=dev) if want_s_final else None
    need = _saved_bytes(B, T, Hk, Hv, K, V, nseq, bf16, int(want_saved))
    saved = torch.empty(need, dtype=torch.uint8, device=dev) if need or want_saved else None
    rc = lib.linattn_forward(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _addr(s_init), _addr(seq_starts), o.data_ptr(), _addr(s_final),
        _addr(saved), _strides(q, k, v), K ** -0.5 if scale is None else scale, fixed, want_saved, B, T, Hk, Hv, K, V, nseq,
        bf16, gdr._raw_stream(dev.index))
    if rc:
        wkv7._check(rc)
    return o, s_final, saved if want_saved else None


def backward(q, k, v, g, do, saved, *, dS_final=None, want_dS_init: bool = True, want_dg: bool = True,
             scale: float | None = None, seq_starts=None, stream=None):
    """Gradients of sum <do, o> + <dS_final, s_final>, with the ``saved`` of a
    ``forward`` of the same inputs and options. Returns dict dq, dk, dv (the
    inputs' type), dg (g's shape; None without want_dg) and dS_init (float32; None
    without want_dS_init)."""
    if stream is not None:
        return _on(stream, backward, q, k, v, g, do, saved, dS_final=dS_final, want_dS_init=want_dS_init, want_dg=want_dg,
                   scale=scale, seq_starts=seq_starts)
    lib = _lib or load()
    torch = gdr._torch
    bf16, dims, fixed, dev = _inputs(q, k, v, g)
    B, T, Hk, Hv, K, V = dims
    n, nseq = _sequences(seq_starts, B, dev)
    _check_tensor("do", do, (B, T, Hv, V), q.dtype, dev)
    if dS_final is not None:
        _check_tensor("dS_final", dS_final, (n, Hv, V, K), torch.float32, dev)
    if saved is None:
        raise ValueError("saved must be what forward(..., want_saved=True) returned")
    _check_tensor("saved", saved, (_saved_bytes(*dims, nseq, bf16, 1),), torch.uint8, dev)

    def empty(like, dtype=torch.float32):
        return torch.empty(like, dtype=dtype, device=dev)

    grads = {"dq": empty(q.shape, q.dtype), "dk": empty(q.shape, q.dtype), "dv": empty(v.shape, q.dtype),
             "dg": empty(g.shape) if want_dg else None, "dS_init": empty((n, Hv, V, K)) if want_dS_init else None}
    work = empty(_backward_bytes(*dims, nseq, int(fixed), bf16), torch.uint8)
    wkv7._check(lib.linattn_backward(*(_addr(x) for x in (q, k, v, g, do, dS_final, seq_starts, saved, work)),
                                     *(_addr(x) for x in grads.values()), _strides(q, k, v), K ** -0.5 if scale is None else scale,
                                     fixed, *dims, nseq, bf16, gdr._raw_stream(dev.index)))
    return grads


def step(q, k, v, g, state, *, slots=None, scale: float | None = None, stream=None):
    """The recurrence for the next token (or few) of each request: q, k
    [R][T][Hk][K], v [R][T][Hv][V], g [R][T][Hv] or [Hv]. ``state`` [n][Hv][V][K]
    float32 is updated in place; slots (int32 [R]) names each request's state,
    each at most once, a negative one to skip the request (its o is 0); None:
    request r has state r. Returns o."""
    if stream is not None:
        return _on(stream, step, q, k, v, g, state, slots=slots, scale=scale)
    lib = _lib or load()
    torch = gdr._torch
    bf16, (R, T, Hk, Hv, K, V), fixed, dev = _inputs(q, k, v, g)
    shape = state.shape
    n = shape[0] if len(shape) == 4 else 0
    if not (shape == (n, Hv, V, K) and state.dtype is torch.float32 and state.device == dev and state.is_contiguous()):
        _check_tensor("state", state, (n, Hv, V, K), torch.float32, dev)
    if slots is not None:
        _check_tensor("slots", slots, (R,), torch.int32, dev)
    o = torch.empty((R, T, Hv, V), dtype=q.dtype, device=dev)
    rc = lib.linattn_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), state.data_ptr(), _addr(slots), o.data_ptr(),
                          _strides(q, k, v), K ** -0.5 if scale is None else scale, fixed, R, T, Hk, Hv, K, V, n, bf16,
                          gdr._raw_stream(dev.index))
    if rc:
        wkv7._check(rc)
    return o
