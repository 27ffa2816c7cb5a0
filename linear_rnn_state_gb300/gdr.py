"""Python binding of the gated delta rule's C ABI (include/gdr.h).

Argument checks and marshalling only: the recurrence runs in the CUDA kernels
of libwkv7.so (the same library as the WKV7 scan). The raw functions carry the
C names and take integer device addresses; ``forward``, ``backward`` and
``step`` take torch tensors, allocate the outputs and workspaces with torch on
the stream they run on (torch's current stream unless ``stream`` is given) and
call the raw functions there. There is no CPU path.

    S_t = e^{g_t} S_{t-1} + beta_t (v_t - e^{g_t} S_{t-1} k_t) k_t^T,   o_t = scale S_t q_t

q, k [B][T][Hk][K]; v, o [B][T][Hv][V] (float32 or bfloat16); g, beta [B][T][Hv]
and states [n][Hv][V][K] float32. q, k, v may be slices of a wider tensor.
"""
from __future__ import annotations

import ctypes
import functools

from . import wkv7

CHUNK = 64  # tokens of a chunk

# C functions declared in include/gdr.h, with their argument counts.
EXPORTS = {
    "gdr_saved_bytes": 9,
    "gdr_backward_bytes": 8,
    "gdr_forward": 22,
    "gdr_forward_bf16": 22,
    "gdr_backward": 27,
    "gdr_backward_bf16": 27,
    "gdr_step": 18,
    "gdr_step_bf16": 18,
}

_lib = None


def load(path: str | None = None):
    """The loaded library with the gdr_* signatures set."""
    global _lib
    lib = wkv7.load(path)
    if path is None:
        _lib = lib
    if not hasattr(lib, "_gdr_typed"):
        vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        lib.gdr_saved_bytes.argtypes = [i] * 9
        lib.gdr_backward_bytes.argtypes = [i] * 8
        for name in ("gdr_saved_bytes", "gdr_backward_bytes"):
            getattr(lib, name).restype = ctypes.c_size_t
        for suffix in ("", "_bf16"):
            getattr(lib, "gdr_forward" + suffix).argtypes = [vp] * 11 + [f] + [i] * 9 + [vp]
            getattr(lib, "gdr_backward" + suffix).argtypes = [vp] * 17 + [f] + [i] * 8 + [vp]
            getattr(lib, "gdr_step" + suffix).argtypes = [vp] * 9 + [f] + [i] * 7 + [vp]
            for name in ("gdr_forward", "gdr_backward", "gdr_step"):
                getattr(lib, name + suffix).restype = i
        lib._gdr_typed = True
    return lib


# ------------------------------------------------------- torch helpers ---
#
# A decoding step takes a few microseconds on the GPU, so the host's part is kept
# small: every check is one comparison on the way through, and what can be looked
# up once is.

_torch = _raw_stream = None


def _setup():
    """torch and the lookup of its current stream's handle, once."""
    global _torch, _raw_stream
    import torch

    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _torch = torch
    return torch


def _addr(t):
    return None if t is None else t.data_ptr()


def _on(stream, fn, *args, **kw):
    """fn with `stream` torch's current one, so that what it allocates belongs to it."""
    with (_torch or _setup()).cuda.stream(stream):
        return fn(*args, **kw)


def _check_tensor(name, t, shape, dtype, device, dense=True):
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_device(device):
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, got {device}")
    if device.index != _torch.cuda.current_device():
        raise ValueError(f"tensors are on {device}, but the current device is cuda:{_torch.cuda.current_device()}")


def _is_bf16(name, t):
    if t.dtype is _torch.bfloat16:
        return 1
    if t.dtype is _torch.float32:
        return 0
    raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def _strides(q, k, v):
    """The strides of q, k, v for the C call, or None where all are dense."""
    if q.is_contiguous() and k.is_contiguous() and v.is_contiguous():
        return None
    for name, t in zip("qkv", (q, k, v)):
        D = t.shape[3]
        if (t.shape[3] > 1 and t.stride(3) != 1) or (t.shape[2] > 1 and t.stride(2) != D):
            raise ValueError(f"{name}: a token's heads must be dense (strides {t.stride()})")
    return (ctypes.c_longlong * 6)(*(x for t in (q, k, v) for x in (t.stride(0), t.stride(1))))


def _inputs(q, k, v, g, beta):
    """Checks the inputs against each other; returns bf16, (B, T, Hk, Hv, K, V), device."""
    if _torch is None:
        _setup()
    dtype, dev, f32 = q.dtype, q.device, _torch.float32
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v must be [B][T][heads][size]")
    B, T, Hk, K = shape = q.shape
    Hv, V = v.shape[2], v.shape[3]
    rows = (B, T, Hv)
    if not (dev.type == "cuda" and dev.index == _torch.cuda.current_device() and k.shape == shape and v.shape == (B, T, Hv, V)
            and g.shape == rows and beta.shape == rows and k.dtype is dtype and v.dtype is dtype and g.dtype is f32
            and beta.dtype is f32 and k.device == dev and v.device == dev and g.device == dev and beta.device == dev
            and g.is_contiguous() and beta.is_contiguous()):  # say which
        _check_device(dev)
        _check_tensor("k", k, shape, dtype, dev, False)
        _check_tensor("v", v, (B, T, Hv, V), dtype, dev, False)
        _check_tensor("g", g, rows, f32, dev)
        _check_tensor("beta", beta, rows, f32, dev)
    return 1 if dtype is _torch.bfloat16 else _is_bf16("q", q), (B, T, Hk, Hv, K, V), dev


def _sequences(seq_starts, B, dev):
    """(states, nseq of the C call)."""
    if seq_starts is None:
        return B, -1
    if seq_starts.dim() != 1 or seq_starts.numel() < 1:
        raise ValueError("seq_starts must hold the sequences' starts and the last one's end")
    n = seq_starts.numel() - 1
    _check_tensor("seq_starts", seq_starts, (n + 1,), _torch.int32, dev)
    return n, n


# The buffers' sizes depend on the arguments alone (a C call takes 1.1 us, the lookup 0.2).
@functools.lru_cache(maxsize=256)
def _saved_bytes(*args):
    return load().gdr_saved_bytes(*args)


@functools.lru_cache(maxsize=256)
def _backward_bytes(*args):
    return load().gdr_backward_bytes(*args)


def saved_bytes(B, T, Hk, Hv, K, V, nseq=-1, *, bf16, for_backward) -> int:
    """Bytes of what ``forward`` keeps for itself and, with for_backward, for ``backward``."""
    return _saved_bytes(B, T, Hk, Hv, K, V, nseq, int(bf16), int(for_backward))


def forward(q, k, v, g, beta, s_init=None, *, scale: float | None = None, qk_l2norm: bool = False, seq_starts=None,
            want_saved: bool = True, want_s_final: bool = True, stream=None):
    """The recurrence over whole sequences, in chunks. scale: K ** -0.5 unless
    given. qk_l2norm divides q and k by their lengths. seq_starts (int32,
    one more than the sequences; B = 1) gives packed sequences' starts; tokens
    before the first and from the last on have outputs and gradients of 0.
    Returns (o, s_final, saved); saved is what ``backward`` needs (None
    without want_saved)."""
    if stream is not None:
        return _on(stream, forward, q, k, v, g, beta, s_init, scale=scale, qk_l2norm=qk_l2norm, seq_starts=seq_starts,
                   want_saved=want_saved, want_s_final=want_s_final)
    lib = _lib or load()
    bf16, dims, dev = _inputs(q, k, v, g, beta)
    B, T, Hk, Hv, K, V = dims
    n, nseq = _sequences(seq_starts, B, dev)
    if s_init is not None:
        _check_tensor("s_init", s_init, (n, Hv, V, K), _torch.float32, dev)
    o = _torch.empty((B, T, Hv, V), dtype=q.dtype, device=dev)
    s_final = _torch.empty((n, Hv, V, K), dtype=_torch.float32, device=dev) if want_s_final else None
    saved = _torch.empty(_saved_bytes(B, T, Hk, Hv, K, V, nseq, bf16, want_saved), dtype=_torch.uint8, device=dev)
    rc = (lib.gdr_forward_bf16 if bf16 else lib.gdr_forward)(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), _addr(s_init), _addr(seq_starts), o.data_ptr(),
        _addr(s_final), saved.data_ptr(), _strides(q, k, v), K ** -0.5 if scale is None else scale, qk_l2norm, want_saved, B, T,
        Hk, Hv, K, V, nseq, _raw_stream(dev.index))
    if rc:
        wkv7._check(rc)
    return o, s_final, saved if want_saved else None


def backward(q, k, v, g, beta, do, saved, *, dS_final=None, want_dS_init: bool = True, scale: float | None = None,
             qk_l2norm: bool = False, seq_starts=None, stream=None):
    """Gradients of sum <do, o> + <dS_final, s_final>, with the ``saved`` of a
    ``forward`` of the same inputs and options. Returns dict dq, dk, dv (the
    inputs' type), dg, dbeta and dS_init (float32; None without
    want_dS_init)."""
    if stream is not None:
        return _on(stream, backward, q, k, v, g, beta, do, saved, dS_final=dS_final, want_dS_init=want_dS_init, scale=scale,
                   qk_l2norm=qk_l2norm, seq_starts=seq_starts)
    lib = _lib or load()
    bf16, dims, dev = _inputs(q, k, v, g, beta)
    B, T, Hk, Hv, K, V = dims
    n, nseq = _sequences(seq_starts, B, dev)
    _check_tensor("do", do, (B, T, Hv, V), q.dtype, dev)
    if dS_final is not None:
        _check_tensor("dS_final", dS_final, (n, Hv, V, K), _torch.float32, dev)
    need = _saved_bytes(*dims, nseq, bf16, 1)
    if saved is None:
        raise ValueError("saved must be what forward(..., want_saved=True) returned")
    _check_tensor("saved", saved, (need,), _torch.uint8, dev)
    def empty(like, dtype=_torch.float32):
        return _torch.empty(like, dtype=dtype, device=dev)

    grads = {"dq": empty(q.shape, q.dtype), "dk": empty(q.shape, q.dtype), "dv": empty(v.shape, q.dtype), "dg": empty(g.shape),
             "dbeta": empty(g.shape), "dS_init": empty((n, Hv, V, K)) if want_dS_init else None}
    work = empty(_backward_bytes(*dims, nseq, bf16), _torch.uint8)
    fn = lib.gdr_backward_bf16 if bf16 else lib.gdr_backward
    wkv7._check(fn(*(_addr(x) for x in (q, k, v, g, beta, do, dS_final, seq_starts, saved, work)),
                   *(_addr(x) for x in grads.values()), _strides(q, k, v), K ** -0.5 if scale is None else scale, qk_l2norm, *dims,
                   nseq, _raw_stream(dev.index)))
    return grads


def step(q, k, v, g, beta, state, *, slots=None, scale: float | None = None, qk_l2norm: bool = False, stream=None):
    """The recurrence for the next token (or few) of each request: q, k
    [R][T][Hk][K], v [R][T][Hv][V], g, beta [R][T][Hv]. ``state`` [n][Hv][V][K]
    float32 is updated in place; slots (int32 [R]) names each request's state,
    each at most once, a negative one to skip the request (its o is 0); None:
    request r has state r. Returns o."""
    if stream is not None:
        return _on(stream, step, q, k, v, g, beta, state, slots=slots, scale=scale, qk_l2norm=qk_l2norm)
    lib = _lib or load()
    bf16, (R, T, Hk, Hv, K, V), dev = _inputs(q, k, v, g, beta)
    shape = state.shape
    n = shape[0] if len(shape) == 4 else 0
    if not (shape == (n, Hv, V, K) and state.dtype is _torch.float32 and state.device == dev and state.is_contiguous()):
        _check_tensor("state", state, (n, Hv, V, K), _torch.float32, dev)
    if slots is not None:
        _check_tensor("slots", slots, (R,), _torch.int32, dev)
    o = _torch.empty((R, T, Hv, V), dtype=q.dtype, device=dev)
    rc = (lib.gdr_step_bf16 if bf16 else lib.gdr_step)(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), state.data_ptr(), _addr(slots), o.data_ptr(),
        _strides(q, k, v), K ** -0.5 if scale is None else scale, qk_l2norm, R, T, Hk, Hv, K, V, n, _raw_stream(dev.index))
    if rc:
        wkv7._check(rc)
    return o
