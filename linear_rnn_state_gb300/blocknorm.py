"""Python binding of the block norms' C ABI (include/blocknorm.h).

Argument checks and marshalling only: the norms run in the CUDA kernels of
libwkv7.so. The functions take torch tensors, allocate outputs and workspaces
with torch on the stream they run on (torch's current stream unless ``stream``
is given) and call the C functions there. There is no CPU path.

    add:    h = residual + scale x,  n = h / rms(h) * weight
    gated:  y = o / rms(o) * weight * z * sigmoid(z)
"""
from __future__ import annotations

import ctypes

from . import gdr, wkv7
from .gdr import _addr, _check_device, _check_tensor, _is_bf16, _on

# C functions declared in include/blocknorm.h, with their argument counts.
EXPORTS = {
    "blocknorm_add_forward": 15,
    "blocknorm_add_backward": 19,
    "blocknorm_gated_forward": 13,
    "blocknorm_gated_backward": 16,
    "blocknorm_part_bytes": 3,
}

_lib = None


def load(path: str | None = None):
    """The loaded library with the blocknorm_* signatures set."""
    global _lib
    lib = wkv7.load(path)
    if path is None:
        _lib = lib
    if gdr._torch is None:
        gdr._setup()
    if not hasattr(lib, "_blocknorm_typed"):
        vp, i, n, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
        lib.blocknorm_add_forward.argtypes = [vp] * 7 + [n] * 3 + [i, f, i, i, vp]
        lib.blocknorm_add_backward.argtypes = [vp] * 12 + [n] * 3 + [i, i, i, vp]
        lib.blocknorm_gated_forward.argtypes = [vp] * 5 + [n] * 3 + [i, i, f, i, vp]
        lib.blocknorm_gated_backward.argtypes = [vp] * 9 + [n] * 3 + [i, i, i, vp]
        lib.blocknorm_part_bytes.argtypes = [n, i, i]
        lib.blocknorm_part_bytes.restype = ctypes.c_size_t
        for name in ("add_forward", "add_backward", "gated_forward", "gated_backward"):
            getattr(lib, "blocknorm_" + name).restype = i
        lib._blocknorm_typed = True
    return lib


def _rows(name, t, inner):
    """(rows, elements from row to row) of a tensor whose last `inner`
    dimensions are a row: dense inside, all rows equally far apart."""
    if t.is_contiguous():
        shape = t.shape
        stride = shape[-1] if inner == 1 else shape[-1] * shape[-2]
        return t.numel() // stride if stride else 0, stride
    dense = 1
    for d in range(t.dim() - 1, t.dim() - 1 - inner, -1):
        if t.shape[d] > 1 and t.stride(d) != dense:
            raise ValueError(f"{name}: a row must be dense (strides {t.stride()})")
        dense *= t.shape[d]
    rows, stride = 1, dense
    for d in range(t.dim() - 1 - inner, -1, -1):
        if t.shape[d] > 1 and rows > 1 and t.stride(d) != rows * stride:
            raise ValueError(f"{name}: rows must be equally far apart (strides {t.stride()})")
        if t.shape[d] > 1 and rows == 1:
            stride = t.stride(d)
        rows *= t.shape[d]
    return rows, stride


def _types(x, residual):
    r = _is_bf16("residual", residual)
    if x is None:
        return r, r
    a = _is_bf16("x", x)
    if r and not a:
        raise TypeError("a float32 x needs a float32 residual")
    return a, r


def _vector(name, t, D, dev):
    if not (t.shape == (D,) and t.dtype is gdr._torch.float32 and t.device == dev and t.is_contiguous()):
        _check_tensor(name, t, (D,), gdr._torch.float32, dev)


def _add_inputs(x, residual, weight, scale):
    """The add norm's inputs checked: bf16 of x and of residual, D, rows, row strides, device."""
    bf16, rbf16 = _types(x, residual)
    shape, dev = residual.shape, residual.device
    D = shape[-1]
    _check_device(dev)
    rows, rs = _rows("residual", residual, 1)
    xs = D
    if x is not None:
        if x.shape != shape or x.device != dev:
            _check_tensor("x", x, shape, x.dtype, dev, False)
        xs = _rows("x", x, 1)[1]
    _vector("weight", weight, D, dev)
    if scale is not None:
        _vector("scale", scale, D, dev)
    return bf16, rbf16, D, rows, xs, rs, dev


def add_forward(x, residual, weight, scale=None, *, eps: float = 1e-6, stream=None):
    """The norm before a block. x (None: the norm of residual alone) and
    residual [...][D]; weight and scale (None: 1) [D] float32. Returns
    (h, n, rstd): h of residual's type (residual itself without x), n of x's
    type (residual's without x), rstd [...] float32 for the backward."""
    if stream is not None:
        return _on(stream, add_forward, x, residual, weight, scale, eps=eps)
    lib = _lib or load()
    torch = gdr._torch
    bf16, rbf16, D, rows, xs, rs, dev = _add_inputs(x, residual, weight, scale)
    shape = residual.shape
    n = torch.empty(shape, dtype=residual.dtype if x is None else x.dtype, device=dev)
    h = None if x is None else torch.empty(shape, dtype=residual.dtype, device=dev)
    rstd = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
    rc = lib.blocknorm_add_forward(_addr(x), residual.data_ptr(), weight.data_ptr(), _addr(scale), _addr(h), n.data_ptr(),
                                   rstd.data_ptr(), xs, rs, rows, D, eps, bf16, rbf16, gdr._raw_stream(dev.index))
    if rc:
        wkv7._check(rc)
    return (residual if x is None else h), n, rstd


def add_backward(x, residual, weight, rstd, dn, dh=None, scale=None, *, stream=None):
    """Gradients of sum <dn, n> + <dh, h> (dh None: 0). Returns dict dresidual,
    dx (None without x), dweight and dscale (None without scale)."""
    if stream is not None:
        return _on(stream, add_backward, x, residual, weight, rstd, dn, dh, scale)
    lib = _lib or load()
    torch = gdr._torch
    bf16, rbf16, D, rows, xs, rs, dev = _add_inputs(x, residual, weight, scale)
    shape, xt = residual.shape, residual.dtype if x is None else x.dtype
    _check_tensor("rstd", rstd, shape[:-1], torch.float32, dev)
    _check_tensor("dn", dn, shape, xt, dev)
    if dh is not None:
        _check_tensor("dh", dh, shape, residual.dtype, dev)
    dres = torch.empty(shape, dtype=residual.dtype, device=dev)
    # without a scale x's gradient is the residual's; it is written apart only in another type
    own_dx = x is not None and (scale is not None or xt is not residual.dtype)
    dx = torch.empty(shape, dtype=xt, device=dev) if own_dx else None
    dw = torch.empty(D, dtype=torch.float32, device=dev)
    ds = torch.empty(D, dtype=torch.float32, device=dev) if scale is not None else None
    part = torch.empty(lib.blocknorm_part_bytes(rows, D, 2), dtype=torch.uint8, device=dev)
    wkv7._check(lib.blocknorm_add_backward(*(_addr(t) for t in (x, residual, weight, scale, rstd, dn, dh, dres, dx, dw, ds, part)),
                                           xs, rs, rows, D, bf16, rbf16, gdr._raw_stream(dev.index)))
    return {"dresidual": dres, "dx": None if x is None else dx if own_dx else dres, "dweight": dw, "dscale": ds}


def _gated(o, z, weight):
    bf16 = _is_bf16("o", o)
    shape, dev = o.shape, o.device
    if len(shape) < 2:
        raise ValueError("o must be [...][H][D]")
    _check_device(dev)
    H, D = shape[-2], shape[-1]
    if not (z.shape == shape and z.dtype is o.dtype and z.device == dev):
        _check_tensor("z", z, shape, o.dtype, dev, False)
    _vector("weight", weight, D, dev)
    tokens, os_ = _rows("o", o, 2)
    return bf16, tokens, H, D, os_, _rows("z", z, 2)[1], dev


def gated_forward(o, z, weight, *, eps: float = 1e-6, stream=None):
    """The gated norm after a block, a head at a time: o, z [...][H][D], weight
    [D] float32. Returns (y, rstd), rstd [...][H] float32 for the backward."""
    if stream is not None:
        return _on(stream, gated_forward, o, z, weight, eps=eps)
    lib = _lib or load()
    torch = gdr._torch
    bf16, tokens, H, D, os_, zs, dev = _gated(o, z, weight)
    y = torch.empty(o.shape, dtype=o.dtype, device=dev)
    rstd = torch.empty(o.shape[:-1], dtype=torch.float32, device=dev)
    rc = lib.blocknorm_gated_forward(o.data_ptr(), z.data_ptr(), weight.data_ptr(), y.data_ptr(), rstd.data_ptr(), os_, zs, tokens, H,
                                     D, eps, bf16, gdr._raw_stream(dev.index))
    if rc:
        wkv7._check(rc)
    return y, rstd


def gated_backward(o, z, weight, rstd, dy, *, stream=None):
    """Gradients of sum <dy, y>. Returns dict do, dz, dweight."""
    if stream is not None:
        return _on(stream, gated_backward, o, z, weight, rstd, dy)
    lib = _lib or load()
    torch = gdr._torch
    bf16, tokens, H, D, os_, zs, dev = _gated(o, z, weight)
    _check_tensor("rstd", rstd, o.shape[:-1], torch.float32, dev)
    _check_tensor("dy", dy, o.shape, o.dtype, dev)
    do, dz = (torch.empty(o.shape, dtype=o.dtype, device=dev) for _ in range(2))
    dw = torch.empty(D, dtype=torch.float32, device=dev)
    part = torch.empty(lib.blocknorm_part_bytes(tokens * H, D, 1), dtype=torch.uint8, device=dev)
    wkv7._check(lib.blocknorm_gated_backward(*(_addr(t) for t in (o, z, weight, rstd, dy, do, dz, dw, part)), os_, zs, tokens, H, D,
                                             bf16, gdr._raw_stream(dev.index)))
    return {"do": do, "dz": dz, "dweight": dw}
