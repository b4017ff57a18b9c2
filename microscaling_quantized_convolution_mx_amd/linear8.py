"""Linear layers in 8 bits: binding of include/mxlinear8.h.

The functions have the names of the C entry points and marshal arguments
only; see the header for the format, and linear.py for the matrices, the
descriptor (linear_desc, with block 1 or 128 here) and the experts' offsets.

A layer that trains, X and dY in 1x128 blocks along each contraction and W in
128x128 blocks:

    d, d1 = (linear_desc(tokens, out_features, in_features, block=b) for b in (128, 1))
    xq, dyq = Linear8QTensor(d1, MX_ROLE_ACT), Linear8QTensor(d1, MX_ROLE_GRAD)
    wq = Linear8QTensor(d, MX_ROLE_WEIGHT)
    ws = torch.empty(max(mx_linear8_workspace_bytes(d), 16), dtype=torch.uint8, device="cuda")
    mx_linear8_quantize(d1, MX_ROLE_ACT, x, xq)
    mx_linear8_quantize(d, MX_ROLE_WEIGHT, w, wq)
    mx_linear8_fwd(d, wq, xq, y, ws)
    mx_linear8_quantize(d1, MX_ROLE_GRAD, dy, dyq)
    mx_linear8_dgrad(d, wq, dyq, dx, ws)
    mx_linear8_wgrad(d, dyq, xq, dw, ws)

and one that serves: quantize W once, then mx_linear8_apply(d, wq, x, y, ws).
"""
from __future__ import annotations

import ctypes

import microscaling_quantized_convolution_mx_amd as _mx

from . import linear as _l
from .linear import MX_FORM_COLS, MX_FORM_ROWS, mx_linear_desc, mx_linear_qtensor

LINEAR8_EXPORTS = ("mx_linear8_code_bytes", "mx_linear8_scale_bytes", "mx_linear8_quantize", "mx_linear8_dequantize",
                   "mx_linear8_workspace_bytes", "mx_linear8_fwd", "mx_linear8_dgrad", "mx_linear8_wgrad",
                   "mx_linear8_apply")

_lib = None


def _load():
    """The library with the argument types of these entry points."""
    global _lib
    if _lib is None:
        _l._load()
        L = _mx.lib()
        D, Q, P = ctypes.POINTER(mx_linear_desc), ctypes.POINTER(mx_linear_qtensor), ctypes.c_void_p
        I, I64, Z = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        product = [D, Q, Q, P, I, I64, P, P, Z, P]
        for name, res, args in (
                ("mx_linear8_code_bytes", Z, [D, I, I]), ("mx_linear8_scale_bytes", Z, [D, I, I]),
                ("mx_linear8_workspace_bytes", Z, [D]), ("mx_linear8_quantize", I, [D, I, P, I, I64, P, Q, P]),
                ("mx_linear8_dequantize", I, [D, I, I, Q, P, I, I64, P, P]),
                ("mx_linear8_fwd", I, product), ("mx_linear8_dgrad", I, product), ("mx_linear8_wgrad", I, product),
                ("mx_linear8_apply", I, [D, Q, P, I, I64, P, I, I64, P, P, Z, P])):
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def mx_linear8_code_bytes(d: mx_linear_desc, role: int, form: int = MX_FORM_ROWS) -> int:
    return _load().mx_linear8_code_bytes(d, role, form)


def mx_linear8_scale_bytes(d: mx_linear_desc, role: int, form: int = MX_FORM_ROWS) -> int:
    return _load().mx_linear8_scale_bytes(d, role, form)


def mx_linear8_workspace_bytes(d: mx_linear_desc) -> int:
    return _load().mx_linear8_workspace_bytes(d)


class Linear8QTensor(_l._QTensor):
    """A matrix in 8 bits.  Buffers made for one block size serve the other."""

    @staticmethod
    def _key(d):
        return bytes(d)[:mx_linear_desc.block.offset]

    @staticmethod
    def _has_cols(d):
        return True

    @staticmethod
    def _form_bytes(d, role, form):
        L = _load()
        return L.mx_linear8_code_bytes(d, role, form), L.mx_linear8_scale_bytes(d, role, form)


def _q(q, d, role, forms, what):
    return _l._q(q, d, role, forms, what, Linear8QTensor)


def mx_linear8_quantize(d: mx_linear_desc, role: int, src, dst, offsets=None, stream=None) -> None:
    """Fills the forms that dst has."""
    L = _load()
    p, dt, ld, at = _l._matrix(src, _l._dims(d, role), "src")
    q, qat = _q(dst, d, role, dst.bytes if isinstance(dst, Linear8QTensor) else (), "dst")
    off, oat = _l._offsets(d, offsets)
    _l._check(L.mx_linear8_quantize(d, role, p, dt, ld, off, q, _mx._stream(stream, at, qat, oat)), "mx_linear8_quantize")


def mx_linear8_dequantize(d: mx_linear_desc, role: int, q, dst, form: int = MX_FORM_ROWS, offsets=None, stream=None) -> None:
    L = _load()
    p, dt, ld, at = _l._matrix(dst, _l._dims(d, role), "dst")
    c, qat = _q(q, d, role, (form,), "q")
    off, oat = _l._offsets(d, offsets)
    _l._check(L.mx_linear8_dequantize(d, role, form, c, p, dt, ld, off, _mx._stream(stream, at, qat, oat)),
              "mx_linear8_dequantize")


def _product(name, d, q1, role1, form1, q2, role2, form2, out, role, what, workspace, offsets, stream):
    L = _load()
    p, dt, ld, at = _l._matrix(out, _l._dims(d, role), what)
    ws, n, wat = _l._bytes(workspace, "workspace")
    off, oat = _l._offsets(d, offsets)
    a, aat = _q(q1, d, role1, (form1,), "wq" if role1 == _mx.MX_ROLE_WEIGHT else "dyq")
    b, bat = _q(q2, d, role2, (form2,), "xq" if role2 == _mx.MX_ROLE_ACT else "dyq")
    _l._check(getattr(L, name)(d, a, b, p, dt, ld, off, ws, n, _mx._stream(stream, at, aat, bat, wat, oat)), name)


def mx_linear8_fwd(d: mx_linear_desc, wq, xq, y, workspace=None, offsets=None, stream=None) -> None:
    """Y = X W^T."""
    _product("mx_linear8_fwd", d, wq, _mx.MX_ROLE_WEIGHT, MX_FORM_ROWS, xq, _mx.MX_ROLE_ACT, MX_FORM_ROWS, y,
             _mx.MX_ROLE_GRAD, "y", workspace, offsets, stream)


def mx_linear8_dgrad(d: mx_linear_desc, wq, dyq, dx, workspace=None, offsets=None, stream=None) -> None:
    """dX = dY W."""
    _product("mx_linear8_dgrad", d, wq, _mx.MX_ROLE_WEIGHT, MX_FORM_COLS, dyq, _mx.MX_ROLE_GRAD, MX_FORM_ROWS, dx,
             _mx.MX_ROLE_ACT, "dx", workspace, offsets, stream)


def mx_linear8_wgrad(d: mx_linear_desc, dyq, xq, dw, workspace=None, offsets=None, stream=None) -> None:
    """dW = dY^T X."""
    _product("mx_linear8_wgrad", d, dyq, _mx.MX_ROLE_GRAD, MX_FORM_COLS, xq, _mx.MX_ROLE_ACT, MX_FORM_COLS, dw,
             _mx.MX_ROLE_WEIGHT, "dw", workspace, offsets, stream)


def mx_linear8_apply(d: mx_linear_desc, wq, x, y, workspace=None, offsets=None, stream=None) -> None:
    """Y = X W^T with X quantized on the way (1x128 blocks)."""
    L = _load()
    px, dx, ldx, xat = _l._matrix(x, (d.tokens, d.in_features), "x")
    py, dy, ldy, yat = _l._matrix(y, (d.tokens, d.out_features), "y")
    ws, n, wat = _l._bytes(workspace, "workspace")
    w, qat = _q(wq, d, _mx.MX_ROLE_WEIGHT, (MX_FORM_ROWS,), "wq")
    off, oat = _l._offsets(d, offsets)
    _l._check(L.mx_linear8_apply(d, w, px, dx, ldx, py, dy, ldy, off, ws, n,
                                 _mx._stream(stream, xat, yat, qat, wat, oat)), "mx_linear8_apply")
