"""The root-mean-square norm with the residual's addition: binding of include/mxnorm.h.

The functions have the names of the C entry points and marshal arguments
only; see the header for what each computes, and linear.py for the matrices.
A block of a model in training, and one whose next layer is in 8 bits:

    d = norm_desc(tokens, features, eps=1e-6)
    mx_norm_fwd(d, x, weight, y, residual=r, total=r, rstd=rstd)      # the residual is updated in place
    ws = torch.empty(mx_norm_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    mx_norm_bwd(d, dy, r, weight, rstd, dx, dweight, dtotal=dr, workspace=ws)

    xq = Linear8QTensor(linear_desc(tokens, out_features, features, block=1), MX_ROLE_ACT)
    mx_norm_fwd(d, x, weight, residual=r, total=r, yq=xq)             # then mx_linear8_fwd(..., xq, ...)
"""
from __future__ import annotations

import ctypes

import microscaling_quantized_convolution_mx_amd as _mx

from . import linear as _l
from . import linear8 as _l8

NORM_EXPORTS = ("mx_norm_fwd", "mx_norm_workspace_bytes", "mx_norm_bwd")


class mx_norm_desc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("features", ctypes.c_int32), ("eps", ctypes.c_float)]


_lib = None


def _load():
    """The library with the argument types of these entry points."""
    global _lib
    if _lib is None:
        _l8._load()
        L = _mx.lib()
        D, Q, P = ctypes.POINTER(mx_norm_desc), ctypes.POINTER(_l.mx_linear_qtensor), ctypes.c_void_p
        I, I64, Z = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        for name, res, args in (
                ("mx_norm_fwd", I, [D, P, I64, P, I64, I, P, I, P, I64, P, I, I64, Q, P, P]),
                ("mx_norm_workspace_bytes", Z, [D]),
                ("mx_norm_bwd", I, [D, P, I, I64, P, I64, P, I64, I, P, I, P, P, I64, P, P, Z, P])):
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def norm_desc(tokens: int, features: int, eps: float = 1e-6) -> mx_norm_desc:
    return mx_norm_desc(tokens, features, eps)


def _vector(t, n: int, what: str):
    """(address, mx_dtype, device) of n contiguous elements."""
    if t is None:
        return None, _l.MX_F32, None
    if not isinstance(t, _l._torch.Tensor):
        raise TypeError(f"{what}: expected a torch tensor, got {type(t).__name__}")
    dt = _l._dtypes.get(t.dtype)
    if dt is None:
        raise ValueError(f"{what}: must be float32, bfloat16 or float16, got {t.dtype}")
    if t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what}: must be {n} contiguous elements, got {tuple(t.shape)}")
    at = t.get_device()
    if at < 0:
        _l._in_host_memory(t, what)
    return t.data_ptr() or None, dt, at


def _f32(t, n: int, what: str):
    """(address, device) of n contiguous fp32 elements."""
    p, dt, at = _vector(t, n, what)
    if dt != _l.MX_F32:
        raise ValueError(f"{what}: must be float32, got {t.dtype}")
    return p, at


def _like(t, shape, dt: int, other: str, what: str):
    """_matrix of a tensor that has the type of `other`; None has any."""
    p, got, ld, at = _l._matrix(t, shape, what)
    if t is not None and got != dt:
        raise ValueError(f"{what}: must have {other}'s type, got {t.dtype}")
    return p, ld, at


def _q(q, d):
    """(mx_linear_qtensor, device) of a tensor whose row form takes the norm in 8 bits."""
    if isinstance(q, _l8.Linear8QTensor):
        padded = (d.tokens + 127) // 128 * ((d.features + 127) // 128)  # blocks of 128x128
        have = q.bytes.get(_l.MX_FORM_ROWS)
        if have is not None and q.is_cuda and have[0] >= 16384 * padded and have[1] >= 128 * padded:
            return q.c, q.device_index
    # what has no room, or is something else, is told apart as the 8-bit layers do
    return _l8._q(q, _l.mx_linear_desc(d.tokens, 1, d.features, 0, 1), _mx.MX_ROLE_ACT, (_l.MX_FORM_ROWS,), "yq")


def mx_norm_fwd(d: mx_norm_desc, x, weight, y=None, residual=None, total=None, yq=None, rstd=None, stream=None) -> None:
    """total = x + residual; y = total * rstd * weight, also or instead in 8 bits (yq, a Linear8QTensor of the
    activation that the next layer takes)."""
    L = _load()
    shape = (d.tokens, d.features)
    px, dt, ldx, xat = _l._matrix(x, shape, "x")
    pr, ldr, rat = _like(residual, shape, dt, "x", "residual")
    pw, wdt, wat = _vector(weight, d.features, "weight")
    pt, ldt, tat = _like(total, shape, dt, "x", "total")
    py, ydt, ldy, yat = _l._matrix(y, shape, "y")
    q = qat = None
    if yq is not None:
        q, qat = _q(yq, d)
    ps, sat = _f32(rstd, d.tokens, "rstd")
    _l._check(L.mx_norm_fwd(d, px, ldx, pr, ldr, dt, pw, wdt, pt, ldt, py, ydt, ldy, q, ps,
                            _mx._stream(stream, xat, rat, wat, tat, yat, qat, sat)), "mx_norm_fwd")


def mx_norm_workspace_bytes(d: mx_norm_desc) -> int:
    return _load().mx_norm_workspace_bytes(d)


def mx_norm_bwd(d: mx_norm_desc, dy, total, weight, rstd, dx=None, dweight=None, dtotal=None, workspace=None,
                stream=None) -> None:
    """dx, which is the gradient of x and of the residual, and dweight."""
    L = _load()
    shape = (d.tokens, d.features)
    pdy, dydt, lddy, dyat = _l._matrix(dy, shape, "dy")
    pt, dt, ldt, tat = _l._matrix(total, shape, "total")
    pdt, lddt, dtat = _like(dtotal, shape, dt, "total", "dtotal")
    pw, wdt, wat = _vector(weight, d.features, "weight")
    ps, sat = _f32(rstd, d.tokens, "rstd")
    pdx, lddx, dxat = _like(dx, shape, dt, "total", "dx")
    pdw, dwat = _f32(dweight, d.features, "dweight")
    ws, n, wsat = _l._bytes(workspace, "workspace")
    _l._check(L.mx_norm_bwd(d, pdy, dydt, lddy, pt, ldt, pdt, lddt, dt, pw, wdt, ps, pdx, lddx, pdw, ws, n,
                            _mx._stream(stream, dyat, tat, dtat, wat, sat, dxat, dwat, wsat)), "mx_norm_bwd")
