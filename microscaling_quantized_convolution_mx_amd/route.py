"""The tokens' way to their experts and back: binding of include/mxroute.h.

The functions have the names of the C entry points and marshal arguments
only; see the header for what each computes.  expert is int32 and weight
float32, contiguous [tokens, choices], the tokens over any leading dimensions,
or flattened; tokens' matrices are [tokens, features], rows' matrices [tokens *
choices, features], as in linear.py.

A layer of experts, each token's weights and experts from its router:

    d = route_desc(tokens, choices, experts, features)
    ws = torch.empty(max(mx_route_workspace_bytes(d), 16), dtype=torch.uint8, device="cuda")
    mx_route_sort(d, expert, offsets, rows, workspace=ws)
    mx_route_gather(d, x, rows, xs)
    ...                                   # mx_linear8_apply(..., xs, ys, ..., offsets=offsets) on tokens * choices tokens
    mx_route_combine(d, ys, rows, weight, out)

and backward:

    mx_route_combine_bwd(d, dout, ys, rows, weight, dys, dweight)
    ...                                   # mx_linear8_dgrad, mx_linear8_wgrad
    mx_route_gather_bwd(d, dxs, rows, dx)
"""
from __future__ import annotations

import ctypes

import microscaling_quantized_convolution_mx_amd as _mx

from . import linear as _l

ROUTE_MAX_CHOICES = 64

ROUTE_EXPORTS = ("mx_route_workspace_bytes", "mx_route_sort", "mx_route_gather", "mx_route_gather_bwd", "mx_route_combine",
                 "mx_route_combine_bwd")


class mx_route_desc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("tokens", "choices", "experts", "features")]


_lib = None


def _load():
    """The library with the argument types of these entry points."""
    global _lib
    if _lib is None:
        _l._load()
        L = _mx.lib()
        D, P, I, I64, Z = ctypes.POINTER(mx_route_desc), ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        move = [D, P, I64, P, P, I64, I, P]
        for name, res, args in (
                ("mx_route_workspace_bytes", Z, [D]), ("mx_route_sort", I, [D, P, P, P, P, P, Z, P]),
                ("mx_route_gather", I, move), ("mx_route_gather_bwd", I, move),
                ("mx_route_combine", I, [D, P, I64, P, P, P, I64, I, P]),
                ("mx_route_combine_bwd", I, [D, P, I64, P, I64, P, P, P, I64, P, I, P])):
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def route_desc(tokens: int, choices: int, experts: int, features: int) -> mx_route_desc:
    return mx_route_desc(tokens, choices, experts, features)


def _array(t, n: int, dtype, what: str, choices: int = 1):
    """(address, device) of n contiguous elements of a type, `choices` of each token."""
    if t is None:
        return None, None
    if not isinstance(t, _l._torch.Tensor):
        raise TypeError(f"{what}: expected a torch tensor, got {type(t).__name__}")
    if t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{what}: must be a contiguous {str(dtype)[6:]} tensor, got {t.dtype}")
    if t.numel() != n:
        raise ValueError(f"{what}: {t.numel()} values, the call needs {n}")
    # (tokens may have any leading dimensions, or all be flattened; a [choices, tokens] tensor is not meant)
    if 1 < choices < n and t.dim() > 1 and t.shape[-1] != choices:
        raise ValueError(f"{what}: must be [{n // choices}, {choices}], got {tuple(t.shape)}")
    at = t.get_device()
    if at < 0:
        _l._in_host_memory(t, what)
    return t.data_ptr() or None, at


def _pair(d, a, b, tokens: str, rows: str):
    """The tokens' matrix a and the rows' matrix b, of one type."""
    pa, dt, lda, aat = _l._matrix(a, (d.tokens, d.features), tokens)
    pb, bt, ldb, bat = _l._matrix(b, (d.tokens * d.choices, d.features), rows)
    if a is not None and b is not None and bt != dt:
        raise ValueError(f"{rows}: must have {tokens}'s type, got {b.dtype}")
    return pa, lda, aat, pb, ldb, bat, dt if a is not None else bt


def mx_route_workspace_bytes(d: mx_route_desc) -> int:
    return _load().mx_route_workspace_bytes(d)


def mx_route_sort(d: mx_route_desc, expert, offsets, rows, order=None, workspace=None, stream=None) -> None:
    L = _load()
    n, i32 = d.tokens * d.choices, _l._torch.int32
    e, eat = _array(expert, n, i32, "expert", d.choices)
    o, oat = _array(offsets, d.experts + 1, i32, "offsets")
    r, rat = _array(rows, n, i32, "rows", d.choices)
    q, qat = _array(order, n, i32, "order")
    ws, nb, wat = _l._bytes(workspace, "workspace")
    _l._check(L.mx_route_sort(d, e, o, r, q, ws, nb, _mx._stream(stream, eat, oat, rat, qat, wat)), "mx_route_sort")


def mx_route_gather(d: mx_route_desc, x, rows, out, stream=None) -> None:
    """out[rows[t][j]] = x[t]."""
    L = _load()
    px, ldx, xat, po, ldo, oat, dt = _pair(d, x, out, "x", "out")
    r, rat = _array(rows, d.tokens * d.choices, _l._torch.int32, "rows", d.choices)
    _l._check(L.mx_route_gather(d, px, ldx, r, po, ldo, dt, _mx._stream(stream, xat, oat, rat)), "mx_route_gather")


def mx_route_gather_bwd(d: mx_route_desc, dout, rows, dx, stream=None) -> None:
    """dx[t] = sum over j of dout[rows[t][j]]."""
    L = _load()
    px, ldx, xat, po, ldo, oat, dt = _pair(d, dx, dout, "dx", "dout")
    r, rat = _array(rows, d.tokens * d.choices, _l._torch.int32, "rows", d.choices)
    _l._check(L.mx_route_gather_bwd(d, po, ldo, r, px, ldx, dt, _mx._stream(stream, xat, oat, rat)), "mx_route_gather_bwd")


def mx_route_combine(d: mx_route_desc, y, rows, weight, out, stream=None) -> None:
    """out[t] = sum over j of weight[t][j] * y[rows[t][j]]."""
    L = _load()
    po, ldo, oat, py, ldy, yat, dt = _pair(d, out, y, "out", "y")
    r, rat = _array(rows, d.tokens * d.choices, _l._torch.int32, "rows", d.choices)
    w, wat = _array(weight, d.tokens * d.choices, _l._torch.float32, "weight", d.choices)
    _l._check(L.mx_route_combine(d, py, ldy, r, w, po, ldo, dt, _mx._stream(stream, oat, yat, rat, wat)), "mx_route_combine")


def mx_route_combine_bwd(d: mx_route_desc, dout, y, rows, weight, dy=None, dweight=None, stream=None) -> None:
    """dy[rows[t][j]] = weight[t][j] * dout[t]; dweight[t][j] = <dout[t], y[rows[t][j]]>."""
    L = _load()
    po, ldo, oat, py, ldy, yat, dt = _pair(d, dout, y, "dout", "y")
    _, _, _, pd, ldd, dat, ddt = _pair(d, None, dy, "dout", "dy")
    if dy is not None and ddt != dt:
        raise ValueError(f"dy: must have dout's type, got {dy.dtype}")
    n = d.tokens * d.choices
    r, rat = _array(rows, n, _l._torch.int32, "rows", d.choices)
    w, wat = _array(weight, n, _l._torch.float32, "weight", d.choices)
    g, gat = _array(dweight, n, _l._torch.float32, "dweight", d.choices)
    _l._check(L.mx_route_combine_bwd(d, po, ldo, py, ldy, r, w, pd, ldd, g, dt,
                                     _mx._stream(stream, oat, yat, dat, rat, wat, gat)), "mx_route_combine_bwd")
