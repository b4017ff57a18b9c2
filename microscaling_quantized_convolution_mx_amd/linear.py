"""Microscaled linear layers and the gradient clip: binding of include/mxlinear.h.

The functions have the names of the C entry points and marshal arguments
only; see the header for what each computes, its layouts and its errors.
Matrices are torch tensors in device memory, float32, bfloat16 or float16,
with unit stride along the last dimension and any stride between rows, all of
a call on the device of its stream:

    X, dX   [tokens, in_features]
    Y, dY   [tokens, out_features]
    W, dW   [out_features, in_features], or [experts, out_features, in_features]

A layer that trains:

    d = linear_desc(tokens, out_features, in_features)
    xq, wq, dyq = (LinearQTensor(d, role) for role in (MX_ROLE_ACT, MX_ROLE_WEIGHT, MX_ROLE_GRAD))
    ws = torch.empty(mx_linear_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    mx_linear_quantize(d, MX_ROLE_ACT, x, xq)
    mx_linear_quantize(d, MX_ROLE_WEIGHT, w, wq)
    mx_linear_fwd(d, wq, xq, y, ws)
    mx_linear_quantize(d, MX_ROLE_GRAD, dy, dyq, MX_SR, seed)
    mx_linear_dgrad(d, wq, dyq, dx, ws)
    mx_linear_wgrad(d, dyq, xq, dw, ws)

and one that serves: quantize W once, then mx_linear_apply(d, wq, x, y, ws).
With experts, every call but W's quantization takes `offsets`, int32
[experts + 1]: tokens are sorted by expert, expert e's are rows
offsets[e] .. offsets[e+1]-1.
"""
from __future__ import annotations

import ctypes

import microscaling_quantized_convolution_mx_amd as _mx

MX_F32, MX_BF16, MX_F16 = 0, 1, 2
MX_FORM_ROWS, MX_FORM_COLS = 0, 1
LINEAR_MAX_EXPERTS = 1024

LINEAR_EXPORTS = ("mx_linear_code_bytes", "mx_linear_scale_bytes", "mx_linear_quantize", "mx_linear_dequantize",
                  "mx_linear_workspace_bytes", "mx_linear_fwd", "mx_linear_dgrad", "mx_linear_wgrad", "mx_linear_apply",
                  "mx_grad_workspace_bytes", "mx_grad_norm", "mx_grad_clip")


class mx_linear_desc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("tokens", "out_features", "in_features", "experts", "block")]


class mx_linear_qtensor(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in ("rows", "row_scales", "cols", "col_scales")]


class mx_grad_list(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int32), ("grads", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("numel", ctypes.c_void_p), ("dtypes", ctypes.c_void_p)]


_lib = None
_torch = None
_dtypes = None


def _load():
    """The library with the argument types of these entry points."""
    global _lib, _torch, _dtypes
    if _lib is None:
        import torch
        _torch = torch
        _dtypes = {torch.float32: MX_F32, torch.bfloat16: MX_BF16, torch.float16: MX_F16}
        L = _mx.lib()
        D, Q, P = ctypes.POINTER(mx_linear_desc), ctypes.POINTER(mx_linear_qtensor), ctypes.c_void_p
        I, I64, Z, G = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.POINTER(mx_grad_list)
        product = [D, Q, Q, P, I, I64, P, P, Z, P]
        for name, res, args in (
                ("mx_linear_code_bytes", Z, [D, I, I]), ("mx_linear_scale_bytes", Z, [D, I, I]),
                ("mx_linear_workspace_bytes", Z, [D]),
                ("mx_linear_quantize", I, [D, I, P, I, I64, P, Q, I, ctypes.c_uint64, P]),
                ("mx_linear_dequantize", I, [D, I, I, Q, P, I, I64, P, P]),
                ("mx_linear_fwd", I, product), ("mx_linear_dgrad", I, product), ("mx_linear_wgrad", I, product),
                ("mx_linear_apply", I, [D, Q, P, I, I64, P, I, I64, P, P, Z, P]),
                ("mx_grad_workspace_bytes", Z, [ctypes.c_int32]), ("mx_grad_norm", I, [G, P, P, Z, P]),
                ("mx_grad_clip", I, [G, ctypes.c_float, P, P, Z, P])):
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def linear_desc(tokens: int, out_features: int, in_features: int, experts: int = 0, block: int = 32) -> mx_linear_desc:
    """experts: 0 for one layer, else the number of weight matrices.
    block: 32 (32x32 blocks, forward and both gradients) or 1 (1x32 blocks,
    forward only)."""
    return mx_linear_desc(tokens, out_features, in_features, experts, block)


def _dims(d: mx_linear_desc, role: int):
    if role == _mx.MX_ROLE_WEIGHT:
        return (d.out_features, d.in_features) if d.experts <= 0 else (d.experts, d.out_features, d.in_features)
    return d.tokens, (d.out_features if role == _mx.MX_ROLE_GRAD else d.in_features)


def _in_host_memory(t, what: str) -> None:
    """Refuses a tensor without a device index that is in host memory."""
    if not t.is_cuda:
        raise ValueError(f"{what}: must be in device memory, got a {t.device.type} tensor")


def _matrix(t, shape, what: str):
    """(address, mx_dtype, row stride, device) of a tensor after checking it:
    nothing that the kernels could not read reaches them.  None passes through
    as a NULL float32 matrix (the library reports MX_ERR_NULL)."""
    if t is None:
        return None, MX_F32, shape[-1], None
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{what}: expected a torch tensor, got {type(t).__name__}")
    dt = _dtypes.get(t.dtype)
    if dt is None:
        raise ValueError(f"{what}: must be float32, bfloat16 or float16, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, the call needs {tuple(shape)}")
    at = t.get_device()
    if at < 0:
        _in_host_memory(t, what)
    if t.is_contiguous():
        return t.data_ptr() or None, dt, shape[-1], at
    st = t.stride()
    rows, cols = shape[-2], shape[-1]
    if st[-1] != 1 and cols > 1:
        raise ValueError(f"{what}: the last dimension must have stride 1, got {st[-1]}")
    ld = st[-2] if rows > 1 else cols
    if len(shape) == 3 and shape[0] > 1:
        ld = st[1] if rows > 1 else st[0]
        if st[0] != rows * ld:
            raise ValueError(f"{what}: experts must follow each other without a gap")
    if ld < cols:
        raise ValueError(f"{what}: rows overlap (row stride {ld}, {cols} columns)")
    return t.data_ptr() or None, dt, ld, at


def _offsets(d: mx_linear_desc, t):
    """(address, device) of the experts' offsets."""
    if d.experts <= 0 or t is None:
        return None, None
    if not isinstance(t, _torch.Tensor) or t.dtype != _torch.int32 or not t.is_contiguous():
        raise ValueError("offsets: must be a contiguous int32 tensor")
    if t.numel() != d.experts + 1:
        raise ValueError(f"offsets: {t.numel()} values, the call needs {d.experts + 1}")
    at = t.get_device()
    if at < 0:
        _in_host_memory(t, "offsets")
    return t.data_ptr(), at


def _bytes(t, what: str):
    """(address, bytes, device) of a workspace tensor of any type."""
    if t is None:
        return None, 0, None
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    at = t.get_device()
    if at < 0:
        _in_host_memory(t, what)
    return t.data_ptr() or None, t.numel() * t.element_size(), at


def mx_linear_code_bytes(d: mx_linear_desc, role: int, form: int = MX_FORM_ROWS) -> int:
    return _load().mx_linear_code_bytes(d, role, form)


def mx_linear_scale_bytes(d: mx_linear_desc, role: int, form: int = MX_FORM_ROWS) -> int:
    return _load().mx_linear_scale_bytes(d, role, form)


def mx_linear_workspace_bytes(d: mx_linear_desc) -> int:
    return _load().mx_linear_workspace_bytes(d)


class LinearQTensor:
    """Device buffers of a quantized matrix (owned by torch), in the forms asked for."""

    def __init__(self, d: mx_linear_desc, role: int, device="cuda", rows: bool = True, cols: bool | None = None):
        """cols: by default where the descriptor has that form (block 32)."""
        import torch
        self.role, self.desc = role, bytes(d)
        cols = d.block == 32 if cols is None else cols
        self.bytes, self.buffers = {}, {}
        for form, wanted in ((MX_FORM_ROWS, rows), (MX_FORM_COLS, cols)):
            n = (mx_linear_code_bytes(d, role, form), mx_linear_scale_bytes(d, role, form))
            if wanted:
                # 16 bytes at least, so that an empty tensor has valid pointers
                self.bytes[form] = n
                self.buffers[form] = tuple(torch.empty(max(b, 16), dtype=torch.uint8, device=device) for b in n)
        self.is_cuda = all(b.is_cuda for f in self.buffers.values() for b in f)
        self.device_index = next((b.get_device() for f in self.buffers.values() for b in f), None)
        none = (None, None)
        self.c = mx_linear_qtensor(*(b.data_ptr() if b is not None else None
                                     for form in (MX_FORM_ROWS, MX_FORM_COLS) for b in self.buffers.get(form, none)))


def _q(q, d: mx_linear_desc, role: int, forms, what: str):
    """(mx_linear_qtensor, device) of q, after checking that its buffers of
    `forms` hold what the call needs.  An mx_linear_qtensor struct passes
    unchecked."""
    if q is None or isinstance(q, mx_linear_qtensor):
        return q, None
    if not isinstance(q, LinearQTensor):
        raise TypeError(f"{what}: expected a LinearQTensor or an mx_linear_qtensor, got {type(q).__name__}")
    same = q.role == role and q.desc == bytes(d)  # sized for this very call
    L = _lib
    for form in forms:
        have = q.bytes.get(form)
        if have is None:
            raise ValueError(f"{what}: has no {'column' if form else 'row'} form")
        if not same and (have[0] < L.mx_linear_code_bytes(d, role, form) or have[1] < L.mx_linear_scale_bytes(d, role, form)):
            raise ValueError(f"{what}: {have[0]} bytes of codes, the call needs {L.mx_linear_code_bytes(d, role, form)}")
    if not q.is_cuda:
        raise ValueError(f"{what}: must be in device memory")
    return q.c, q.device_index


def _check(status: int, where: str) -> None:
    if status != 0:
        raise _mx.MxError(status, where)


def mx_linear_quantize(d: mx_linear_desc, role: int, src, dst, rounding: int = 0, seed: int = 0, offsets=None,
                       stream=None) -> None:
    """Fills the forms that dst has."""
    L = _load()
    p, dt, ld, at = _matrix(src, _dims(d, role), "src")
    q, qat = _q(dst, d, role, dst.bytes if isinstance(dst, LinearQTensor) else (), "dst")
    off, oat = _offsets(d, offsets)
    _check(L.mx_linear_quantize(d, role, p, dt, ld, off, q, rounding, seed & (2 ** 64 - 1),
                                _mx._stream(stream, at, qat, oat)), "mx_linear_quantize")


def mx_linear_dequantize(d: mx_linear_desc, role: int, q, dst, form: int = MX_FORM_ROWS, offsets=None, stream=None) -> None:
    L = _load()
    p, dt, ld, at = _matrix(dst, _dims(d, role), "dst")
    c, qat = _q(q, d, role, (form,), "q")
    off, oat = _offsets(d, offsets)
    _check(L.mx_linear_dequantize(d, role, form, c, p, dt, ld, off, _mx._stream(stream, at, qat, oat)), "mx_linear_dequantize")


def _product(name, d, q1, role1, form1, q2, role2, form2, out, role, what, workspace, offsets, stream):
    L = _load()
    p, dt, ld, at = _matrix(out, _dims(d, role), what)
    ws, n, wat = _bytes(workspace, "workspace")
    off, oat = _offsets(d, offsets)
    a, aat = _q(q1, d, role1, (form1,), "wq" if role1 == _mx.MX_ROLE_WEIGHT else "dyq")
    b, bat = _q(q2, d, role2, (form2,), "xq" if role2 == _mx.MX_ROLE_ACT else "dyq")
    _check(getattr(L, name)(d, a, b, p, dt, ld, off, ws, n, _mx._stream(stream, at, aat, bat, wat, oat)), name)


def mx_linear_fwd(d: mx_linear_desc, wq, xq, y, workspace=None, offsets=None, stream=None) -> None:
    """Y = X W^T."""
    _product("mx_linear_fwd", d, wq, _mx.MX_ROLE_WEIGHT, MX_FORM_ROWS, xq, _mx.MX_ROLE_ACT, MX_FORM_ROWS, y,
             _mx.MX_ROLE_GRAD, "y", workspace, offsets, stream)


def mx_linear_dgrad(d: mx_linear_desc, wq, dyq, dx, workspace=None, offsets=None, stream=None) -> None:
    """dX = dY W."""
    _product("mx_linear_dgrad", d, wq, _mx.MX_ROLE_WEIGHT, MX_FORM_COLS, dyq, _mx.MX_ROLE_GRAD, MX_FORM_ROWS, dx,
             _mx.MX_ROLE_ACT, "dx", workspace, offsets, stream)


def mx_linear_wgrad(d: mx_linear_desc, dyq, xq, dw, workspace=None, offsets=None, stream=None) -> None:
    """dW = dY^T X."""
    _product("mx_linear_wgrad", d, dyq, _mx.MX_ROLE_GRAD, MX_FORM_COLS, xq, _mx.MX_ROLE_ACT, MX_FORM_COLS, dw,
             _mx.MX_ROLE_WEIGHT, "dw", workspace, offsets, stream)


def mx_linear_apply(d: mx_linear_desc, wq, x, y, workspace=None, offsets=None, stream=None) -> None:
    """Y = X W^T with X quantized on the way (1x32 blocks)."""
    L = _load()
    px, dx, ldx, xat = _matrix(x, (d.tokens, d.in_features), "x")
    py, dy, ldy, yat = _matrix(y, (d.tokens, d.out_features), "y")
    ws, n, wat = _bytes(workspace, "workspace")
    w, qat = _q(wq, d, _mx.MX_ROLE_WEIGHT, (MX_FORM_ROWS,), "wq")
    off, oat = _offsets(d, offsets)
    _check(L.mx_linear_apply(d, w, px, dx, ldx, py, dy, ldy, off, ws, n, _mx._stream(stream, xat, yat, qat, wat, oat)),
           "mx_linear_apply")


class GradList:
    """Gradients of many parameters and where their clipped values go (by
    default the gradients themselves).  Holds the tensors; their addresses are
    laid out here, once, for every call with this list."""

    def __init__(self, grads, out=None):
        import torch
        _load()
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        if len(self.out) != len(self.grads):
            raise ValueError(f"{len(self.grads)} gradients, {len(self.out)} outputs")
        for i, (g, o) in enumerate(zip(self.grads, self.out)):
            for t, what in ((g, "gradient"), (o, "output")):
                if not isinstance(t, torch.Tensor):
                    raise TypeError(f"{what} {i}: expected a torch tensor, got {type(t).__name__}")
                if t.dtype not in _dtypes:
                    raise ValueError(f"{what} {i}: must be float32, bfloat16 or float16, got {t.dtype}")
                if not t.is_contiguous():
                    raise ValueError(f"{what} {i}: must be contiguous")
                if not t.is_cuda:
                    raise ValueError(f"{what} {i}: must be in device memory, got a {t.device.type} tensor")
            if g.dtype != o.dtype or g.numel() != o.numel():
                raise ValueError(f"output {i}: must have its gradient's type and size")
        at = {t.get_device() for t in (*self.grads, *self.out)}
        if len(at) > 1:
            raise ValueError(f"gradients and outputs on devices {sorted(at)}, one list is of one device")
        self.device_index = at.pop() if at else None
        n = max(len(self.grads), 1)
        self._a = ((ctypes.c_void_p * n)(*(g.data_ptr() or None for g in self.grads)),
                   (ctypes.c_void_p * n)(*(o.data_ptr() or None for o in self.out)),
                   (ctypes.c_int64 * n)(*(g.numel() for g in self.grads)),
                   (ctypes.c_int32 * n)(*(_dtypes[g.dtype] for g in self.grads)))
        self.c = mx_grad_list(len(self.grads), *(ctypes.addressof(a) for a in self._a))

    def __len__(self) -> int:
        return len(self.grads)


def mx_grad_workspace_bytes(grads) -> int:
    """grads: a GradList, or the number of tensors."""
    return _load().mx_grad_workspace_bytes(grads if isinstance(grads, int) else len(grads))


def mx_grad_norm(grads: GradList, norm, workspace=None, stream=None) -> None:
    """norm[0] = the norm over all gradients."""
    ws, n, at = _bytes(workspace, "workspace")
    _check(_load().mx_grad_norm(grads.c, _mx._buf(norm, 4, "norm"), ws, n,
                                _mx._stream(stream, grads.device_index, at, _mx._index(norm))), "mx_grad_norm")


def mx_grad_clip(grads: GradList, max_norm: float, norm, workspace=None, stream=None) -> None:
    """norm[0] = the norm over all gradients, which are then scaled by
    min(1, max_norm / (norm + 1e-6)) into their outputs."""
    ws, n, at = _bytes(workspace, "workspace")
    _check(_load().mx_grad_clip(grads.c, max_norm, _mx._buf(norm, 4, "norm"), ws, n,
                                _mx._stream(stream, grads.device_index, at, _mx._index(norm))), "mx_grad_clip")
