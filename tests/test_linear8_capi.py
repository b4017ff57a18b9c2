"""C ABI and binding of the linear layers in 8 bits, without a GPU: exports,
buffer sizes, every refusal on the host, and tensors on the wrong device."""
import os
import re

import pytest
import torch

import microscaling_quantized_convolution_mx_amd as mx
from microscaling_quantized_convolution_mx_amd import linear8 as M8
from test_linear_capi import A16, GOOD, ROOT, qt
from test_linear_devices import Stream, on

D8 = dict(GOOD, block=128)


def test_exports_every_declared_function():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mxlinear8.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(mx_[a-z0-9_]+)\s*\(", text))
    assert names == set(mx.LINEAR8_EXPORTS)
    for n in names:
        assert hasattr(mx.lib(), n) and hasattr(mx, n)


def test_buffer_sizes():
    for block in (1, 128):
        # padded to 128 both ways: a byte per code, a byte per 128 codes
        d = mx.linear_desc(100, 70, 200, block=block)
        for role, r, c in ((mx.MX_ROLE_ACT, 128, 256), (mx.MX_ROLE_WEIGHT, 128, 256), (mx.MX_ROLE_GRAD, 128, 128)):
            for form in (mx.MX_FORM_ROWS, mx.MX_FORM_COLS):
                assert mx.mx_linear8_code_bytes(d, role, form) == r * c
                assert mx.mx_linear8_scale_bytes(d, role, form) == r * c // 128
    d = mx.linear_desc(100, 70, 200, experts=5, block=1)
    assert mx.mx_linear8_code_bytes(d, mx.MX_ROLE_ACT) == 768 * 256
    assert mx.mx_linear8_code_bytes(d, mx.MX_ROLE_WEIGHT) == 5 * 128 * 256
    d = mx.linear_desc(0, 70, 200, block=1)
    assert mx.mx_linear8_code_bytes(d, mx.MX_ROLE_ACT) == 0 and mx.mx_linear8_workspace_bytes(d) == 0
    assert mx.mx_linear8_code_bytes(d, 7) == 0 and mx.mx_linear8_code_bytes(d, 0, 2) == 0
    # far sizes that a descriptor may have
    assert mx.mx_linear8_code_bytes(mx.linear_desc(2 ** 21, 128, 2 ** 15, block=1), 0) == 2 ** 36


def raw(name, d, *args):
    M8._load()
    return getattr(mx.lib(), name)(d, *args)


def quant(d, role=0, src=A16, dt=0, ld=200, off=None, q="ok"):
    return raw("mx_linear8_quantize", d, role, src, dt, ld, off, qt() if q == "ok" else q, None)


@pytest.mark.parametrize("change,status", [
    (dict(block=32), -4), (dict(block=0), -4), (dict(block=64), -4), (dict(tokens=-1), -2), (dict(out_features=0), -2),
    (dict(in_features=-3), -2), (dict(experts=-1), -2), (dict(experts=1025), -2), (dict(tokens=2 ** 31 - 1), -2),
    (dict(out_features=2 ** 31 - 1), -2), (dict(in_features=2 ** 31 - 1), -2), (dict(out_features=2 ** 22, experts=1024), -2),
    (dict(tokens=2 ** 30, out_features=2 ** 30, in_features=2 ** 30), -2)])
def test_descriptor_validation(change, status):
    d = mx.linear_desc(**dict(D8, **change))
    assert quant(d, ld=2 ** 31) == status
    assert mx.mx_linear8_workspace_bytes(d) == 0 and mx.mx_linear8_code_bytes(d, 0) == 0


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_refusals(block):
    d = mx.linear_desc(**dict(D8, block=block))
    assert quant(None) == -1
    assert quant(d, role=3) == -7
    assert quant(d, dt=3) == -3 and quant(d, dt=-1) == -3
    assert quant(d, ld=199) == -2 and quant(d, ld=2 ** 62) == -2
    assert quant(d, src=None) == -1 and quant(d, q=None) == -1
    assert quant(d, src=A16 + 2) == -5 and quant(d, src=A16 + 1, dt=1) == -5
    assert quant(d, q=qt(None, A16, None, None)) == -1
    assert quant(d, q=qt(A16, None)) == -1 and quant(d, q=qt(cs=None)) == -1
    assert quant(d, q=qt(rows=A16 + 8)) == -5 and quant(d, q=qt(cs=A16 + 4)) == -5
    e = mx.linear_desc(**dict(D8, block=block), experts=4)
    assert quant(e) == -1 and quant(e, off=A16 + 2) == -5

    def deq(form=0, q=None, dst=A16, role=0, dt=0):
        return raw("mx_linear8_dequantize", d, role, form, q or qt(), dst, dt, 200, None, None)
    assert deq(form=2) == -3 and deq(dst=None) == -1 and deq(role=5) == -7 and deq(dt=7) == -3
    assert deq(q=qt(rows=None)) == -1 and deq(form=1, q=qt(cols=None)) == -1
    # no tokens: nothing is needed, nothing runs
    none = mx.linear_desc(0, 70, 200, block=block)
    assert raw("mx_linear8_quantize", none, 0, None, 0, 200, None, qt(None, None, None, None), None) == 0


@pytest.mark.parametrize("name", ["mx_linear8_fwd", "mx_linear8_dgrad", "mx_linear8_wgrad"])
def test_product_refusals(name):
    d = mx.linear_desc(64, 128, 8192, block=128)
    need = mx.mx_linear8_workspace_bytes(d)

    def call(d, a="ok", b="ok", out=A16, dt=0, ld=8192, off=None, ws=A16, n=need):
        return raw(name, d, qt() if a == "ok" else a, qt() if b == "ok" else b, out, dt, ld, off, ws, n, None)
    assert call(None) == -1
    assert call(d, a=None) == -1 and call(d, b=None) == -1 and call(d, out=None) == -1
    assert call(d, a=qt(None, None, None, None)) == -1 and call(d, b=qt(A16, None, A16, None)) == -1
    assert call(d, dt=9) == -3 and call(d, ld=1) == -2 and call(d, out=A16 + 2) == -5
    assert call(d, b=qt(A16 + 1, A16, A16 + 1, A16)) == -5
    assert call(d, ws=A16 + 8) == -5
    assert call(mx.linear_desc(64, 128, 8192, experts=2, block=128)) == -1
    assert call(mx.linear_desc(64, 128, 8192, block=32)) == -4


def test_apply_refusals():
    d = mx.linear_desc(500, 128, 256, block=128)

    def call(d, w="ok", x=A16, xt=1, ldx=256, y=A16, yt=1, ldy=128, off=None, ws=A16, n=1 << 30):
        return raw("mx_linear8_apply", d, qt() if w == "ok" else w, x, xt, ldx, y, yt, ldy, off, ws, n, None)
    assert call(None) == -1 and call(d, w=None) == -1 and call(d, w=qt(rows=None)) == -1
    assert call(d, x=None) == -1 and call(d, y=None) == -1
    assert call(d, xt=4) == -3 and call(d, yt=4) == -3
    assert call(d, ldx=255) == -2 and call(d, ldy=127) == -2
    assert call(d, x=A16 + 1) == -5 and call(d, y=A16 + 1) == -5
    assert call(d, ws=None) == -6 and call(d, n=15) == -6
    assert call(mx.linear_desc(500, 128, 256, experts=3, block=128)) == -1
    assert call(mx.linear_desc(0, 128, 256, block=128), x=None, y=None, ws=None, n=0) == 0


def test_binding_rejects_unusable_tensors():
    d = mx.linear_desc(**D8)
    x = torch.zeros(100, 200)
    q = mx.Linear8QTensor(d, mx.MX_ROLE_ACT, device="cpu")
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        mx.mx_linear8_quantize(d, 0, x.double(), q)
    with pytest.raises(ValueError, match="shape"):
        mx.mx_linear8_quantize(d, 0, x[:99], q)
    with pytest.raises(ValueError, match="device memory"):
        mx.mx_linear8_quantize(d, 0, x, q)
    with pytest.raises(ValueError, match="no column form"):
        mx.mx_linear8_wgrad(d, mx.Linear8QTensor(d, 2, "cpu", cols=False), q, None)
    with pytest.raises(ValueError, match="no row form"):
        mx.mx_linear8_fwd(d, mx.Linear8QTensor(d, 1, "cpu", rows=False), q, None)
    with pytest.raises(ValueError, match="the call needs"):
        mx.mx_linear8_fwd(d, mx.Linear8QTensor(mx.linear_desc(1, 8, 8, block=1), 1, "cpu"), q, None)
    with pytest.raises(TypeError):
        mx.mx_linear8_fwd(d, 5, q, None)
    with pytest.raises(mx.MxError) as err:
        mx.mx_linear8_quantize(d, 0, None, qt(), stream=0)
    assert err.value.status == -1


def test_tensors_in_4_and_8_bits_are_told_apart():
    d4, d8 = mx.linear_desc(**GOOD), mx.linear_desc(**D8)
    q4, q8 = mx.LinearQTensor(d4, 0, "cpu"), mx.Linear8QTensor(d8, 0, "cpu")
    with pytest.raises(TypeError, match="Linear8QTensor"):
        mx.mx_linear8_fwd(d8, q4, q8, None)
    with pytest.raises(TypeError, match="LinearQTensor"):
        mx.mx_linear_fwd(d4, q8, q4, None)
    # one made for a block size serves the other
    assert q8.desc == mx.Linear8QTensor(mx.linear_desc(**GOOD, block=1), 0, "cpu").desc


CALLS = {"quantize": ("src", "q", "offsets"), "dequantize": ("dst", "q", "offsets"), "fwd": ("wq", "q", "y", "ws", "offsets"),
         "dgrad": ("wq", "dyq", "dx", "ws", "offsets"), "wgrad": ("dyq", "q", "dw", "ws", "offsets"),
         "apply": ("wq", "x", "y", "ws", "offsets")}


@pytest.fixture
def reached(monkeypatch):
    """The calls that reach the library; the current device is 0, its stream 0x1000."""
    M8._load()
    calls = []

    class Lib:
        def __getattr__(self, name):
            real = getattr(mx.lib(), name)
            return real if name.endswith("_bytes") else lambda *a: calls.append((name, a[-1])) or 0
    monkeypatch.setattr(M8, "_lib", Lib())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0x1000 + d, raising=False)
    for name in ("_current_device", "_current_stream"):
        monkeypatch.setattr(mx, name, None, raising=False)
    return calls


def run(call, where, stream=None):
    """`call` with each argument on the device that where(argument) gives."""
    m, n, k = 40, 32, 64
    d = mx.linear_desc(m, n, k, experts=2, block=128)

    def t(name, *shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(on(where(name)))

    def q(name, role):
        v = mx.Linear8QTensor(d, role, "cpu")
        v.is_cuda, v.device_index = True, where(name)
        return v
    off, ws = t("offsets", 3, dtype=torch.int32), t("ws", 1 << 20, dtype=torch.uint8)
    {"quantize": lambda: mx.mx_linear8_quantize(d, 0, t("src", m, k), q("q", 0), off, stream),
     "dequantize": lambda: mx.mx_linear8_dequantize(d, 0, q("q", 0), t("dst", m, k), 0, off, stream),
     "fwd": lambda: mx.mx_linear8_fwd(d, q("wq", 1), q("q", 0), t("y", m, n), ws, off, stream),
     "dgrad": lambda: mx.mx_linear8_dgrad(d, q("wq", 1), q("dyq", 2), t("dx", m, k), ws, off, stream),
     "wgrad": lambda: mx.mx_linear8_wgrad(d, q("dyq", 2), q("q", 0), t("dw", 2, n, k), ws, off, stream),
     "apply": lambda: mx.mx_linear8_apply(d, q("wq", 1), t("x", m, k), t("y", m, n), ws, off, stream)}[call]()


@pytest.mark.parametrize("call,odd", [(c, a) for c, args in CALLS.items() for a in args])
def test_one_tensor_on_another_device(reached, call, odd):
    for stream in (None, 0, 0x7000, Stream(0)):
        with pytest.raises(ValueError, match="device"):
            run(call, lambda name: int(name == odd), stream)
    assert not reached


@pytest.mark.parametrize("call", list(CALLS))
def test_tensors_on_the_streams_device_pass(reached, call):
    for device, stream, handle in ((0, None, 0x1000), (0, 0, 0), (0, Stream(0), 0x5000), (1, Stream(1), 0x5000),
                                   (1, 0x7000, 0x7000)):
        run(call, lambda name: device, stream)
        (name, got), = reached
        assert name.endswith(call) and got == handle
        reached.clear()
