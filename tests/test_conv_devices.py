"""Convolution calls whose tensors lie on different GPUs, or on another than
the call's stream, are refused before anything is launched (host logic, as
in test_linear_devices.py)."""
import pytest
import torch

import microscaling_quantized_convolution_mx_amd as mx
from test_linear_devices import Stream, on

CALLS = {"quantize_cbf": ("src", "q"), "conv_fwd": ("wq", "xq", "y"), "conv_fwd_amax": ("wq", "xq", "y", "amax"),
         "conv_dgrad": ("wq", "dyq", "dx"), "conv_wgrad": ("dyq", "xq", "dw", "ws"), "conv_wgrad_noalloc": ("dyq", "xq", "dw"),
         "im2col_cbf": ("x", "xcol"), "dequantize": ("q", "dst")}
CASES = [(c, a) for c, args in CALLS.items() for a in args]


@pytest.fixture
def reached(monkeypatch):
    """The calls that reach the library; the current device is 0, its stream 0x1000."""
    calls, real = [], mx.lib()

    class Lib:
        def __getattr__(self, name):
            f = getattr(real, name)
            return f if name.endswith("_bytes") else lambda *a: calls.append((name, a[-1])) or 0
    fake = Lib()
    monkeypatch.setattr(mx, "lib", lambda: fake)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0x1000 + d, raising=False)
    for name in ("_current_device", "_current_stream"):  # not those of another test
        monkeypatch.setattr(mx, name, None)
    return calls


def run(call, where, stream=None, part="codes"):
    """`call` with each argument on the device that where(argument) gives (of a QTensor: its buffer `part`, the rest on 0)."""
    d = mx.desc(32, 32, 32, 4, 4, 3, 3)

    def t(name, *shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(on(where(name)))

    def q(name, role):
        v = mx.QTensor(d, role, "cpu")
        for b in ("codes", "scales", "tensor_scale", "amax"):
            setattr(v, b, getattr(v, b).as_subclass(on(where(name) if part in (b, "all") else 0)))
        return v
    x, y, w = (mx.role_numel(d, r) for r in (mx.MX_ROLE_ACT, mx.MX_ROLE_GRAD, mx.MX_ROLE_WEIGHT))
    wq, xq, dyq = (lambda: q("wq", mx.MX_ROLE_WEIGHT)), (lambda: q("xq", mx.MX_ROLE_ACT)), (lambda: q("dyq", mx.MX_ROLE_GRAD))
    f = getattr(mx, "mx_" + call)
    args = {"quantize_cbf": lambda: (d, 0, t("src", x), q("q", 0)), "conv_fwd": lambda: (d, wq(), xq(), t("y", y)),
            "conv_fwd_amax": lambda: (d, wq(), xq(), t("y", y), t("amax", 1 << 16)),
            "conv_dgrad": lambda: (d, wq(), dyq(), t("dx", x)), "conv_wgrad": lambda: (d, dyq(), xq(), t("dw", w), t("ws", 1 << 16)),
            "conv_wgrad_noalloc": lambda: (d, dyq(), xq(), t("dw", w)), "im2col_cbf": lambda: (d, t("x", x), t("xcol", 9 * x)),
            "dequantize": lambda: (d, 0, q("q", 0), t("dst", x))}[call]()
    f(*args, stream=stream)


@pytest.mark.parametrize("call,odd", CASES)
def test_one_tensor_on_another_device(reached, call, odd):
    for stream in (None, 0, 0x7000, Stream(0)):
        for part in ("codes", "scales", "tensor_scale", "amax") if odd.endswith("q") else ("codes",):
            with pytest.raises(ValueError, match="device"):
                run(call, lambda name: int(name == odd), stream, part)
    assert not reached


@pytest.mark.parametrize("call", list(CALLS))
def test_tensors_on_the_streams_device_pass(reached, call):
    for device, stream, handle in ((0, None, 0x1000), (0, 0, 0), (0, Stream(0), 0x5000), (1, Stream(1), 0x5000),
                                   (0, 0x7000, 0x7000), (1, 0x7000, 0x7000)):
        run(call, lambda name: device, stream, "all")
        (name, got), = reached
        assert name == "mx_" + call and got == handle
        reached.clear()
    with pytest.raises(ValueError, match="device 1"):
        run(call, lambda name: 1, None, "all")


def test_raw_addresses_pass(reached):
    d = mx.desc(32, 32, 32, 4, 4, 3, 3)
    raw = mx.mx_qtensor(0x10000, 0x10000, 0x10000, 0x10000)
    mx.mx_conv_fwd(d, raw, raw, 0x10000)
    mx.mx_conv_fwd(d, raw, raw, 0x10000, stream=0x7000)
    assert [h for _, h in reached] == [0x1000, 0x7000]
