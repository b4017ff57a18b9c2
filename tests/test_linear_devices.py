"""Calls on the linear layers and the clip whose tensors lie on different GPUs,
or on another than the call's stream, are refused before anything is
launched (host logic: tensors that say which device they are on, and a library
that records what reaches it)."""
import pytest
import torch

import microscaling_quantized_convolution_mx_amd as mx
from microscaling_quantized_convolution_mx_amd import linear as ML


def on(index):
    """Tensors that say they are in the memory of this device."""
    class OnDevice(torch.Tensor):
        is_cuda = True
        device = torch.device("cuda", index)

        def get_device(self):
            return index
    return OnDevice


class Stream:
    def __init__(self, device, handle=0x5000):
        self.device_index, self.cuda_stream = device, handle


M, N, K = 40, 32, 64
CALLS = {
    "quantize": ("src", "q", "offsets"), "dequantize": ("dst", "q", "offsets"), "fwd": ("wq", "q", "y", "ws", "offsets"),
    "dgrad": ("wq", "dyq", "dx", "ws", "offsets"), "wgrad": ("dyq", "q", "dw", "ws", "offsets"),
    "apply": ("wq", "x", "y", "ws", "offsets"), "norm": ("list", "norm", "gws"), "clip": ("list", "norm", "gws")}
CASES = [(c, a) for c, args in CALLS.items() for a in args]


@pytest.fixture
def reached(monkeypatch):
    """The calls that reach the library; the current device is 0, its stream 0x1000."""
    ML._load()
    calls = []

    class Lib:
        def __getattr__(self, name):
            real = getattr(mx.lib(), name)
            return real if name.endswith("_bytes") else lambda *a: calls.append((name, a[-1])) or 0
    monkeypatch.setattr(ML, "_lib", Lib())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0x1000 + d, raising=False)
    for name in ("_current_device", "_current_stream"):  # not those of another test
        monkeypatch.setattr(mx, name, None, raising=False)
    return calls


def run(call, where, stream=None):
    """`call` with each argument on the device that where(argument) gives."""
    d = mx.linear_desc(M, N, K, experts=2)

    def t(name, *shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(on(where(name)))

    def q(name, role):
        v = mx.LinearQTensor(d, role, "cpu")
        v.is_cuda, v.device_index = True, where(name)
        return v
    off = t("offsets", 3, dtype=torch.int32)
    ws = t("ws", 1 << 20, dtype=torch.uint8)
    if call == "quantize":
        mx.mx_linear_quantize(d, mx.MX_ROLE_ACT, t("src", M, K), q("q", mx.MX_ROLE_ACT), offsets=off, stream=stream)
    elif call == "dequantize":
        mx.mx_linear_dequantize(d, mx.MX_ROLE_ACT, q("q", mx.MX_ROLE_ACT), t("dst", M, K), offsets=off, stream=stream)
    elif call == "fwd":
        mx.mx_linear_fwd(d, q("wq", 1), q("q", 0), t("y", M, N), ws, off, stream)
    elif call == "dgrad":
        mx.mx_linear_dgrad(d, q("wq", 1), q("dyq", 2), t("dx", M, K), ws, off, stream)
    elif call == "wgrad":
        mx.mx_linear_wgrad(d, q("dyq", 2), q("q", 0), t("dw", 2, N, K), ws, off, stream)
    elif call == "apply":
        mx.mx_linear_apply(d, q("wq", 1), t("x", M, K), t("y", M, N), ws, off, stream)
    else:
        lst = mx.GradList([t("list", 5), t("list", 7)])
        norm, gws = t("norm", 1), t("gws", 8192, dtype=torch.uint8)
        if call == "norm":
            mx.mx_grad_norm(lst, norm, gws, stream)
        else:
            mx.mx_grad_clip(lst, 1.0, norm, gws, stream)


def test_roles_are_numbered_as_used_here():
    assert (mx.MX_ROLE_ACT, mx.MX_ROLE_WEIGHT, mx.MX_ROLE_GRAD) == (0, 1, 2)


@pytest.mark.parametrize("call,odd", CASES)
def test_one_tensor_on_another_device(reached, call, odd):
    for stream in (None, 0, 0x7000, Stream(0)):
        with pytest.raises(ValueError, match="device"):
            run(call, lambda name: int(name == odd), stream)
    assert not reached


@pytest.mark.parametrize("call", list(CALLS))
def test_all_tensors_on_another_device_than_the_stream(reached, call):
    for stream in (None, 0, Stream(0)):
        with pytest.raises(ValueError, match="device 1"):
            run(call, lambda name: 1, stream)
    assert not reached


@pytest.mark.parametrize("call", list(CALLS))
def test_tensors_on_the_streams_device_pass(reached, call):
    for device, stream, handle in ((0, None, 0x1000), (0, 0, 0), (0, Stream(0), 0x5000), (1, Stream(1), 0x5000),
                                   (0, 0x7000, 0x7000), (1, 0x7000, 0x7000)):
        run(call, lambda name: device, stream)
        (name, got), = reached
        assert name.endswith(call) and got == handle
        reached.clear()


def test_a_list_of_two_devices(reached):
    a, b = torch.zeros(4).as_subclass(on(0)), torch.zeros(4).as_subclass(on(1))
    for grads, out in (([a, b], None), ([a, a], [a, b]), ([b], [a])):
        with pytest.raises(ValueError, match="devices"):
            mx.GradList(grads, out)
    assert mx.GradList([a, a]).device_index == 0 and mx.GradList([]).device_index is None
