"""Every variant of the linear layers' products and of the few-token kernel,
in every type, at the cases of linear_variants.  Quantized operands are
taken from the dequantizer, which test_gpu_linear.py holds to a 64-bit
implementation; every output is compared with the 64-bit product of them."""
import pytest
import torch

import linear_variants as V
import microscaling_quantized_convolution_mx_amd as mx
from gpu_util import say

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACT, WEIGHT, GRAD = mx.MX_ROLE_ACT, mx.MX_ROLE_WEIGHT, mx.MX_ROLE_GRAD


def rand(seed, *shape, dt):
    """Values over some octaves, with exact zeros among them."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(*shape, device=DEV, generator=g) * torch.exp2(4 * torch.rand(*shape, device=DEV, generator=g) - 2)
    return (x * (torch.rand(*shape, device=DEV, generator=g) >= 0.05)).to(TYPES[dt])


def padded(pad, dt, *shape):
    """NaN outputs with `pad` elements of 7 between rows, starting at an odd element if there are any."""
    rows, cols = torch.Size(shape[:-1]).numel(), shape[-1]
    buf = torch.full((rows * (cols + pad) + 65,), 7.0, dtype=TYPES[dt], device=DEV)
    v = buf[1 if pad else 0:][:rows * (cols + pad)].view(*shape[:-1], cols + pad)[..., :cols]
    return v.fill_(float("nan"))


def check_gaps(t, pad):
    if pad:
        rows, cols = t.shape[:-1].numel(), t.shape[-1]
        full = t.as_strided((rows, cols + pad), (cols + pad, 1))
        assert bool((full[:-1, cols:] == 7.0).all())


def check(got, p, q, contracted, dt, what):
    """got against p @ q: the bound of `contracted` fp32 additions in any order
    (2^-23 of the magnitudes each) and of one rounding to the type."""
    ref, mags = p @ q, p.abs() @ q.abs()
    unit = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dt]
    s = contracted * 2.0 ** -23 * mags
    lim = s + unit * (ref.abs() + s) + (2.0 ** -25 if dt == "f16" else 0.0) + 2.0 ** -148
    err = (got.double() - ref).abs()
    assert bool((err <= lim).all()), f"{what}: {float((err / lim).nan_to_num(1e30).max())} of the bound"


def quantized(d, role, t, off=None, **kw):
    q = mx.LinearQTensor(d, role, DEV, **kw)
    for f in q.buffers.values():
        for b in f:
            b.fill_(0xFF)
    mx.mx_linear_quantize(d, role, t, q, offsets=off)
    return q


def values(d, role, q, like, off=None):
    out = torch.zeros(like.shape, device=DEV)
    mx.mx_linear_dequantize(d, role, q, out, offsets=off)
    return out.double()


def setup(case):
    m, n, k, lens = case
    e = len(lens or ())
    ends = torch.tensor([0] + list(lens or [m])).cumsum(0).tolist()
    off = torch.tensor(ends, dtype=torch.int32, device=DEV) if e else None
    return mx.linear_desc(m, n, k, experts=e), off, list(zip(ends[:-1], ends[1:])), ((e,) if e else ())


def workspace(d):
    return torch.full((max(mx.mx_linear_workspace_bytes(d), 16),), 0xFF, dtype=torch.uint8, device=DEV)


def products(case, dt, pad, calls, seed=1):
    m, n, k, lens = case
    d, off, segs, lead = setup(case)
    ws = workspace(d)
    x, dy, w = rand(seed, m, k, dt=dt), rand(seed + 1, m, n, dt=dt), rand(seed + 2, *lead, n, k, dt=dt)
    xq, dyq, wq = quantized(d, ACT, x, off), quantized(d, GRAD, dy, off), quantized(d, WEIGHT, w)
    xv, dyv, wv = values(d, ACT, xq, x, off), values(d, GRAD, dyq, dy, off), values(d, WEIGHT, wq, w).reshape(-1, n, k)
    if V.FWD in calls:
        y = padded(pad, dt, m, n)
        mx.mx_linear_fwd(d, wq, xq, y, ws, offsets=off)
        check_gaps(y, pad)
        for i, (a, b) in enumerate(segs):
            if b > a:
                check(y[a:b], xv[a:b], wv[i].T, k, dt, f"y of {i}")
    if V.DGRAD in calls:
        dx = padded(pad, dt, m, k)
        mx.mx_linear_dgrad(d, wq, dyq, dx, ws, offsets=off)
        check_gaps(dx, pad)
        for i, (a, b) in enumerate(segs):
            if b > a:
                check(dx[a:b], dyv[a:b], wv[i], n, dt, f"dx of {i}")
    if V.WGRAD in calls:
        dw = padded(pad, dt, *lead, n, k)
        mx.mx_linear_wgrad(d, dyq, xq, dw, ws, offsets=off)
        check_gaps(dw, pad)
        for i, (a, b) in enumerate(segs):
            check(dw[i] if lens else dw, dyv[a:b].T, xv[a:b], b - a, dt, f"dw of {i}")


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("case", [c[0] for c in V.PRODUCTS], ids=lambda c: "x".join(map(str, c[:3])) + ("e" if c[3] else ""))
def test_products(case, dt):
    """Contiguous rows, and rows with gaps between them that start at any element."""
    for pad in (0, 5):
        say("products", case, dt, pad)
        products(case, dt, pad, (V.FWD, V.DGRAD, V.WGRAD))


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("case", [c[0] for c in V.FEW_TOKENS], ids=lambda c: "x".join(map(str, c[:3])) + ("e" if c[3] else ""))
def test_few_tokens(case, dt):
    m, n, k, lens = case
    d, off, segs, lead = setup(case)
    for pad in (0, 5):
        say("few", case, dt, pad)
        products(case, dt, pad, (V.FWD, V.DGRAD))
        x, w = padded(pad, dt, m, k), rand(8, *lead, n, k, dt="bf16")
        x.copy_(rand(7, m, k, dt=dt))
        one = mx.linear_desc(m, n, k, experts=d.experts, block=1)
        xv = values(one, ACT, quantized(one, ACT, x, off), x, off)
        wq = quantized(d, WEIGHT, w, cols=False)
        wv = values(d, WEIGHT, wq, w).reshape(-1, n, k)
        y = padded(pad, dt, m, n)
        mx.mx_linear_apply(d, wq, x, y, workspace(d), offsets=off)
        check_gaps(y, pad)
        for i, (a, b) in enumerate(segs):
            if b > a:
                check(y[a:b], xv[a:b], wv[i].T, k, dt, f"apply, {i}")


@pytest.mark.parametrize("case,dt,calls,size", [
    ((8200, 8300, 300, None), "f32", (V.FWD,), 128), ((8200, 16391, 130, None), "f16", (V.FWD,), 128),
    ((11500, 11504, 3500, None), "f32", (V.FWD,), 256), ((11500, 11721, 4900, None), "bf16", (V.FWD,), 256),
    ((3500, 11500, 11501, None), "f32", (V.WGRAD,), 256), ((0, 8200, 8201, None), "f32", (V.WGRAD,), 64)])
def test_outputs_past_the_caches(case, dt, calls, size):
    """256 MiB of output and more, rows aligned and not, from each tile."""
    say("past the caches", case, dt, calls)
    m, n, k, _ = case
    d = mx.linear_desc(m, n, k)
    rows, cols = ((m, n), (m, k), (n, k))[calls[0]]
    assert rows * cols * TYPES[dt].itemsize >= 1 << 28
    assert V.variant(d, calls[0])[:3] == (V.PRODUCT, size, 1)
    products(case, dt, 0, calls)
