"""Rows of very large and very small values through the norm: what a finite row
gives depends on its values alone, not on how the row is held, and is right over
fp32's whole range."""
import numpy as np
import pytest
import torch

import microscaling_quantized_convolution_mx_amd as mx
import norm_ref as R
from gpu_util import say
from test_gpu_linear import f64, rand
from test_gpu_norm import DEV, TYPES, check_codes, nans, tensor8

pytestmark = pytest.mark.gpu

# a wave's rows and a workgroup's of one and two pieces, and rows read twice
LENGTHS = [128, 512, 1000, 1024, 4096, 16384, 17000, 33000]
# a power of two that the rows are scaled with: squares past fp32 on either side, and sums past it whose squares are not
SCALES = [-120, -100, -75, -64, 59, 60, 62, 63, 64, 100, 124]


def rows(k, dt, e):
    """Rows of elements between 2^(e-2) and 2^e of either sign, exact in the type."""
    x = rand(3, 4, k, dt="f32")
    x = torch.copysign(0.25 + 0.75 * (x.abs() % 1.0), x).to(TYPES["bf16"]).float()
    return torch.ldexp(x, torch.tensor(e)).to(TYPES[dt])


@pytest.mark.parametrize("k", LENGTHS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_large_and_small_rows(k, dt):
    """The squares of 4 * 2^124 * 2^124 are past fp32, those of 2^-75 and less below its subnormals: with eps = 0, y and the codes are those of the rows between 1/4 and 1."""
    w = (1 + 0.5 * rand(5, k).abs().clamp(max=2)).to(DEV)
    d = mx.norm_desc(4, k, 0.0)
    x0 = rows(k, dt, 0)
    ref, rs = R.norm(f64(x0), f64(w), 0.0)
    dy = rand(6, 4, k)
    ws = torch.empty(mx.mx_norm_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    for e in SCALES:
        say("range", k, dt, e)
        x = rows(k, dt, e)
        assert np.array_equal(f64(x), np.ldexp(f64(x0), e))
        y, rstd, q = nans(4, k, dt="f32"), torch.full((4,), float("nan"), device=DEV), tensor8(4, k)
        mx.mx_norm_fwd(d, x.to(DEV), w, y, yq=q, rstd=rstd)
        torch.cuda.synchronize()
        # scaling by a power of two is exact: rstd is the other rows' times its inverse, rounded to fp32
        want = np.ldexp(rs[:, 0], -e)
        assert np.all(np.abs(f64(rstd) - want) <= want * (R.rstd_error(k) + R.U))
        assert np.all(np.abs(f64(y) - ref) <= R.bound(ref, np.abs(ref) * R.y_error(k), "f32"))
        check_codes(q, ref, R.y_error(k), 4, k)
        # and back, from that rstd
        dx, dw = nans(4, k, dt="f32") if dt == "f32" else None, torch.full((k,), float("nan"), device=DEV)
        mx.mx_norm_bwd(d, dy.to(DEV), x.to(DEV), w, rstd, dx, dw, workspace=ws)
        want, err, dwr, dwe = R.grads(f64(dy), f64(x), f64(w), f64(rstd)[:, None], 0.0)
        assert np.all(np.abs(f64(dw) - dwr) <= dwe + R.TINY["f32"])
        if dx is not None:
            # (below fp32's normal values each of its six roundings is half a step of its subnormals, at most)
            assert np.all(np.abs(f64(dx) - want) <= R.bound(want, err + 6 * R.TINY["f32"], "f32"))


def test_many_large_rows():
    """... in the kernel that writes the codes of four rows together."""
    m, k = 1100, 640
    for e in (-75, 62, 64):
        x = rows(k, "f32", 0).repeat(275, 1)
        w = torch.ones(k, device=DEV)
        ref, _ = R.norm(f64(x), f64(w), 0.0)
        q = tensor8(m, k)
        mx.mx_norm_fwd(mx.norm_desc(m, k, 0.0), torch.ldexp(x, torch.tensor(e)).to(DEV), w, yq=q)
        torch.cuda.synchronize()
        check_codes(q, ref, R.y_error(k), m, k)


@pytest.mark.parametrize("k", LENGTHS)
def test_ends_of_the_range(k):
    """fp32's largest value, whose rstd is a subnormal, and its smallest normal one."""
    w = torch.ones(k, device=DEV)
    x = torch.tensor([3.4028234663852886e38, 1.1754943508222875e-38])[:, None].repeat(1, k)
    y, rstd = nans(2, k), torch.full((2,), float("nan"), device=DEV)
    mx.mx_norm_fwd(mx.norm_desc(2, k, 0.0), x.to(DEV), w, y, rstd=rstd)
    want = 1.0 / f64(x)[:, 0]
    lim = want * R.rstd_error(k) + np.maximum(want * R.U, 2.0 ** -150)  # half a step of a normal or subnormal value
    assert np.all(np.abs(f64(rstd) - want) <= lim)
    # y takes that error of rstd, and two products
    assert np.all(np.abs(f64(y) - 1.0) <= (lim * f64(x)[:, 0])[:, None] + 2.02 * R.U)


@pytest.mark.parametrize("k", LENGTHS)
def test_infinities_and_zeros(k):
    """A row with an Inf has an rstd of 0, one of zeros without eps of Inf; the others are their own."""
    x = rows(k, "f32", 0)
    x[1, k - 1], x[2] = float("inf"), 0.0
    w = torch.ones(k, device=DEV)
    y, rstd = nans(4, k), torch.full((4,), float("nan"), device=DEV)
    mx.mx_norm_fwd(mx.norm_desc(4, k, 0.0), x.to(DEV), w, y, rstd=rstd)
    r, v = f64(rstd), f64(y)
    assert r[1] == 0.0 and np.isposinf(r[2]) and np.isfinite(r[[0, 3]]).all() and (r[[0, 3]] > 0).all()
    assert np.isnan(v[1, k - 1]) and not v[1, :k - 1].any() and np.isnan(v[2]).all() and np.isfinite(v[[0, 3]]).all()
