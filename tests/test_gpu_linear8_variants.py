"""Every kernel that a product in 8 bits can take, in every type, against the
64-bit product of the quantized operands."""
import numpy as np
import pytest
import torch

import linear8_ref as R
import linear8_variants as V
import microscaling_quantized_convolution_mx_amd as mx
from gpu_util import say
from test_gpu_linear import f64, offsets_of, rand, strided
from test_gpu_linear8 import ACT, DEV, GRAD, TYPES, WEIGHT, product_case, quantize, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [p[0] for p in V.PRODUCTS], ids=lambda c: str(c)[:40])
@pytest.mark.parametrize("dt", list(TYPES))
def test_products(case, dt):
    m, n, k, lens = case
    say("products", case, dt)
    product_case(m, n, k, dt, lens, rows=48)
    if m * n < 2 ** 23:
        product_case(m, n, k, dt, lens, rows=48, pad=3, block=128)


@pytest.mark.parametrize("case", [f[0] for f in V.FEW_TOKENS], ids=lambda c: str(c)[:40])
@pytest.mark.parametrize("dt", list(TYPES))
def test_few_tokens(case, dt):
    m, n, k, lens = case
    say("few tokens", case, dt)
    e = len(lens) if lens else 0
    off = offsets_of(lens) if e else None
    ol = off.tolist() if e else None
    d, d1 = (mx.linear_desc(m, n, k, experts=e, block=b) for b in (128, 1))
    x, dy, w = rand(1, m, k, dt=dt), rand(2, m, n, dt=dt), rand(3, max(e, 1), n, k, dt="bf16")
    wq = quantize(d, WEIGHT, (w if e else w[0]).to(DEV))
    xq, dyq = quantize(d1, ACT, x.to(DEV), off=off), quantize(d1, GRAD, dy.to(DEV), off=off)
    ws = workspace(d)
    xv, dyv = R.form_tokens(f64(x), 1, 0, ol), R.form_tokens(f64(dy), 1, 0, ol)
    wv = {i: R.form(f64(w[i]), 128, 0) for i, (a, b) in enumerate(R.segments(m, ol)) if b > a}
    for pad in (0, 3):
        y, dx, ya = (strided(torch.full((m, c), float("nan"), dtype=TYPES[dt]), pad, pad and 1) for c in (n, k, n))
        mx.mx_linear8_fwd(d, wq, xq, y, ws, offsets=off)
        mx.mx_linear8_dgrad(d, wq, dyq, dx, ws, offsets=off)
        mx.mx_linear8_apply(d, wq, x.to(DEV), ya, ws, offsets=off)
        for i, (a, b) in enumerate(R.segments(m, ol)):
            if a == b:
                continue
            for got, p, q, c in ((y, xv, wv[i].T, k), (ya, xv, wv[i].T, k), (dx, dyv, wv[i], n)):
                ref = p[a:b] @ q
                lim = R.bound(c, p[a:b], q, ref, dt)
                err = np.abs(f64(got[a:b]) - ref)
                if dt == "f16":
                    err = np.where(np.abs(ref) + lim > 65519, 0.0, err)
                assert np.all(err <= lim), np.max(err / lim)
        if pad:
            for t in (y, dx, ya):
                assert bool((t.as_strided((m, t.shape[1] + pad), (t.shape[1] + pad, 1))[:-1, t.shape[1]:] == 7.0).all())


@pytest.mark.parametrize("dt,n", [("bf16", 16384), ("bf16", 16391), ("f32", 8192)])
def test_outputs_past_the_caches(dt, n):
    """256 MiB of output and more, rows aligned and not."""
    m, k = 8200, 128
    d, d1 = (mx.linear_desc(m, n, k, block=b) for b in (128, 1))
    x, w = rand(1, m, k, dt=dt), rand(2, n, k, dt=dt)
    y = torch.full((m, n), float("nan"), dtype=TYPES[dt], device=DEV)
    mx.mx_linear8_fwd(d, quantize(d, WEIGHT, w.to(DEV)), quantize(d1, ACT, x.to(DEV)), y, workspace(d))
    assert not bool(torch.isnan(y).any())
    at = np.unique(np.concatenate([np.random.default_rng(1).integers(0, m, 60), [0, m - 1]]))
    xv, wv = R.form(f64(x)[at], 1, 0), R.form(f64(w), 128, 0)
    ref = xv @ wv.T
    assert np.all(np.abs(f64(y[torch.from_numpy(at).to(DEV)]) - ref) <= R.bound(k, xv, wv.T, ref, dt))
