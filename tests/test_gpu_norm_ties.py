"""The norm's 8-bit output is rounded once: products next to a tie of E4M3, or to
the border between two scales, go to the side that the exact product is on."""
import numpy as np
import pytest
import torch

import linear8_ref as R8
import microscaling_quantized_convolution_mx_amd as mx
from gpu_util import say
from test_gpu_linear import f64, rand
from test_gpu_norm import DEV, TYPES, tensor8

pytestmark = pytest.mark.gpu

LD = np.longdouble  # 64 bits of significand here: a product of three is off by 2^-62
assert np.finfo(LD).nmant >= 63


def exact_codes(y, m, k):
    """(code, scale code) of every element of y (longdouble), rounded once."""
    kp = -(-k // 128) * 128
    b = np.pad(y, ((0, 0), (0, kp - k))).reshape(m, kp // 128, 128)
    top = np.abs(b).max(2)
    e = np.frexp(top)[1] - 9
    e = np.maximum(e + (top > np.ldexp(LD(448), e)), -127)
    v = np.ldexp(b, -e[..., None])
    step = np.ldexp(LD(1), np.maximum(np.frexp(np.abs(v))[1] - 1, -6) - 3)
    c = R8.code_bits(np.copysign(np.rint(v / step) * step, v).astype(np.float64))
    return c.reshape(m, kp)[:, :k], (e + 127).astype(np.uint8)


def stored(q, m, k):
    codes, scales = (b.cpu().numpy() for b in q.buffers[0])
    kp = -(-k // 128) * 128
    r, c = np.meshgrid(np.arange(m), np.arange(k), indexing="ij")
    code = codes[((r // 32) * (kp // 64) + c // 64) * 2048 + (c // 32 % 2) * 1024 + (c // 16 % 2) * 512 + (r % 32) * 16 + c % 16]
    r, c = np.meshgrid(np.arange(m), np.arange(kp // 128), indexing="ij")
    return code, scales[(r // 128 * (kp // 128) + c) * 128 + r % 32 * 4 + r // 32 % 4]


def near(k, dt, seed, border):
    """A row, and weights that put its products next to ties: on the nearest fp32 weight and up to two beside it.
    border: the largest product of each block is put next to 448 instead, the border of two scales."""
    g = np.random.default_rng(seed)
    n = g.standard_normal(k)
    t = torch.from_numpy((n + np.copysign(0.1, n)).astype(np.float32)).to(TYPES[dt])
    tl = f64(t).astype(LD)
    r = 1 / np.sqrt((tl * tl).sum() / k)
    col = np.arange(k) % 128
    # midpoints between neighbours from 2^-9 on: the odd multiples of half a step
    ex = g.integers(-6, 8, k)
    tie = np.where(g.random(k) < 0.2, np.ldexp(2.0 * g.integers(0, 8, k) + 1, -10), np.ldexp(2.0 * g.integers(8, 16, k) + 1, ex - 4))
    tie = np.minimum(tie, 432.0)
    tie = np.where(col == 0, 448.0 if border else 440.0, tie) * np.where(g.random(k) < 0.5, 1, -1)
    w = (tie / (tl * r)).astype(np.float32)
    for _ in range(2):
        w = np.where(g.random(k) < 0.4, np.nextafter(w, np.where(g.random(k) < 0.5, np.inf, -np.inf).astype(np.float32)), w)
    return t, w, tl, r


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("k", [128, 300, 512, 1000, 2048, 4100, 9000, 16384, 17000])
def test_products_next_to_ties(k, dt):
    """Every row is the same but for a power of two, which eps = 0 takes out again; 1030 rows take the kernel that writes four together.

    fp64 sums of the squares, a root and two products are off by some (k / 1024 + 30) 2^-53 at most.  Products nearer to
    a tie than that, of which there should be none, are left out."""
    for seed in range(4 if k <= 4100 else 2):
        for border in (False, True):
            say("ties", k, dt, seed, border)
            t, w, tl, r = near(k, dt, seed, border)
            y = tl * r * w.astype(LD)
            code, scale = exact_codes(y[None], 1, k)
            err = LD(2) ** -53 * (k / 1024 + 30) + LD(2) ** -61
            lo, hi = (exact_codes(y[None] * (1 + s * err), 1, k) for s in (-1, 1))
            sure = (lo[0] == hi[0])[0]
            assert sure.mean() > 0.99 and np.array_equal(lo[1], hi[1])
            for m in (3, 1030):
                p = torch.ldexp(t[None].float(), torch.arange(m)[:, None] % 3 - 1).to(TYPES[dt])
                assert np.array_equal(f64(p), np.ldexp(f64(t)[None], np.arange(m)[:, None] % 3 - 1))
                q = tensor8(m, k)
                mx.mx_norm_fwd(mx.norm_desc(m, k, 0.0), p.to(DEV), torch.from_numpy(w).to(DEV), yq=q)
                torch.cuda.synchronize()
                got, s = stored(q, m, k)
                assert np.array_equal(s, np.broadcast_to(scale, s.shape))
                bad = (got != code)[:, sure]
                assert not bad.any(), f"{bad.sum()} of {bad.size}"


def test_subnormal_products():
    """Outputs among fp32's subnormals, whose scale is the smallest: ties are odd multiples of 2^-137, and the products
    2^-160 and less beside them."""
    k = 256
    g = np.random.default_rng(10)
    t = np.ldexp(g.uniform(1, 2, k), -70).astype(np.float32)
    t[::128] = 1.0  # these make rstd, and have a weight of 0
    tl = t.astype(LD)
    r = 1 / np.sqrt((tl * tl).sum() / k)
    tie = np.ldexp(2.0 * g.integers(0, 16, k) + 1, -137)
    w = (tie / (tl * r)).astype(np.float32)
    w[::128] = 0.0
    y = tl * r * w.astype(LD)
    code, scale = exact_codes(y[None], 1, k)
    assert not scale.any()
    lo, hi = (exact_codes(y[None] * (1 + s * LD(2) ** -48), 1, k) for s in (-1, 1))
    sure = (lo[0] == hi[0])[0]
    assert sure.mean() > 0.99
    q = tensor8(1, k)
    mx.mx_norm_fwd(mx.norm_desc(1, k, 0.0), torch.from_numpy(t)[None].to(DEV), torch.from_numpy(w).to(DEV), yq=q)
    got, s = stored(q, 1, k)
    assert not s.any() and np.array_equal(got[:, sure], code[:, sure])
