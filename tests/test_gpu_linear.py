"""Microscaled linear layers on the GPU against a plain 64-bit implementation.

Quantized tensors must agree exactly.  Products are held to the error that
fp32 sums in any order can have on those operands (linear_ref.bound)."""
import numpy as np
import pytest
import torch

import linear_ref as R
import microscaling_quantized_convolution_mx_amd as mx
from gpu_util import say

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACT, WEIGHT, GRAD = mx.MX_ROLE_ACT, mx.MX_ROLE_WEIGHT, mx.MX_ROLE_GRAD


def rand(seed, *shape, dt="f32", spread=2.0):
    """Values over some octaves, with exact zeros among them."""
    g = np.random.default_rng(seed)
    x = g.standard_normal(shape) * np.exp2(g.uniform(-spread, spread, shape))
    x[g.random(shape) < 0.05] = 0.0
    return torch.from_numpy(x.astype(np.float32)).to(TYPES[dt])


def f64(t):
    return t.detach().double().cpu().numpy()


def offsets_of(lens, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int32), device=DEV)


def strided(t, pad, shift=0):
    """t on the device with `pad` more elements between rows, starting `shift` elements into its storage."""
    rows, cols = t.shape[:-1].numel(), t.shape[-1]
    buf = torch.full((rows * (cols + pad) + shift + 64,), 7.0, dtype=t.dtype, device=DEV)
    v = buf[shift:shift + rows * (cols + pad)].view(*t.shape[:-1], cols + pad)[..., :cols]
    v.copy_(t)
    return v


def workspace(d, fill=0xFF):
    return torch.full((max(mx.mx_linear_workspace_bytes(d), 16),), fill, dtype=torch.uint8, device=DEV)


def qtensor(d, role, **kw):
    q = mx.LinearQTensor(d, role, DEV, **kw)
    for f in q.buffers.values():
        for b in f:
            b.fill_(0xFF)  # a scale that the call leaves out would be NaN
    return q


def quantize(d, role, t, rounding=mx.MX_RNE, seed=0, off=None, **kw):
    q = qtensor(d, role, **kw)
    mx.mx_linear_quantize(d, role, t, q, rounding, seed, offsets=off)
    return q


def values(d, role, q, form, like, off=None):
    out = torch.full(like.shape, 99.0, dtype=torch.float32, device=DEV)
    mx.mx_linear_dequantize(d, role, q, out, form, offsets=off)
    return f64(out)


def same(a, b, what=""):
    np.testing.assert_array_equal(a, b, err_msg=what)


# ---------------------------------------------------------------- quantizer

SHAPES = [(1, 1), (1, 33), (5, 32), (31, 64), (32, 31), (33, 96), (127, 129), (128, 128), (129, 257), (300, 500)]


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("block,sr", [(1, False), (1, True), (32, False), (32, True)])
def test_quantize_values(dt, block, sr):
    for i, (m, k) in enumerate(SHAPES):
        say("quantize", dt, block, sr, m, k)
        x = rand(10 + i, m, k, dt=dt)
        seed = 12345678901234567890 if sr else 0
        ref = R.quantize(f64(x), block, R.draws(m, k, seed) if sr else None)[2]
        d = mx.linear_desc(m, 8, k, block=block)
        for t in (x.to(DEV), strided(x, 8), strided(x, 3, 1)):
            q = quantize(d, ACT, t, mx.MX_SR if sr else mx.MX_RNE, seed)
            for form in q.bytes:
                same(values(d, ACT, q, form, x), ref, f"{m}x{k} form {form}")


def test_stored_layout():
    """Codes and scale bytes where the header puts them, padding zero."""
    m, k = 70, 150
    x = rand(3, m, k)
    codes, scale, _ = R.quantize(f64(x), 32)
    d = mx.linear_desc(m, 8, k)
    q = quantize(d, ACT, x.to(DEV))
    mp, kp = 128, 256
    for form, c, s in ((0, codes, scale), (1, codes.T, scale.T)):
        rows, cols = (mp, kp) if form == 0 else (kp, mp)
        want_c, want_s = np.zeros(rows * cols // 2, np.uint8), np.zeros(rows * cols // 32, np.uint8)
        for r in range(c.shape[0]):
            for j in range(c.shape[1]):
                at = ((r // 32) * (cols // 64) + j // 64) * 1024 + (j // 32 % 2) * 512 + (r % 32) * 16 + (j % 32) // 2
                want_c[at] |= c[r, j] << (4 * (j % 2))
                want_s[((r // 128) * (cols // 64) + j // 64) * 256 + (j // 32 % 2) * 128 + (r % 32) * 4 + r // 32 % 4] = s[r, j]
        got_c, got_s = (b.cpu().numpy() for b in q.buffers[form])
        same(got_c, want_c)
        # rows of a 32x32 block past the matrix share its scale: their codes are zero
        for r in range(rows):
            for j in range(0, cols, 32):
                at = ((r // 128) * (cols // 64) + j // 64) * 256 + (j // 32 % 2) * 128 + (r % 32) * 4 + r // 32 % 4
                if r < c.shape[0] and j < c.shape[1]:
                    assert got_s[at] == want_s[at]
                else:
                    assert got_s[at] != 0xFF


@pytest.mark.parametrize("block", [1, 32])
def test_quantize_special_values(block):
    m, k = 96, 96
    x = rand(5, m, k).numpy()
    x[3, 40] = np.nan
    x[40, 3], x[41, 70] = np.inf, -np.inf
    x[64:, :32] = 0.0
    x[64:, 32:64] = np.ldexp(np.float32(1), -149) * np.arange(32)  # subnormal: the scale is clamped at 2^-127
    x[64:, 64:] = np.float32(3e38) * np.linspace(-1, 1, 32, dtype=np.float32)
    x[0, 0] = -0.0
    x = torch.from_numpy(x)
    _, _, ref = R.quantize(f64(x), block)
    d = mx.linear_desc(m, 8, k, block=block)
    q = quantize(d, ACT, x.to(DEV))
    for form in q.bytes:
        got = values(d, ACT, q, form, x)
        same(got, ref)
        same(np.signbit(got[~np.isnan(ref)]), np.signbit(ref[~np.isnan(ref)]))


@pytest.mark.parametrize("dt", list(TYPES))
def test_quantize_ties(dt):
    """Every midpoint of the grid and its neighbours, below each power of two."""
    v = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.5])
    eps = {"f32": 2.0 ** -23, "bf16": 2.0 ** -7, "f16": 2.0 ** -10}[dt]
    row = np.concatenate([v, v * (1 + eps), v * (1 - eps)])
    x = np.zeros((8, 32))
    for i in range(8):
        x[i, :30] = row * (-1) ** i * 2.0 ** (i - 4)
        x[i, 30] = 4.0 * 2.0 ** (i - 4)
    x = torch.from_numpy(x.astype(np.float32)).to(TYPES[dt])
    d = mx.linear_desc(8, 8, 32, block=1)
    q = quantize(d, ACT, x.to(DEV))
    same(values(d, ACT, q, 0, x), R.quantize(f64(x), 1)[2])


def test_quantize_experts_and_weights():
    """Blocks count from each expert's first row; W's experts are matrices of their own."""
    lens = [0, 45, 1, 0, 128, 33, 0]
    m, n, k = sum(lens) + 9, 70, 130  # 4 rows before the first expert, 5 after the last
    off = offsets_of(lens, 4)
    d = mx.linear_desc(m, n, k, experts=len(lens))
    x = rand(7, m, k, dt="bf16")
    q = quantize(d, ACT, x.to(DEV), mx.MX_SR, 99, off=off)
    ref = R.quantize_tokens(f64(x), 32, off.tolist(), R.draws(m, k, 99))
    ref[:4] = ref[m - 5:] = 99.0  # no expert's rows stay as they were
    for form in (0, 1):
        same(values(d, ACT, q, form, x, off), ref, f"form {form}")
    w = rand(8, len(lens), n, k, dt="f16")
    for t in (w.to(DEV), strided(w, 5, 1)):
        q = quantize(d, WEIGHT, t, mx.MX_SR, 98)
        u = R.draws(len(lens) * n, k, 98).reshape(len(lens), n, k)
        ref = np.stack([R.quantize(f64(a), 32, b)[2] for a, b in zip(w, u)])
        for form in (0, 1):
            same(values(d, WEIGHT, q, form, w), ref, f"weights, form {form}")


# ---------------------------------------------------------------- products

def product_case(m, n, k, dt, lens=None, first=0, seed=1, pad=0, spread=2.0):
    """All three products against 64 bits; returns what the GPU gave."""
    e = len(lens) if lens is not None else 0
    off = offsets_of(lens, first) if e else None
    ol = off.tolist() if e else None
    d = mx.linear_desc(m, n, k, experts=e)
    x, dy = rand(seed, m, k, dt=dt, spread=spread), rand(seed + 1, m, n, dt=dt, spread=spread)
    w = rand(seed + 2, max(e, 1), n, k, dt=dt, spread=spread)
    xv, dyv = R.quantize_tokens(f64(x), 32, ol), R.quantize_tokens(f64(dy), 32, ol, R.draws(m, n, 7) if m else None)
    wv = np.stack([R.quantize(f64(a), 32)[2] for a in w])
    xq, wq = quantize(d, ACT, x.to(DEV), off=off), quantize(d, WEIGHT, (w if e else w[0]).to(DEV))
    dyq = quantize(d, GRAD, dy.to(DEV), mx.MX_SR, 7, off=off)
    ws = workspace(d)

    def out(*shape):
        return strided(torch.full(shape, float("nan"), dtype=TYPES[dt]), pad, 1 if pad else 0)
    y, dx, dw = out(m, n), out(m, k), out(*((e, n, k) if e else (n, k)))
    mx.mx_linear_fwd(d, wq, xq, y, ws, offsets=off)
    mx.mx_linear_dgrad(d, wq, dyq, dx, ws, offsets=off)
    mx.mx_linear_wgrad(d, dyq, xq, dw, ws, offsets=off)
    torch.cuda.synchronize()
    gy, gdx, gdw = f64(y), f64(dx), f64(dw).reshape(max(e, 1), n, k)
    for i, (a, b) in enumerate(R.segments(m, ol)):
        for got, p, q, c, what in ((gy[a:b], xv[a:b], wv[i].T, k, "y"), (gdx[a:b], dyv[a:b], wv[i], n, "dx"),
                                   (gdw[i], dyv[a:b].T, xv[a:b], b - a, "dw")):
            ref, mags = p @ q, np.abs(p) @ np.abs(q)
            err, lim = np.abs(got - ref), R.bound(c, mags, ref, dt)
            if dt == "f16":  # sums past the type's largest value are infinite
                over = np.abs(ref) + R.bound(c, mags, ref, "f32") > 65519
                err = np.where(over, 0.0, err)
            assert np.all(err <= lim), f"{what} of {i}: {np.max(err / lim)} of the bound at {np.argmax(err / lim)}"
    if e:  # rows of no expert are left as they were
        assert np.isnan(gy[:first]).all() and np.isnan(gy[first + sum(lens):]).all()
        assert np.isnan(gdx[:first]).all() and np.isnan(gdx[first + sum(lens):]).all()
    if pad:  # nor does anything land between the rows
        for t in (y, dx, dw):
            full = t.as_strided((t.shape[:-1].numel(), t.shape[-1] + pad), (t.shape[-1] + pad, 1))
            assert bool((full[:-1, t.shape[-1]:] == 7.0).all())
    return y, dx, dw


@pytest.mark.parametrize("m,n,k", [
    (1, 1, 1), (1, 130, 70), (31, 32, 33), (33, 65, 127), (64, 128, 256), (127, 129, 128), (129, 127, 385), (260, 300, 200),
    (5, 40, 2000), (40, 2000, 5), (2000, 40, 5), (3, 17, 5000)])
@pytest.mark.parametrize("dt", list(TYPES))
def test_products(m, n, k, dt):
    say("products", m, n, k, dt)
    product_case(m, n, k, dt)


@pytest.mark.parametrize("m,n,k", [(33, 65, 127), (260, 300, 200)])
@pytest.mark.parametrize("dt", list(TYPES))
def test_products_strided(m, n, k, dt):
    product_case(m, n, k, dt, pad=5)
    product_case(m, n, k, dt, pad=8)


@pytest.mark.parametrize("m,n,k", [(4100, 4200, 300), (300, 4100, 4200), (4200, 300, 4100)])
def test_products_large_tiles(m, n, k):
    """Enough output tiles for the largest ones, ragged at both edges, with few
    steps, an odd number of them and many."""
    product_case(m, n, k, "bf16")


@pytest.mark.parametrize("lens,first,rest", [
    ([5], 0, 0), ([0, 0, 3], 0, 0), ([1, 1, 1, 1], 0, 0), ([0, 200, 0, 1, 129, 0], 3, 4), ([128, 256, 127], 0, 0),
    ([0, 0, 0], 0, 0), ([0, 0], 2, 1), ([300] + [0] * 70 + [2, 40] + [0] * 60 + [7], 0, 1)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_experts(lens, first, rest, dt):
    say("experts", lens[:8], first, rest, dt)
    product_case(first + sum(lens) + rest, 70, 200, dt, lens, first)


def test_experts_large():
    product_case(3000, 520, 700, "bf16", [0, 1500, 3, 900, 0, 597], 0)


@pytest.mark.parametrize("e", [0, 3])
def test_no_tokens(e):
    """dW is zero; Y and dX have no element to touch."""
    product_case(0, 70, 200, "f32", [0] * e if e else None)
    d = mx.linear_desc(0, 70, 200, experts=e)
    off = offsets_of([0] * e) if e else None
    wq = quantize(d, WEIGHT, rand(1, *((e,) if e else ()), 70, 200).to(DEV))
    y = torch.empty(0, 70, device=DEV)
    mx.mx_linear_apply(d, wq, torch.empty(0, 200, device=DEV), y, offsets=off)
    torch.cuda.synchronize()


def test_offsets_out_of_order():
    """Offsets that decrease or leave the range count as their running maximum
    clamped to it, so such a call stays within the buffers."""
    m, n, k = 100, 64, 96
    bad = torch.tensor([-5, 40, 20, 2 ** 31 - 1, -2 ** 31, 60], dtype=torch.int32, device=DEV)
    good = torch.tensor([0, 40, 40, 100, 100, 100], dtype=torch.int32, device=DEV)
    d = mx.linear_desc(m, n, k, experts=5)
    x, w, dy = rand(1, m, k).to(DEV), rand(2, 5, n, k).to(DEV), rand(3, m, n).to(DEV)
    wq = quantize(d, WEIGHT, w)
    got = []
    for off in (bad, good):
        xq, dyq = quantize(d, ACT, x, off=off), quantize(d, GRAD, dy, off=off)
        y, dx, dw, ya = torch.zeros_like(dy), torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(dy)
        ws = workspace(d)
        mx.mx_linear_fwd(d, wq, xq, y, ws, offsets=off)
        mx.mx_linear_dgrad(d, wq, dyq, dx, ws, offsets=off)
        mx.mx_linear_wgrad(d, dyq, xq, dw, ws, offsets=off)
        mx.mx_linear_apply(d, wq, x, ya, ws, offsets=off)
        got.append((y, dx, dw, ya))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_non_finite_operands():
    """A NaN or Inf makes NaN of every output that its block enters, and of no other."""
    m, n, k = 70, 80, 300
    x, w, dy = rand(1, m, k), rand(2, n, k), rand(3, m, n)
    x[35, 290] = float("inf")   # the last block of the odd step
    w[3, 5] = float("nan")
    d = mx.linear_desc(m, n, k)
    xq, wq, dyq = quantize(d, ACT, x.to(DEV)), quantize(d, WEIGHT, w.to(DEV)), quantize(d, GRAD, dy.to(DEV))
    ws = workspace(d)
    y, dx, dw = torch.zeros(m, n, device=DEV), torch.zeros(m, k, device=DEV), torch.zeros(n, k, device=DEV)
    mx.mx_linear_fwd(d, wq, xq, y, ws)
    mx.mx_linear_dgrad(d, wq, dyq, dx, ws)
    mx.mx_linear_wgrad(d, dyq, xq, dw, ws)
    ny, nx, nw = (np.isnan(f64(t)) for t in (y, dx, dw))
    want = np.zeros((m, n), bool)
    want[32:64] = True
    want[:, :32] = True
    same(ny, want)
    want = np.zeros((m, k), bool)
    want[:, :32] = True
    same(nx, want)
    want = np.zeros((n, k), bool)
    want[:, 288:] = True
    same(nw, want)


@pytest.mark.parametrize("ex,ew", [(100, -100), (-120, 100), (-60, -60), (60, 60)])
def test_far_scales(ex, ew):
    """Scales far from 1 on either side of a product whose result is in range."""
    m, n, k = 40, 50, 100
    x, w = rand(1, m, k) * 2.0 ** ex, rand(2, n, k) * 2.0 ** ew
    d = mx.linear_desc(m, n, k)
    xq, wq = quantize(d, ACT, x.to(DEV)), quantize(d, WEIGHT, w.to(DEV))
    y = torch.zeros(m, n, device=DEV)
    mx.mx_linear_fwd(d, wq, xq, y, workspace(d))
    xv, wv = R.quantize(f64(x), 32)[2], R.quantize(f64(w), 32)[2]
    ref, mags = xv @ wv.T, np.abs(xv) @ np.abs(wv.T)
    assert np.all(np.abs(f64(y) - ref) <= R.bound(k, mags, ref, "f32"))


def test_gradients_are_differences():
    """The layer is linear in its quantized operands: where a step to the next
    grid value leaves the block's scale alone, the difference quotient of
    <dY, Y> is the gradient.  All numbers are small integers over a power of
    two, so sums are exact and the quotients too."""
    m, n, k = 40, 35, 50
    g = np.random.default_rng(5)
    x, w, dy = (g.choice([-1.0, -0.5, 0.0, 0.5, 1.0], s) for s in ((m, k), (n, k), (m, n)))
    for a in (x, w, dy):
        for i in range(0, a.shape[0], 32):
            for j in range(0, a.shape[1], 32):
                a[i, j] = 4.0  # fixes the block's scale at 1
    d = mx.linear_desc(m, n, k)
    ws = workspace(d)

    def t(a):
        return torch.from_numpy(a.astype(np.float32)).to(DEV)

    def loss(x, w):
        y = torch.empty(m, n, device=DEV)
        mx.mx_linear_fwd(d, quantize(d, WEIGHT, t(w)), quantize(d, ACT, t(x)), y, ws)
        return float((f64(y) * dy).sum())
    dyq, xq, wq = quantize(d, GRAD, t(dy)), quantize(d, ACT, t(x)), quantize(d, WEIGHT, t(w))
    dx, dw = torch.empty(m, k, device=DEV), torch.empty(n, k, device=DEV)
    mx.mx_linear_dgrad(d, wq, dyq, dx, ws)
    mx.mx_linear_wgrad(d, dyq, xq, dw, ws)
    same(f64(dx), dy @ w)
    same(f64(dw), dy.T @ x)
    at = loss(x, w)
    for i, j in ((1, 1), (33, 49), (39, 2), (31, 31)):
        x2 = x.copy()
        x2[i, j] += 0.5
        assert (loss(x2, w) - at) / 0.5 == f64(dx)[i, j]
    for i, j in ((1, 1), (34, 49), (33, 2)):
        w2 = w.copy()
        w2[i, j] -= 0.5
        assert (loss(x, w2) - at) / -0.5 == f64(dw)[i, j]


# ---------------------------------------------------------------- serving

@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 70, 4000), (2, 33, 64), (7, 129, 65), (16, 40, 100), (17, 64, 1000), (31, 300, 130),
                                   (32, 65, 4100), (33, 128, 200), (64, 500, 300), (200, 100, 150), (3, 40, 200000)])
def test_apply(m, n, k, dt):
    """The values of quantize and fwd, whichever way the call takes."""
    say("apply", m, n, k, dt)
    x, w = rand(m, m, k, dt=dt), rand(n, n, k, dt="bf16")
    one = mx.linear_desc(m, n, k, block=1)
    xv, wv = R.quantize(f64(x), 1)[2], R.quantize(f64(w), 32)[2]
    ref, mags = xv @ wv.T, np.abs(xv) @ np.abs(wv.T)
    d = mx.linear_desc(m, n, k)
    wq = quantize(d, WEIGHT, w.to(DEV), cols=False)
    for tx, pad in ((x.to(DEV), 0), (strided(x, 8), 8), (strided(x, 3, 1), 3)):
        y = strided(torch.full((m, n), float("nan"), dtype=TYPES[dt]), pad, 1 if pad == 3 else 0)
        mx.mx_linear_apply(d, wq, tx, y, workspace(d))
        assert np.all(np.abs(f64(y) - ref) <= R.bound(k, mags, ref, dt))
        if pad:
            assert bool((y.as_strided((m, n + pad), (n + pad, 1))[:-1, n:] == 7.0).all())
    # a token's output does not depend on the others
    if m > 1:
        d1 = mx.linear_desc(1, n, k)
        y1 = torch.empty(1, n, dtype=torch.float32, device=DEV)
        mx.mx_linear_apply(d1, wq, x[m - 1:].to(DEV), y1, workspace(d1))
        assert np.all(np.abs(f64(y1) - ref[m - 1:]) <= R.bound(k, mags[m - 1:], ref[m - 1:], "f32"))
    # the weight in 1x32 blocks goes the same way
    wq = quantize(one, WEIGHT, w.to(DEV))
    wv = R.quantize(f64(w), 1)[2]
    y = torch.empty(m, n, dtype=torch.float32, device=DEV)
    mx.mx_linear_apply(one, wq, x.to(DEV), y, workspace(one))
    ref, mags = xv @ wv.T, np.abs(xv) @ np.abs(wv.T)
    assert np.all(np.abs(f64(y) - ref) <= R.bound(k, mags, ref, "f32"))


@pytest.mark.parametrize("lens,first,rest", [
    ([1, 0, 1, 2], 0, 0), ([0, 0, 0, 9], 0, 0), ([40, 0, 1, 0, 0, 0, 0, 0], 2, 1), ([0, 0], 0, 3), ([70, 90], 0, 0),
    ([0] * 66 + [3, 1] + [0] * 60 + [5], 0, 0), ([33, 1, 64, 0, 5] + [0] * 10, 1, 0)])
def test_apply_experts(lens, first, rest):
    say("apply experts", lens[:8], first, rest)
    m, n, k, e = first + sum(lens) + rest, 70, 300, len(lens)
    off = offsets_of(lens, first)
    d = mx.linear_desc(m, n, k, experts=e)
    x, w = rand(1, m, k, dt="bf16"), rand(2, e, n, k, dt="bf16")
    wq = quantize(d, WEIGHT, w.to(DEV), cols=False)
    y = torch.full((m, n), float("nan"), dtype=torch.float32, device=DEV)
    mx.mx_linear_apply(d, wq, x.to(DEV), y, workspace(d), offsets=off)
    got, xv = f64(y), R.quantize(f64(x), 1)[2]
    for i, (a, b) in enumerate(R.segments(m, off.tolist())):
        wv = R.quantize(f64(w[i]), 32)[2]
        ref, mags = xv[a:b] @ wv.T, np.abs(xv[a:b]) @ np.abs(wv.T)
        assert np.all(np.abs(got[a:b] - ref) <= R.bound(k, mags, ref, "f32"))
    assert np.isnan(got[:first]).all() and np.isnan(got[first + sum(lens):]).all()


@pytest.mark.parametrize("m", [3, 200])
def test_apply_non_finite(m):
    n, k = 70, 200
    x, w = rand(1, m, k), rand(2, n, k)
    x[1, 150], x[2, 3], w[40, 7] = float("nan"), float("-inf"), float("inf")
    d = mx.linear_desc(m, n, k)
    y = torch.zeros(m, n, device=DEV)
    mx.mx_linear_apply(d, quantize(d, WEIGHT, w.to(DEV)), x.to(DEV), y, workspace(d))
    want = np.zeros((m, n), bool)
    want[1:3] = True
    want[:, 32:64] = True
    same(np.isnan(f64(y)), want)


# ---------------------------------------------------------------- repeatability, graphs, streams

def test_results_repeat_bit_for_bit():
    m, n, k = 300, 400, 3000
    d = mx.linear_desc(m, n, k)
    x, w, dy = rand(1, m, k, dt="bf16").to(DEV), rand(2, n, k, dt="bf16").to(DEV), rand(3, m, n, dt="bf16").to(DEV)
    xq, wq, dyq = quantize(d, ACT, x), quantize(d, WEIGHT, w), quantize(d, GRAD, dy, mx.MX_SR, 4)
    first = None
    for _ in range(4):
        y, dx, dw = torch.empty(m, n, device=DEV), torch.empty(m, k, device=DEV), torch.empty(n, k, device=DEV)
        ws = workspace(d)
        mx.mx_linear_fwd(d, wq, xq, y, ws)
        mx.mx_linear_dgrad(d, wq, dyq, dx, ws)
        mx.mx_linear_wgrad(d, dyq, xq, dw, ws)
        got = [t.view(torch.int32).clone() for t in (y, dx, dw)]
        first = first or got
        for a, b in zip(got, first):
            assert torch.equal(a, b)


def test_graph_and_stream():
    """A captured step, replayed on changing inputs with eager work between, equals the eager one."""
    m, n, k, e = 90, 130, 260, 4
    off = offsets_of([20, 0, 69, 1])
    d = mx.linear_desc(m, n, k, experts=e)
    x, w, dy = rand(1, m, k).to(DEV), rand(2, e, n, k).to(DEV), rand(3, m, n).to(DEV)
    xq, wq, dyq = (mx.LinearQTensor(d, r) for r in (ACT, WEIGHT, GRAD))
    out = [torch.empty(m, n, device=DEV), torch.empty(m, k, device=DEV), torch.empty(e, n, k, device=DEV),
           torch.empty(e, n, k, device=DEV), torch.empty(1, device=DEV), torch.empty(m, n, device=DEV)]
    ws = workspace(d)
    grads = mx.GradList([out[2]], [out[3]])
    gws = torch.empty(mx.mx_grad_workspace_bytes(grads), dtype=torch.uint8, device=DEV)

    def step():
        mx.mx_linear_quantize(d, ACT, x, xq, offsets=off)
        mx.mx_linear_quantize(d, WEIGHT, w, wq)
        mx.mx_linear_fwd(d, wq, xq, out[0], ws, offsets=off)
        mx.mx_linear_quantize(d, GRAD, dy, dyq, mx.MX_SR, 11, offsets=off)
        mx.mx_linear_dgrad(d, wq, dyq, out[1], ws, offsets=off)
        mx.mx_linear_wgrad(d, dyq, xq, out[2], ws, offsets=off)
        mx.mx_grad_clip(grads, 1.0, out[4], gws)
        mx.mx_linear_apply(d, wq, x, out[5], ws, offsets=off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(rand(20 + i, m, k))
        dy.copy_(rand(30 + i, m, n))
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for t in out:
            t.fill_(float("nan"))
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, out):
            assert torch.equal(a, b) and not bool(torch.isnan(a).any())


# ---------------------------------------------------------------- sizes that take the larger tiles

def sampled_case(m, n, k, dt, lens=None, seed=1, rows=96, fwd=True, dgrad=True, wgrad=True):
    """The products on rows (of y, dx and dw) drawn at random, the first and the last among them."""
    e = len(lens) if lens is not None else 0
    off = offsets_of(lens) if e else None
    segs = R.segments(m, off.tolist() if e else None)
    d = mx.linear_desc(m, n, k, experts=e)
    g = np.random.default_rng(seed)
    x, dy, w = rand(seed, m, k, dt=dt), rand(seed + 1, m, n, dt=dt), rand(seed + 2, max(e, 1), n, k, dt=dt)
    ws = workspace(d)
    wq = quantize(d, WEIGHT, (w if e else w[0]).to(DEV))
    xq = quantize(d, ACT, x.to(DEV), off=off)
    xv, wv = R.quantize_tokens(f64(x), 32, off.tolist() if e else None), [R.quantize(f64(a), 32)[2] for a in w]
    pick = np.unique(np.concatenate([g.integers(0, m, rows), [0, m - 1]]))

    def check(got, p, q, c, what):
        ref, mags = p @ q, np.abs(p) @ np.abs(q)
        assert np.all(np.abs(got - ref) <= R.bound(c, mags, ref, dt)), what

    def rows_of(t, i):
        return f64(t[torch.from_numpy(i).to(DEV)])
    if fwd:
        y = torch.full((m, n), float("nan"), dtype=TYPES[dt], device=DEV)
        mx.mx_linear_fwd(d, wq, xq, y, ws, offsets=off)
        assert not bool(torch.isnan(y).any())
        for i, (a, b) in enumerate(segs):
            at = pick[(pick >= a) & (pick < b)]
            check(rows_of(y, at), xv[at], wv[i].T, k, f"y of {i}")
        del y
    if not (dgrad or wgrad):
        return
    dyq = quantize(d, GRAD, dy.to(DEV), off=off)
    dyv = R.quantize_tokens(f64(dy), 32, off.tolist() if e else None)
    if dgrad:
        dx = torch.full((m, k), float("nan"), dtype=TYPES[dt], device=DEV)
        mx.mx_linear_dgrad(d, wq, dyq, dx, ws, offsets=off)
        assert not bool(torch.isnan(dx).any())
        for i, (a, b) in enumerate(segs):
            at = pick[(pick >= a) & (pick < b)]
            check(rows_of(dx, at), dyv[at], wv[i], n, f"dx of {i}")
    if wgrad:
        dw = torch.full((max(e, 1), n, k), float("nan"), dtype=TYPES[dt], device=DEV)
        mx.mx_linear_wgrad(d, dyq, xq, dw if e else dw[0], ws, offsets=off)
        assert not bool(torch.isnan(dw).any())
        at = np.unique(np.concatenate([g.integers(0, n, rows), [0, n - 1]]))
        for i, (a, b) in enumerate(segs):
            check(rows_of(dw[i], at), dyv[a:b, at].T, xv[a:b], b - a, f"dw of {i}")


@pytest.mark.parametrize("m,n,k,dt", [
    (1100, 4000, 1000, "bf16"), (1100, 4001, 1000, "f32"),     # 128x128 tiles
    (4100, 4200, 2100, "bf16"), (4099, 4201, 2051, "f16"),     # 256x256 tiles, ragged at both edges, an odd number of steps
    (4300, 4100, 2304, "f32"), (100, 200, 9000, "bf16")])      # and a split contraction
def test_products_by_every_tile(m, n, k, dt):
    say("sampled", m, n, k, dt)
    sampled_case(m, n, k, dt)


@pytest.mark.parametrize("lens,n,k", [([2000, 1500, 0, 600], 2048, 2048), ([3000, 1, 0, 2500, 500], 2304, 2304),
                                      ([300] * 7, 1000, 1100)])
def test_experts_by_every_tile(lens, n, k):
    say("sampled experts", lens, n, k)
    sampled_case(sum(lens), n, k, "bf16", lens)


@pytest.mark.parametrize("n", [16384, 16391])
def test_outputs_past_the_caches(n):
    """256 MiB of output and more, rows aligned and not."""
    sampled_case(8200, n, 128, "bf16", dgrad=False, wgrad=False)


def test_matrices_past_32_bits():
    """More than 2^32 elements: codes, draws and products at the far end."""
    m, k, n = 40000, 110016, 64
    d = mx.linear_desc(m, n, k)
    x = torch.empty(m, k, dtype=torch.bfloat16, device=DEV)
    tail = rand(1, 96, k, dt="bf16")
    for a in range(0, m, 8000):
        x[a:a + 8000] = torch.randn(min(8000, m - a), k, device=DEV, dtype=torch.bfloat16)
    x[m - 96:] = tail.to(DEV)
    w = rand(2, n, k, dt="bf16")
    wv = R.quantize(f64(w), 32)[2]
    first = (m - 96) * k  # index of the tail's first element
    i = np.arange(96 * k, dtype=np.uint64) + np.uint64(first)
    with np.errstate(over="ignore"):
        z = np.uint64(77) ^ (np.uint64(0x9E3779B97F4A7C15) * (i // np.uint64(2) + np.uint64(1)))
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        z ^= z >> np.uint64(31)
    u = (np.where(i & np.uint64(1), z >> np.uint64(16), z >> np.uint64(40)) & np.uint64(0xFFFFFF)) / 2.0 ** 24
    tv = R.quantize(f64(tail), 32, u.reshape(96, k))[2]
    q = quantize(d, ACT, x, mx.MX_SR, 77)
    for form in (0, 1):
        mx.mx_linear_dequantize(d, ACT, q, x, form)
        same(f64(x[m - 96:]), tv, f"form {form}")
    y = torch.empty(m, n, device=DEV)
    mx.mx_linear_fwd(d, quantize(d, WEIGHT, w.to(DEV)), q, y, workspace(d))
    ref, mags = tv @ wv.T, np.abs(tv) @ np.abs(wv.T)
    assert np.all(np.abs(f64(y[m - 96:]) - ref) <= R.bound(k, mags, ref, "f32"))
