"""What the products in 8 bits sum to where single groups of 8 products show:
cut as linear8_sums has it for 16-bit outputs of many tokens, exact for fp32
outputs and few tokens."""
import numpy as np
import pytest
import torch

import linear8_sums as S
import microscaling_quantized_convolution_mx_amd as mx
from gpu_util import say
from test_gpu_linear import f64
from test_linear8_sums import codes

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def operands(m, n, k, subnormals, seed):
    """Codes of x and w, k a multiple of 128.  The last two columns of each 128 hold 448 in one of them and 0 in the other: scales
    are 1 and that product is nothing.  A row of x has one group of 8 besides."""
    g = np.random.default_rng(seed)
    x, w = codes(g, (m, k), subnormals), codes(g, (n, k), subnormals)
    c = np.arange(k)
    x[(c // 8)[None, :] != np.arange(m)[:, None] % (k // 8)] = 0
    x[:, c % 128 >= 126] = w[:, c % 128 >= 126] = 0
    x[:, c % 128 == 126] = w[:, c % 128 == 127] = 0x7E
    return S.values(x), S.values(w)


def products(x, w, dt, block, scale):
    """X W^T of values that both quantize to themselves, w times 2^scale."""
    m, n, k = len(x), len(w), x.shape[1]
    d, d1 = mx.linear_desc(m, n, k, block=block), mx.linear_desc(m, n, k, block=1)
    xq, wq = mx.Linear8QTensor(d1, mx.MX_ROLE_ACT, DEV), mx.Linear8QTensor(d, mx.MX_ROLE_WEIGHT, DEV)
    xt, wt = (torch.from_numpy(v.astype(np.float32)).to(DEV) for v in (x, np.ldexp(w, scale)))
    mx.mx_linear8_quantize(d1, mx.MX_ROLE_ACT, xt, xq)
    mx.mx_linear8_quantize(d, mx.MX_ROLE_WEIGHT, wt, wq)
    for q, role, t in ((xq, mx.MX_ROLE_ACT, xt), (wq, mx.MX_ROLE_WEIGHT, wt)):
        back = torch.empty_like(t)
        mx.mx_linear8_dequantize(d, role, q, back)
        assert torch.equal(back, t)
    y = torch.full((m, n), float("nan"), dtype=TYPES[dt], device=DEV)
    ws = torch.empty(max(16, mx.mx_linear8_workspace_bytes(d)), dtype=torch.uint8, device=DEV)
    mx.mx_linear8_fwd(d, wq, xq, y, ws)
    torch.cuda.synchronize()
    return f64(y)


def rounded(v, dt):
    return f64(torch.from_numpy(v).to(TYPES[dt]))


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("subnormals", [0.0, 0.4, 0.8])
@pytest.mark.parametrize("m", [20, 200, 2100])
def test_single_groups(m, subnormals, block):
    """One group a row is one sum of at most 8 products, which fp32 holds as it is cut: 16-bit outputs are its rounding.  fp32 outputs and
    few tokens' are the exact sum's, of products added in fp32 in any order."""
    n, k = 90, 256
    x, w = operands(m, n, k, subnormals, 7)
    cut, exact, mags = S.groups(x, w)
    cut, exact, mags = cut.sum(2), exact.sum(2), mags.sum(2)  # (one of them is not 0)
    differ = 0
    for dt in TYPES:
        say("groups", m, subnormals, block, dt)
        y = np.ldexp(products(x, w, dt, block, -10), 10)
        want = cut if dt != "f32" and m > 32 else exact
        step = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dt]
        tiny = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25 * 2.0 ** 10}[dt]
        if want is cut:
            assert np.array_equal(cut, cut.astype(np.float32))
            assert np.array_equal(y, np.ldexp(rounded(np.ldexp(cut, -10), dt), 10))
            differ += int((cut != exact).sum())
            assert np.all(np.abs(y - exact) <= (S.MOST * mags + step * np.abs(exact)) * (1 + step) + tiny)
        else:
            # eight products and the zeros beside them, which add nothing
            assert np.all(np.abs(y - exact) <= (8 * 2.0 ** -24 * mags + step * np.abs(exact)) * (1 + step) * 1.01 + tiny)
    if m > 32 and subnormals < 0.5:
        assert differ > 1000
