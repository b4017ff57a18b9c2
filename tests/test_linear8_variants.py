"""The rules that choose the kernels of the layers in 8 bits, held to the cases
that the GPU tests reach every kernel with (no GPU)."""
import pytest

import linear8_variants as V
import microscaling_quantized_convolution_mx_amd as mx


def desc(m, n, k, lens):
    return mx.linear_desc(m, n, k, experts=len(lens) if lens else 0, block=128)


@pytest.mark.parametrize("case,narrow,wide", V.PRODUCTS, ids=lambda c: str(c)[:40])
def test_products(case, narrow, wide):
    d = desc(*case)
    for dtype, wanted in ((mx.MX_BF16, narrow), (mx.MX_F16, narrow), (mx.MX_F32, wide)):
        for call, (size, split) in zip((V.FWD, V.DGRAD, V.WGRAD), wanted):
            v = V.variant(d, call, dtype)
            assert (v.kernel, v.size, v.splits > 1) == (V.PRODUCT, size, split)
            assert v.threads == (512 if size == 64 and dtype == mx.MX_F32 else 256) and v.workgroups % 8 == 0 and v.workgroups > 0


def test_every_tile_is_reached_by_every_product():
    for k, wide in ((1, False), (2, True)):
        for op in range(3):
            assert {p[k][op] for p in V.PRODUCTS} >= {(64, False), (64, True), (128, False), (256, False)}, (op, wide)
        with_experts = [p for p in V.PRODUCTS if p[0][3]]
        for op in range(3):
            assert {p[k][op][0] for p in with_experts} == {64, 128, 256}, (op, wide)


@pytest.mark.parametrize("case,fwd,dgrad,apply", V.FEW_TOKENS, ids=lambda c: str(c)[:40])
def test_few_tokens(case, fwd, dgrad, apply):
    d = desc(*case)
    for call, size in ((V.FWD, fwd), (V.DGRAD, dgrad)):
        for dtype in (mx.MX_F32, mx.MX_BF16):
            v = V.variant(d, call, dtype)
            assert (v.kernel, v.size) == (V.FEW, size)
    v = V.variant(d, V.APPLY, mx.MX_BF16)
    assert (v.kernel, v.size) == (V.FUSED if apply[1] else V.FEW, apply[0])


def test_the_workspace_serves_both_types():
    """mx_linear8_workspace_bytes covers a split product whichever type its output has."""
    for m, n, k in ((256, 1024, 4096), (203, 130, 4100), (100, 200, 9000)):
        d = desc(m, n, k, None)
        need = mx.mx_linear8_workspace_bytes(d)
        for dtype in (mx.MX_F32, mx.MX_BF16):
            v = V.variant(d, V.FWD, dtype)
            if v.splits > 1:
                assert need >= 4 * v.splits * m * n


def test_no_tokens():
    d = mx.linear_desc(0, 100, 200, block=128)
    assert V.variant(d, V.FWD, 0).kernel == V.NONE and V.variant(d, V.WGRAD, 0).kernel == V.PRODUCT


@pytest.mark.parametrize("m,e,k,n", [(1, 0, 2 ** 28, 64), (2 ** 28, 0, 64, 64), (5, 1024, 2 ** 17, 64), (2 ** 24, 1024, 64, 64), (0, 0, 2 ** 16, 2 ** 20)])
def test_launches_fit(m, e, k, n):
    """Far sizes that a descriptor may have: every launch within 2^32 threads."""
    d = mx.linear_desc(m, n, k, experts=e, block=128)
    assert mx.mx_linear8_code_bytes(d, mx.MX_ROLE_WEIGHT) > 0
    for call in (V.FWD, V.DGRAD, V.WGRAD):
        for dtype in (mx.MX_F32, mx.MX_BF16):
            v = V.variant(d, call, dtype)
            assert v.workgroups * v.threads < 2 ** 32
