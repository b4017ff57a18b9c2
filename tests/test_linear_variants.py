"""Which kernel a call takes (on the host): the cases of the GPU tests reach
every variant of the products and of the few-token kernel."""
import pytest

import linear_variants as V
import microscaling_quantized_convolution_mx_amd as mx
from linear_variants import variant


def describe(c):
    m, n, k, lens = c
    assert lens is None or sum(lens) == m
    return mx.linear_desc(m, n, k, experts=len(lens or ()))


@pytest.mark.parametrize("case", V.PRODUCTS, ids=lambda c: f"{c[0][:3]}")
def test_products_take_the_tile_that_the_case_is_for(case):
    d = describe(case[0])
    for call, want in enumerate(case[1:]):
        v = variant(d, call)
        assert (v.kernel, v.size, v.splits > 1) == (V.PRODUCT, *want), call
        assert mx.mx_linear_workspace_bytes(d) > 0 or v.splits == 1


@pytest.mark.parametrize("case", V.FEW_TOKENS, ids=lambda c: f"{c[0][:3]}")
def test_few_tokens_take_the_stripes_that_the_case_is_for(case):
    d = describe(case[0])
    for call, want in ((V.FWD, case[1]), (V.DGRAD, case[2])):
        v = variant(d, call)
        assert (v.kernel, v.size) == (V.FEW, want), call
    v = variant(d, V.APPLY)
    assert (v.size, v.kernel) == (case[3][0], V.FUSED if case[3][1] else V.FEW)


def test_the_cases_reach_every_variant():
    product = {(call, *w, c[0][3] is not None) for c in V.PRODUCTS for call, w in enumerate(c[1:])}
    for call in (V.FWD, V.DGRAD, V.WGRAD):
        for size in (64, 128, 256):
            assert (call, size, False, False) in product and (call, size, False, True) in product
        assert (call, 64, True, False) in product
    for experts in (False, True):
        few = [c for c in V.FEW_TOKENS if (c[0][3] is not None) == experts]
        for stripes in (2, 4) if experts else (1, 2, 4):
            assert any(stripes in c[1:3] for c in few)
            assert any(c[3] == (stripes, True) for c in few)


def test_no_tokens():
    d = mx.linear_desc(0, 70, 200)
    assert [variant(d, c).kernel for c in (V.FWD, V.DGRAD, V.WGRAD, V.APPLY)] == [V.NONE, V.NONE, V.PRODUCT, V.NONE]


@pytest.mark.parametrize("call,shape", [(V.FWD, (203, 130, 4100)), (V.DGRAD, (203, 4100, 130)), (V.WGRAD, (4097, 65, 67))])
def test_every_split_product_refuses_a_short_workspace(call, shape):
    m, n, k = shape
    d = mx.linear_desc(m, n, k)
    v = variant(d, call)
    rows, cols = ((m, n), (m, k), (n, k))[call]
    need = v.splits * rows * ((cols + 3) // 4 * 4) * 4
    q = mx.mx_linear_qtensor(*(0x10000,) * 4)
    f = getattr(mx.lib(), ("mx_linear_fwd", "mx_linear_dgrad", "mx_linear_wgrad")[call])
    for ws, n_bytes in ((None, need), (0x10000, need - 1), (0x10000, 0)):
        assert f(d, q, q, 0x10000, 0, cols, None, ws, n_bytes, None) == -6
    assert mx.mx_linear_workspace_bytes(d) >= need


@pytest.mark.parametrize("shape", [
    (0, 8192, 8192, 1024), (1, 8192, 8192, 1024), (2 ** 20, 8192, 8192, 1024), (0, 2 ** 18, 2 ** 18, 0), (33, 2 ** 18, 2 ** 18, 0),
    (2 ** 30 - 200, 100, 100, 0), (2 ** 30 - 2 ** 18, 100, 100, 1024), (2 ** 23, 16000, 16000, 0), (2, 2 ** 30 - 200, 100, 0),
    (2, 100, 2 ** 30 - 200, 0), (16384, 2 ** 19, 100, 1023), (100, 1, 2 ** 19, 1023)])
def test_every_launch_fits_the_threads_of_one(shape):
    """2^32 - 1 threads, also where the contraction is empty and the output large."""
    m, n, k, e = shape
    d = mx.linear_desc(m, n, k, experts=e)
    for call in (V.FWD, V.DGRAD, V.WGRAD, V.APPLY):
        v = variant(d, call)
        assert v.workgroups * v.threads < 2 ** 32, (call, v)


@pytest.mark.parametrize("m,n,k,e", [(1024, 2048, 2048, 64), (16384, 512, 512, 1024), (301, 300, 260, 40), (16, 2048, 1024, 64)])
def test_few_tokens_of_one_expert_are_not_walked_one_after_the_other(m, n, k, e):
    """Whatever the routing, each 32 tokens of an expert and each group of its weight's stripes have a workgroup."""
    d = mx.linear_desc(m, n, k, experts=e)
    for call, lines in ((V.FWD, n), (V.DGRAD, k), (V.APPLY, n)):
        v = variant(d, call)
        assert v.kernel in (V.FEW, V.FUSED)
        stripes = (lines + 31) // 32
        for used in (1, min(m, e)):
            passes = used - 1 + (m - used + 1 + 31) // 32
            assert v.workgroups >= passes * ((stripes + v.size - 1) // v.size)


@pytest.mark.parametrize("m,n,k,e,fused", [
    (32, 8192, 2048, 0, False), (31, 8192, 2048, 0, True),             # 256 groups of one stripe
    (32, 8191, 2048, 0, False), (32, 8160, 2048, 0, True),             # 256 and 255
    (31, 16400, 1024, 0, True), (31, 16385, 1920, 0, True), (32, 16352, 2048, 0, False),  # 257, 257 and 256 of two
    (1023, 2048, 1024, 64, True), (1024, 2048, 1024, 64, False)])      # 16 groups of four in each expert
def test_tokens_are_quantized_on_the_way_below_2_24_elements(m, n, k, e, fused):
    """Tokens x padded features x groups of stripes of one expert, those that the launch has."""
    v = variant(mx.linear_desc(m, n, k, experts=e), V.APPLY)
    assert v.kernel == (V.FUSED if fused else V.FEW)
    groups = -(-(-(-n // 32)) // v.size)
    assert (m * -(-k // 128) * 128 * groups < 2 ** 24) == fused


@pytest.mark.parametrize("shape,call,dtype,cols,want", [
    ((8200, 16384, 128, 0), V.FWD, mx.MX_BF16, 16384, True), ((8200, 16384, 128, 0), V.FWD, mx.MX_BF16, 16416, True),
    ((8200, 16384, 128, 0), V.FWD, mx.MX_BF16, 16400, False), ((8200, 16384, 128, 0), V.FWD, mx.MX_BF16, 16391, False),
    ((8200, 8192, 128, 0), V.FWD, mx.MX_F32, 8192, True), ((8200, 8192, 128, 0), V.FWD, mx.MX_F32, 8208, True),
    ((8200, 8192, 128, 0), V.FWD, mx.MX_F32, 8196, False), ((8200, 8192, 128, 0), V.FWD, mx.MX_F16, 8192, False),
    ((8200, 128, 16384, 0), V.DGRAD, mx.MX_F16, 16384, True), ((8200, 128, 16384, 0), V.DGRAD, mx.MX_F16, 16385, False),
    ((100, 4096, 4096, 16), V.WGRAD, mx.MX_F32, 4096, True), ((100, 4096, 4096, 16), V.WGRAD, mx.MX_F32, 4100, False),
    ((100, 4096, 4096, 0), V.WGRAD, mx.MX_F32, 4096, False), ((4096, 4096, 4096, 0), V.FWD, mx.MX_BF16, 4096, False)])
def test_outputs_past_the_caches_have_rows_of_whole_64_bytes(shape, call, dtype, cols, want):
    """Rows that share lines are slower past the caches than through them."""
    m, n, k, e = shape
    d = mx.linear_desc(m, n, k, experts=e)
    assert V.streams(d, call, 0x10000, dtype, cols) == want
    assert not V.streams(d, call, 0x10020, dtype, cols)


@pytest.mark.parametrize("dtype,ld,want", [
    (mx.MX_BF16, 8192, True), (mx.MX_BF16, 8224, True), (mx.MX_BF16, 8208, False), (mx.MX_BF16, 8200, False), (mx.MX_BF16, 8191, False),
    (mx.MX_F32, 8208, True), (mx.MX_F32, 8200, False), (mx.MX_F32, 8196, False), (mx.MX_F16, 32, True), (mx.MX_F16, 8, False)])
def test_dequantized_rows_past_the_caches_are_of_whole_64_bytes(dtype, ld, want):
    d = mx.linear_desc(100, 128, ld)
    assert V.streams(d, V.DEQUANTIZE, 0x10000, dtype, ld) == want
    assert not V.streams(d, V.DEQUANTIZE, 0x10010, dtype, ld)
