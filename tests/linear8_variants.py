"""The kernels that the library chooses for calls on the layers in 8 bits, and
the cases that reach each of them, as linear_variants.py has them for 4 bits.
Products with fp32 outputs (exact ones) choose for themselves."""
from __future__ import annotations

import ctypes

import microscaling_quantized_convolution_mx_amd as mx
from linear_variants import APPLY, DGRAD, FEW, FUSED, FWD, NONE, PRODUCT, WGRAD, Variant  # noqa: F401
from microscaling_quantized_convolution_mx_amd import linear8 as M8


def variant(d, call: int, dtype: int) -> Variant:
    M8._load()
    f = mx.lib().mx_internal_linear8_variant
    f.restype, f.argtypes = ctypes.c_int, [ctypes.POINTER(mx.mx_linear_desc), ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    out = (ctypes.c_int64 * 5)()
    assert f(d, call, dtype, ctypes.addressof(out)) == 0
    return Variant(*out)


# (tokens, out features, in features, tokens of each expert); of _fwd, _dgrad and _wgrad the tile's rows and whether
# the contraction is split, with 16-bit outputs and with fp32 ones
PRODUCTS = [
    ((260, 300, 200, None), ((64, False),) * 3, ((64, False),) * 3),
    ((203, 130, 4100, None), ((64, True), (64, False), (64, False)), ((64, True), (64, False), (64, False))),
    ((203, 4100, 130, None), ((64, False), (64, True), (64, False)), ((64, False), (64, True), (64, False))),
    ((4097, 65, 67, None), ((64, False), (64, False), (64, True)), ((64, False), (64, False), (64, True))),
    ((2050, 2070, 2090, None), ((128, False),) * 3, ((128, False),) * 3),
    ((4090, 4090, 4090, None), ((256, False),) * 3, ((256, False),) * 3),
    ((700, 300, 260, [130, 0, 500, 70]), ((64, False),) * 3, ((64, False),) * 3),
    ((4201, 2090, 2050, [1600, 2, 0, 2599]), ((128, False),) * 3, ((128, False),) * 3),
    ((6001, 2304, 2300, [3000, 1, 0, 2500, 500]), ((256, False), (256, False), (128, False)), ((256, False), (256, False), (128, False))),
    ((9000, 3900, 3850, [9000]), ((128, False), (128, False), (256, False)), ((128, False), (128, False), (256, False))),
]

# (tokens, out features, in features, tokens of each expert), what _fwd, _dgrad and
# _apply take of the few-token kernel: stripes per workgroup, and for _apply whether it quantizes
FEW_TOKENS = [
    ((9, 300, 500, None), 1, 1, (1, True)),
    ((32, 200, 16400, None), 1, 2, (1, False)),
    ((3, 16400, 300, None), 2, 1, (2, True)),
    ((31, 16400, 2100, None), 2, 1, (2, False)),
    ((5, 200, 65600, None), 1, 2, (1, False)),
    ((64, 1030, 300, [1, 0, 7, 0] * 4 + [0] * 47 + [32]), 2, 2, (2, True)),
    ((300, 900, 1000, [40, 0, 1, 100] + [9] * 15 + [24]), 2, 2, (2, True)),
    ((1000, 1030, 2100, [70, 0, 1] + [15] * 60 + [29]), 2, 2, (2, False)),
    ((301, 300, 260, [301] + [0] * 39), 1, 1, (1, True)),
]
