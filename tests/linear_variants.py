"""The kernels that the library chooses for the linear layers' calls, and the
cases that reach each of them: `wanted` says of a case which one a call takes,
so that no change of the rules can leave a kernel without a test unnoticed."""
from __future__ import annotations

import ctypes
from collections import namedtuple

import microscaling_quantized_convolution_mx_amd as mx
from microscaling_quantized_convolution_mx_amd import linear as ML

FWD, DGRAD, WGRAD, APPLY, DEQUANTIZE = range(5)
NONE, FEW, FUSED, PRODUCT = range(4)
Variant = namedtuple("Variant", "kernel size splits threads workgroups")


def variant(d, call: int) -> Variant:
    """What `call` launches on descriptor d: size is the stripes per workgroup
    of the few-token kernel, or the rows of a product's tile."""
    ML._load()
    f = mx.lib().mx_internal_linear_variant
    f.restype, f.argtypes = ctypes.c_int, [ctypes.POINTER(mx.mx_linear_desc), ctypes.c_int, ctypes.c_void_p]
    out = (ctypes.c_int64 * 5)()
    assert f(d, call, ctypes.addressof(out)) == 0
    return Variant(*out)


# (tokens, out features, in features, tokens of each expert), what _fwd, _dgrad
# and _wgrad take: the tile's rows, and whether the contraction is split
PRODUCTS = [
    ((260, 300, 200, None), (64, False), (64, False), (64, False)),
    ((203, 130, 4100, None), (64, True), (64, False), (64, False)),
    ((203, 4100, 130, None), (64, False), (64, True), (64, False)),
    ((4097, 65, 67, None), (64, False), (64, False), (64, True)),
    ((2050, 2070, 2090, None), (128, False), (128, False), (128, False)),
    ((4090, 4090, 4090, None), (256, False), (256, False), (256, False)),
    ((700, 300, 260, [130, 0, 500, 70]), (64, False), (64, False), (64, False)),
    ((4201, 2090, 2050, [1600, 2, 0, 2599]), (128, False), (128, False), (128, False)),
    ((6001, 2304, 2300, [3000, 1, 0, 2500, 500]), (256, False), (256, False), (128, False)),
    ((12000, 2300, 2200, [7001, 0, 4999]), (128, False), (128, False), (256, False)),
]

# (tokens, out features, in features, tokens of each expert), what _fwd, _dgrad and
# _apply take of the few-token kernel: stripes per workgroup, and for _apply whether it quantizes
FEW_TOKENS = [
    ((9, 300, 500, None), 1, 1, (1, True)),
    ((32, 200, 16400, None), 1, 2, (1, False)),
    ((3, 16400, 300, None), 2, 1, (2, True)),
    ((31, 16400, 2100, None), 2, 1, (2, False)),
    ((5, 65600, 200, None), 4, 1, (4, True)),
    ((7, 65600, 2100, None), 4, 1, (4, True)),
    ((32, 65600, 2000, None), 4, 1, (4, False)),
    ((5, 200, 65600, None), 1, 4, (1, False)),
    ((64, 1030, 300, [1, 0, 7, 0] * 4 + [0] * 47 + [32]), 4, 2, (4, True)),
    ((300, 900, 1000, [40, 0, 1, 100] + [9] * 15 + [24]), 2, 2, (2, True)),
    ((1000, 1030, 2100, [70, 0, 1] + [15] * 60 + [29]), 4, 4, (4, False)),
    ((999, 300, 260, [0] * 40 + [999] + [0] * 23), 2, 2, (2, True)),
    ((301, 300, 260, [301] + [0] * 39), 1, 1, (1, True)),
]


def streams(d, call: int, out: int, dtype: int, ld: int) -> bool:
    """Whether `call` would write its output, at this address and row stride, past the caches."""
    ML._load()
    f = mx.lib().mx_internal_linear_streams
    f.restype = ctypes.c_int
    f.argtypes = [ctypes.POINTER(mx.mx_linear_desc), ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_int64]
    return bool(f(d, call, out, dtype, ld))
