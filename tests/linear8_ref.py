"""Plain 64-bit implementation of the 8-bit linear layers' format (numpy on the
CPU), written from its definition, for the tests to compare with."""
from __future__ import annotations

import numpy as np

from linear_ref import bound as bound32, segments  # noqa: F401


def round_e4m3(v):
    """v (448 at most in magnitude) on the E4M3 grid, ties to even: 4
    significant bits, and multiples of 2^-9 below 2^-6."""
    e = np.maximum(np.frexp(np.abs(v))[1] - 1, -6)
    step = np.ldexp(1.0, e - 3)
    return np.copysign(np.rint(v / step) * step, v)


def exponent(top):
    """The smallest e >= -127 with top <= 448 * 2^e."""
    e = np.frexp(top)[1] - 9  # 448 = 0.875 * 2^9
    e = e + (top > np.ldexp(448.0, e))
    return np.where(top == 0, -127, np.maximum(e, -127))


def quantize(x, rows: int, cols: int):
    """(values on the grid, scale code of each element) of x in float64, in
    blocks of rows x cols counted from the first element."""
    r, c = x.shape
    if x.size == 0:
        return np.zeros((r, c)), np.zeros((r, c), np.uint8)
    b = np.pad(x, ((0, -r % rows), (0, -c % cols)))
    b = b.reshape(b.shape[0] // rows, rows, b.shape[1] // cols, cols)
    finite = np.isfinite(b).all(axis=(1, 3), keepdims=True)
    b = np.where(finite, b, 0.0)
    e = exponent(np.abs(b).max(axis=(1, 3), keepdims=True))
    val = np.where(finite, np.ldexp(round_e4m3(np.ldexp(b, -e)), e), np.nan)
    code = np.broadcast_to(np.where(finite, e + 127, 255), b.shape).astype(np.uint8)

    def back(a):
        return a.reshape(a.shape[0] * rows, -1)[:r, :c]
    return back(val), back(code)


def form(x, block: int, f: int):
    """Values that form f (0: rows, 1: columns) of a matrix holds."""
    return quantize(x, *((128, 128) if block == 128 else (1, 128) if f == 0 else (128, 1)))[0]


def form_tokens(x, block: int, f: int, offsets=None):
    """... of a matrix of tokens, blocks counted from each expert's first one."""
    val = np.zeros(x.shape)
    for a, b in segments(len(x), offsets):
        val[a:b] = form(x[a:b], block, f)
    return val


def code_bits(v):
    """E4M3 codes of values on the grid."""
    a = np.abs(v)
    e = np.maximum(np.frexp(a)[1] - 1, -6)
    m = np.ldexp(a, 3 - e).astype(int)  # 8..15, or below 8 for subnormals
    c = np.where(m >= 8, ((e + 7) << 3) + m - 8, m)
    return (c + 128 * np.signbit(v)).astype(np.uint8)


def bound(c: int, p, q, ref, dtype: str):
    """Largest distance of an output ref = p @ q over c contracted elements.

    fp32: c exact products summed in fp32 in any order.  16 bits: before the
    fp32 sums, of the 8 products of elements 8i .. 8i+7 each is cut towards zero
    to a multiple of 2^(E - 13), E the largest sum of two operands' exponents
    among them: at most 2^(E - 13) lost each, and 2^E <= the largest product's
    magnitude <= the largest |p| among the 8 times the largest |q|.  The rounded
    output follows."""
    mags = np.abs(p) @ np.abs(q)
    lim = bound32(c, mags, ref, dtype)
    if dtype != "f32" and p.size:
        pad = -p.shape[1] % 8
        a = np.pad(np.abs(p), ((0, 0), (0, pad))).reshape(len(p), -1, 8)
        b = np.pad(np.abs(q), ((0, pad), (0, 0))).reshape(-1, 8, q.shape[1])
        # the largest product of a group is below the largest of each times the other's largest
        cut = 8 * 2.0 ** -13 * (a.max(2) @ b.max(1))
        lim = lim + cut * (1 + {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype])
    return lim
