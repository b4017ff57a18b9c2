"""Plain 64-bit implementation of the microscaled linear layers (numpy on the
CPU), written from the format's definition, for the tests to compare with."""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def draws(rows: int, cols: int, seed: int) -> np.ndarray:
    """24-bit uniforms of the stochastic rounding, as fractions."""
    i = np.arange(rows * cols, dtype=np.uint64)
    with np.errstate(over="ignore"):
        z = np.uint64(seed) ^ (np.uint64(0x9E3779B97F4A7C15) * (i // np.uint64(2) + np.uint64(1)))
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        z ^= z >> np.uint64(31)
    u = np.where(i & np.uint64(1), z >> np.uint64(16), z >> np.uint64(40)) & np.uint64(0xFFFFFF)
    return (u.astype(np.float64) / 2.0 ** 24).reshape(rows, cols)


def quantize(x: np.ndarray, block: int, u: np.ndarray | None = None):
    """(codes 0..15, scale codes of each element, values) of x in float64,
    blocks counted from the first row."""
    r, c = x.shape
    codes = np.zeros((r, c), dtype=np.uint8)
    scale = np.zeros((r, c), dtype=np.uint8)
    val = np.zeros((r, c))
    for i in range(0, r, block):
        for j in range(0, c, 32):
            b = x[i:i + block, j:j + 32]
            s = (slice(i, i + b.shape[0]), slice(j, j + b.shape[1]))
            if not np.isfinite(b).all():
                scale[s], val[s] = 255, np.nan
                continue
            top = np.abs(b).max()
            e = -127 if top == 0 else int(np.clip(np.frexp(top)[1] - 1 - 2, -127, 127))
            v = np.minimum(np.ldexp(np.abs(b), -e), 6.0)
            lo = np.clip(np.searchsorted(GRID, v, side="right") - 1, 0, 6)
            f = (v - GRID[lo]) / (GRID[lo + 1] - GRID[lo])
            up = (f > 0.5) | ((f == 0.5) & (lo % 2 == 1)) if u is None else u[s] < f
            m = lo + up
            codes[s] = m + 8 * np.signbit(b)
            scale[s] = e + 127
            val[s] = np.copysign(np.ldexp(GRID[m], e), b)
    return codes, scale, val


def segments(m: int, offsets=None):
    """(first row, last row + 1) of each expert; one for a single layer."""
    return [(0, m)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))


def quantize_tokens(x, block, offsets=None, u=None):
    val = np.zeros(x.shape)
    for a, b in segments(len(x), offsets):
        val[a:b] = quantize(x[a:b], block, None if u is None else u[a:b])[2]
    return val


def bound(k: int, mags, y, dtype: str):
    """Largest distance of a sum of k exact products with magnitudes adding up
    to `mags`, summed in fp32 in any order (k roundings of 2^-23 relative to
    the running sum, truncation allowed) and rounded once to `dtype`."""
    out = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    tiny = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}[dtype]
    s = k * 2.0 ** -23 * mags
    return s + out * (np.abs(y) + s) + tiny + 2.0 ** -148
