"""Plain 64-bit implementation of the norm and its gradients (numpy on the
CPU), with the error that fp32 arithmetic in any order of the sums can have."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of fp32
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # eps / 2, relative to the value
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}    # half a step of the subnormals, at least


def norm(total, w, eps):
    rstd = 1.0 / np.sqrt((total ** 2).mean(1, keepdims=True) + eps)
    return total * rstd * w, rstd


def rstd_error(k: int) -> float:
    """Relative: k squares and sums, all positive, with a rounding each, the
    division by k and eps' addition, halved by the root; the root and the
    reciprocal."""
    return ((k + 1 + 2) * U) / 2 * 1.01 + 2 * U


def y_error(k: int) -> float:
    """... and two products, before the rounding to y's type."""
    return rstd_error(k) + 2 * U * 1.01


def grads(dy, total, w, rstd, dtotal):
    """(dx, its bound in fp32 before the last rounding, dweight, its bound)."""
    k = total.shape[1]
    h, g = total * rstd, dy * w
    gh = g * h
    m = gh.mean(1, keepdims=True)
    # h, g and their product one rounding each, k additions, the division
    m_err = (k + 4) * U * 1.01 * np.abs(gh).mean(1, keepdims=True)
    inner = g - h * m
    # g: 1, h: 1, h m: 1, the difference: 1; times rstd: 1; plus dtotal: 1
    err = np.abs(rstd) * (np.abs(g) * 3 * U + np.abs(h * m) * 4 * U + np.abs(h) * m_err) * 1.01
    dx = rstd * inner + dtotal
    err = err + U * 1.01 * (np.abs(dx) + err)
    dw = (dy * h).sum(0)
    dw_err = (len(dy) + 3) * U * 1.01 * np.abs(dy * h).sum(0)
    return dx, err, dw, dw_err


def bound(ref, err, dtype: str):
    """Of a value with error `err` rounded once to the type."""
    return err + HALF_STEP[dtype] * (np.abs(ref) + err) + TINY[dtype]
