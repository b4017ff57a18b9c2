"""The norm, the routing and the products in 8 bits run together as a layer of
experts uses them (examples/expert_layer8.py): each stage of a forward and
backward pass against 64 bits on what the stage before it gave, and the
example itself."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

import linear8_ref as R8
import microscaling_quantized_convolution_mx_amd as mx
import norm_ref as RN
from test_gpu_linear import f64, same
from test_gpu_route import places

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer8.py")
    spec = importlib.util.spec_from_file_location("expert_layer8", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def within(got, ref, lim):
    err = np.abs(f64(got) - ref)
    assert np.all(err <= lim), np.max(err / lim)


@pytest.mark.parametrize("tokens", [1, 37, 700])
def test_stages(example, tokens):
    E, C, F = example.EXPERTS, example.CHOICES, example.FEATURES
    layer = example.Layer(tokens, 4)
    x = torch.randn(tokens, F, device=DEV, generator=torch.Generator(device=DEV).manual_seed(5)).bfloat16()
    dout = torch.randn(tokens, F, device=DEV, generator=torch.Generator(device=DEV).manual_seed(6)).bfloat16()
    layer.norm.copy_(torch.linspace(0.5, 1.5, F))
    for t in (layer.ys, layer.hs, layer.dys, layer.dhs):
        t.fill_(float("nan"))  # every row is a choice's
    layer.forward(x)
    # the norm
    h, rstd = RN.norm(f64(x), f64(layer.norm), float(np.float32(1e-6)))
    within(layer.h, h, RN.bound(h, np.abs(h) * RN.y_error(F), "bf16"))
    # places and rows
    offsets, rows, _ = places(layer.expert.int().cpu().numpy(), E)
    same(f64(layer.offsets), offsets)
    same(f64(layer.rows), rows)
    hs = f64(layer.hs)
    for j in range(C):
        same(hs[rows[:, j]], f64(layer.h))
    # the product
    w = [R8.form(f64(a), 128, 0) for a in layer.w]
    xv, xc = (R8.form_tokens(hs, 1, f, offsets) for f in (0, 1))
    segs = R8.segments(len(hs), offsets)
    for e, (a, b) in enumerate(segs):
        if b > a:
            y = xv[a:b] @ w[e].T
            within(layer.ys[a:b], y, R8.bound(F, xv[a:b], w[e].T, y, "bf16"))
    # and back
    ys, wt = f64(layer.ys), f64(layer.weight)
    out = sum(ys[rows[:, j]] * wt[:, j, None] for j in range(C))
    mags = sum(np.abs(ys[rows[:, j]] * wt[:, j, None]) for j in range(C))
    within(layer.out, out, RN.bound(out, (C + 1) * RN.U * 1.01 * mags, "bf16"))

    layer.backward(dout)
    do, dys = f64(dout), f64(layer.dys)
    for j in range(C):
        ref = do * wt[:, j, None]
        within(layer.dys[torch.from_numpy(rows[:, j].astype(np.int64)).to(DEV)], ref, RN.bound(ref, RN.U * np.abs(ref), "bf16"))
        terms = do * ys[rows[:, j]]
        within(layer.dweight[:, j], terms.sum(1), (F + 2) * RN.U * 1.01 * np.abs(terms).sum(1))
    dv, dc = (R8.form_tokens(dys, 1, f, offsets) for f in (0, 1))
    for e, (a, b) in enumerate(segs):
        if b > a:
            ref = dv[a:b] @ w[e]
            within(layer.dhs[a:b], ref, R8.bound(F, dv[a:b], w[e], ref, "bf16"))
        ref = dc[a:b].T @ xc[a:b]
        within(layer.dw[e], ref, R8.bound(b - a, dc[a:b].T, xc[a:b], ref, "f32"))
    dx, err, dn, dn_err = RN.grads(f64(layer.dh), f64(x), f64(layer.norm), f64(layer.rstd)[:, None], 0.0)
    within(layer.dx, dx, RN.bound(dx, err, "bf16"))
    within(layer.dnorm, dn, dn_err + RN.TINY["f32"])
    # what the layer adds up itself: the rows' gradients, then the router's
    dhs = f64(layer.dhs)
    ref = sum(dhs[rows[:, j]] for j in range(C))
    alone = torch.empty_like(layer.dh)
    mx.mx_route_gather_bwd(layer.rd, layer.dhs, layer.rows, alone)
    within(alone, ref, RN.bound(ref, C * RN.U * 1.01 * sum(np.abs(dhs[rows[:, j]]) for j in range(C)), "bf16"))


def test_serving_takes_the_same_products(example):
    """A served token is what the training pass gives, but for the rounding of the sums."""
    layer = example.Layer(40, 7)
    x = torch.randn(40, example.FEATURES, device=DEV).bfloat16()
    trained = f64(layer.forward(x))
    hs, offsets = f64(layer.hs), layer.offsets.tolist()
    ys = f64(layer.ys)
    served = f64(layer.serve(x))
    xv = R8.form_tokens(hs, 1, 0, offsets)
    for e, (a, b) in enumerate(R8.segments(len(hs), offsets)):
        if b > a:
            w = R8.form(f64(layer.w[e]), 128, 0)
            y = xv[a:b] @ w.T
            lim = R8.bound(example.FEATURES, xv[a:b], w.T, y, "bf16")
            assert np.all(np.abs(f64(layer.ys[a:b]) - y) <= lim) and np.all(np.abs(ys[a:b] - y) <= lim)
    assert served.shape == trained.shape and np.isfinite(served).all()


def test_a_step_in_a_graph(example):
    """Forward and backward captured, replayed on other tokens with eager steps between: the eager results."""
    layer, eager = example.Layer(90, 8), example.Layer(90, 8)
    x, dout = (torch.randn(90, example.FEATURES, device=DEV).bfloat16() for _ in range(2))

    def step(one):
        one.forward(x)
        one.backward(dout)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(layer)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(layer)
    for i in range(4):
        x.copy_(torch.randn(90, example.FEATURES))
        dout.copy_(torch.randn(90, example.FEATURES))
        graph.replay()
        torch.cuda.synchronize()
        step(eager)
        torch.cuda.synchronize()
        for name in ("out", "dx", "dw", "dnorm", "dweight", "offsets", "rows"):
            assert torch.equal(getattr(layer, name), getattr(eager, name)), name


def test_example_runs(example):
    losses, off = example.main(steps=4)
    assert len(losses) == 4 and all(math.isfinite(v) for v in losses) and math.isfinite(off)


@pytest.mark.parametrize("tokens", [1, 37, 700])
def test_router_gradient(example, tokens):
    """The router's gradient and its part of the tokens', which the example adds up itself: against the formula in 64 bits, and
    against differences of the loss."""
    E, C, F = example.EXPERTS, example.CHOICES, example.FEATURES
    layer = example.Layer(tokens, 14)
    g = torch.Generator(device=DEV).manual_seed(15)
    x, dout = (torch.randn(tokens, F, device=DEV, generator=g).bfloat16() for _ in range(2))
    layer.norm.copy_(torch.linspace(0.5, 1.5, F))
    layer.forward(x)
    layer.backward(dout)
    w, dw, h, router = f64(layer.weight), f64(layer.dweight), f64(layer.h), f64(layer.router)
    expert, rows = layer.expert.cpu().numpy(), layer.rows.long()
    inner = (w * dw).sum(1, keepdims=True)
    # C products and their sum, a difference and a product: C + 3 roundings, none of a larger value than this
    d, d_err = w * (dw - inner), (C + 3) * RN.U * 1.01 * w * (np.abs(dw) + np.abs(w * dw).sum(1, keepdims=True))
    logits, err = np.zeros((tokens, E)), np.zeros((tokens, E))
    np.put_along_axis(logits, expert, d, 1)
    np.put_along_axis(err, expert, d_err, 1)
    ref = logits.T @ h
    within(layer.drouter, ref, err.T @ np.abs(h) + (tokens + 2) * RN.U * 1.01 * (np.abs(logits) + err).T @ np.abs(h))
    # its part of dh is rounded to bf16, and so is the sum with the rows' part
    alone = torch.empty_like(layer.dh)
    mx.mx_route_gather_bwd(layer.rd, layer.dhs, layer.rows, alone)
    part = logits @ router
    lim = err @ np.abs(router) + (E + 2) * RN.U * 1.01 * (np.abs(logits) + err) @ np.abs(router)
    lim = RN.bound(part, lim, "bf16")
    within(layer.dh, f64(alone) + part, RN.bound(f64(alone) + part, lim, "bf16"))

    # <dout, out> over the routers with the same choices and rows of the experts.  A weight's third derivative by a logit is at most
    # 1/8, so a step of 2^-10 in an element of size h moves the quotient by 2^-20 / 6 * h^3 / 8 of the terms, and 64-bit rounding by 2^-52 / 2^-10
    ys = f64(layer.ys)
    parts = np.stack([f64(dout) * ys[rows[:, j].cpu().numpy()] for j in range(C)], 1)
    terms, mags = parts.sum(2), np.abs(parts).sum(2).max(1)

    def loss(r):
        z = np.take_along_axis(h @ r.T, expert, 1)
        p = np.exp(z - z.max(1, keepdims=True))
        return float((p / p.sum(1, keepdims=True) * terms).sum())
    step = 2.0 ** -10
    for e, c in ((0, 0), (3, 200), (int(expert[0, 0]), 17), (int(expert[-1, 1]), F - 1)):
        a, b = router.copy(), router.copy()
        a[e, c] += step
        b[e, c] -= step
        got, diff = f64(layer.drouter)[e, c], (loss(a) - loss(b)) / (2 * step)
        slack = (np.abs(h[:, c]) ** 3 * 2.0 ** -23 * np.abs(terms).sum(1)).sum() + 2.0 ** -40 * np.abs(terms).sum()
        # dweight and the weights come in fp32: F products and their sum; a matrix product of F for the logits, each of which moves
        # a weight by at most a quarter of its error, an exponential, a sum and a quotient
        z_err = (F + 2) * RN.U * (np.abs(h) @ np.abs(router).T).max(1)
        slack += ((np.abs(terms).sum(1) * (z_err + 8 * RN.U) + (F + 2) * RN.U * mags) * 2 * np.abs(h[:, c])).sum()
        slack += (err.T @ np.abs(h) + (tokens + 2) * RN.U * np.abs(logits).T @ np.abs(h))[e, c] * 1.01
        assert abs(got - diff) <= slack


@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_serving_adds_the_products_up(example, tokens):
    """What is served is the weighted sum of its products."""
    C = example.CHOICES
    layer = example.Layer(tokens, 17)
    x = torch.randn(tokens, example.FEATURES, device=DEV, generator=torch.Generator(device=DEV).manual_seed(18)).bfloat16()
    layer.ys.fill_(float("nan"))
    served = layer.serve(x)
    rows, ys, wt = layer.rows.cpu().numpy(), f64(layer.ys), f64(layer.weight)
    out = sum(ys[rows[:, j]] * wt[:, j, None] for j in range(C))
    mags = sum(np.abs(ys[rows[:, j]] * wt[:, j, None]) for j in range(C))
    within(served, out, RN.bound(out, (C + 1) * RN.U * 1.01 * mags, "bf16"))
    # through the norm, the places and the rows that the training pass has
    h, _ = RN.norm(f64(x), f64(layer.norm), float(np.float32(1e-6)))
    within(layer.h, h, RN.bound(h, np.abs(h) * RN.y_error(example.FEATURES), "bf16"))
    for j in range(C):
        same(f64(layer.hs)[rows[:, j]], f64(layer.h))
