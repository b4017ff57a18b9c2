"""Calls that run at once on two streams, with workspaces, buffers and outputs of
their own: the results of the same calls one after the other, bit for bit."""
import numpy as np
import pytest
import torch

import microscaling_quantized_convolution_mx_amd as mx
from linear8_variants import APPLY, DGRAD, FWD, PRODUCT, WGRAD, variant
from test_gpu_linear import rand
from test_gpu_route import choices

pytestmark = pytest.mark.gpu

DEV = "cuda"


def at_once(jobs, times=10):
    """jobs: two of (call(stream), outputs, buffers that the call writes besides).  Alone, then together."""
    want = []
    for call, outs, _ in jobs:
        call(None)
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    for _, outs, scratch in jobs:
        for t in (*outs, *scratch):
            t.view(torch.uint8).fill_(0xFF)
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(times):
        for s, (call, _, _) in zip(streams, jobs):
            call(s)
    torch.cuda.synchronize()
    for (_, outs, _), w in zip(jobs, want):
        for a, b in zip(outs, w):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def workspace(n):
    return torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_split_products(dt):
    """Products whose contraction is split over workgroups, which leave partial sums in the workspace."""
    kind = mx.MX_F32 if dt == torch.float32 else mx.MX_BF16
    for call, sizes in ((FWD, (203, 130, 4100)), (DGRAD, (203, 4100, 130)), (WGRAD, (4097, 65, 67))):
        m, n, k = sizes
        d = mx.linear_desc(m, n, k, block=1)
        v = variant(d, call, kind)
        assert v.kernel == PRODUCT and v.splits > 1
        f, ra, rb = {FWD: (mx.mx_linear8_fwd, mx.MX_ROLE_WEIGHT, mx.MX_ROLE_ACT), DGRAD: (mx.mx_linear8_dgrad, mx.MX_ROLE_WEIGHT, mx.MX_ROLE_GRAD),
                     WGRAD: (mx.mx_linear8_wgrad, mx.MX_ROLE_GRAD, mx.MX_ROLE_ACT)}[call]
        shape = {FWD: (m, n), DGRAD: (m, k), WGRAD: (n, k)}[call]
        dims = {mx.MX_ROLE_ACT: (m, k), mx.MX_ROLE_WEIGHT: (n, k), mx.MX_ROLE_GRAD: (m, n)}

        def job(seed):
            q = []
            for role in (ra, rb):
                q.append(mx.Linear8QTensor(d, role, DEV))
                mx.mx_linear8_quantize(d, role, rand(seed + role, *dims[role]).to(DEV), q[-1])
            out, ws = torch.empty(shape, dtype=dt, device=DEV), workspace(mx.mx_linear8_workspace_bytes(d))
            return lambda s: f(d, *q, out, ws, stream=s), [out], [ws]
        at_once([job(1), job(11)])


def test_apply_with_tokens_in_the_workspace():
    """Tokens that are quantized into the workspace before the product, dense and by expert."""
    for m, n, k, lens in ((301, 500, 700, None), (2000, 300, 260, [900, 0, 1100])):
        d = mx.linear_desc(m, n, k, experts=len(lens or ()), block=128)
        assert variant(d, APPLY, mx.MX_BF16).kernel == PRODUCT
        off = None if lens is None else torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), device=DEV)

        def job(seed):
            wq = mx.Linear8QTensor(d, mx.MX_ROLE_WEIGHT, DEV)
            mx.mx_linear8_quantize(d, mx.MX_ROLE_WEIGHT, rand(seed, *((len(lens),) if lens else ()), n, k).to(DEV), wq)
            x, y = rand(seed + 1, m, k, dt="bf16").to(DEV), torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
            ws = workspace(mx.mx_linear8_workspace_bytes(d))
            return lambda s: mx.mx_linear8_apply(d, wq, x, y, ws, offsets=off, stream=s), [y], [ws]
        at_once([job(1), job(11)])


@pytest.mark.parametrize("m,k", [(1500, 900), (600, 17000)])
def test_norm_forward_and_backward(m, k):
    """Parts of the weight's gradient in the workspace."""
    d = mx.norm_desc(m, k)

    def job(seed):
        x, r, dy, dt = (rand(seed + i, m, k, dt="bf16").to(DEV) for i in range(4))
        w = rand(seed + 4, k).to(DEV)
        total, y, dx = (torch.empty_like(x) for _ in range(3))
        rstd, dw, ws = torch.empty(m, device=DEV), torch.empty(k, device=DEV), workspace(mx.mx_norm_workspace_bytes(d))
        q = mx.Linear8QTensor(mx.linear_desc(m, 8, k, block=1), mx.MX_ROLE_ACT, DEV, cols=False)

        def call(s):
            mx.mx_norm_fwd(d, x, w, y, residual=r, total=total, yq=q, rstd=rstd, stream=s)
            mx.mx_norm_bwd(d, dy, total, w, rstd, dx, dw, dtotal=dt, workspace=ws, stream=s)
        return call, [total, y, rstd, dx, dw, *q.buffers[0]], [ws]
    at_once([job(1), job(11)])


def test_route_there_and_back():
    m, c, e, k = 5000, 4, 40, 300
    d = mx.route_desc(m, c, e, k)

    def job(seed):
        a = choices(seed, m, c, e, 0.1)
        expert, used = torch.from_numpy(a).to(DEV), int(((a >= 0) & (a < e)).sum())
        x, y, dout = (rand(seed + i, n, k, dt="bf16").to(DEV) for i, n in ((1, m), (2, m * c), (3, m)))
        w = rand(seed + 4, m, c).to(DEV)
        i32 = dict(dtype=torch.int32, device=DEV)
        offsets, rows = torch.empty(e + 1, **i32), torch.empty(m, c, **i32)
        out, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
        xs, dy = torch.zeros_like(y), torch.zeros_like(y)  # (rows of no choice stay as they are: not outputs)
        ws = workspace(mx.mx_route_workspace_bytes(d))

        def call(s):
            mx.mx_route_sort(d, expert, offsets, rows, workspace=ws, stream=s)
            mx.mx_route_gather(d, x, rows, xs, stream=s)
            mx.mx_route_combine(d, y, rows, w, out, stream=s)
            mx.mx_route_combine_bwd(d, dout, y, rows, w, dy, dw, stream=s)
            mx.mx_route_gather_bwd(d, dy, rows, dx, stream=s)
        return call, [offsets, rows, out, dx, dw, xs[:used], dy[:used]], [ws]
    at_once([job(1), job(11)])
