"""A layer of experts, trained and served in microscaled 4-bit floating point.

Tokens choose one expert each by a fixed router; the experts' weights learn to
reproduce a teacher's.  A training step quantizes the tokens (sorted by expert),
the weights and the output gradients once each, multiplies them in the three
directions, and clips the weight gradients by their global norm before the
update of the fp32 weights.  Then single tokens are served from weights kept in
4 bits.

    python examples/expert_layer.py [steps]
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import microscaling_quantized_convolution_mx_amd as mx

TOKENS, EXPERTS, OUT, IN = 2000, 6, 384, 512


def route(x, router):
    """Tokens in the order of their experts, and where each expert's begin."""
    expert = (x @ router).argmax(1)
    order = torch.argsort(expert, stable=True)
    count = torch.bincount(expert, minlength=EXPERTS)
    offsets = torch.zeros(EXPERTS + 1, dtype=torch.int32, device=x.device)
    offsets[1:] = count.cumsum(0)
    return order, offsets, expert


def main(steps: int = 60, device: str = "cuda"):
    g = torch.Generator(device=device).manual_seed(0)
    randn = lambda *s: torch.randn(*s, device=device, generator=g)  # noqa: E731
    router, teacher = randn(IN, EXPERTS), randn(EXPERTS, OUT, IN) / IN ** 0.5
    w = torch.zeros(EXPERTS, OUT, IN, device=device)

    d = mx.linear_desc(TOKENS, OUT, IN, experts=EXPERTS)
    xq, wq, dyq = (mx.LinearQTensor(d, r, device) for r in (mx.MX_ROLE_ACT, mx.MX_ROLE_WEIGHT, mx.MX_ROLE_GRAD))
    ws = torch.empty(max(mx.mx_linear_workspace_bytes(d), 16), dtype=torch.uint8, device=device)
    y = torch.empty(TOKENS, OUT, device=device, dtype=torch.bfloat16)
    dx = torch.empty(TOKENS, IN, device=device, dtype=torch.bfloat16)
    dw = torch.empty_like(w)
    grads = mx.GradList([dw])
    norm = torch.empty(1, device=device)
    gws = torch.empty(mx.mx_grad_workspace_bytes(grads), dtype=torch.uint8, device=device)

    losses = []
    for step in range(steps):
        x = randn(TOKENS, IN)
        order, offsets, expert = route(x, router)
        want = torch.empty(TOKENS, OUT, device=device)
        for e in range(EXPERTS):
            want[expert == e] = x[expert == e] @ teacher[e].T
        x, want = x[order].bfloat16(), want[order]

        mx.mx_linear_quantize(d, mx.MX_ROLE_ACT, x, xq, offsets=offsets)
        mx.mx_linear_quantize(d, mx.MX_ROLE_WEIGHT, w, wq)
        mx.mx_linear_fwd(d, wq, xq, y, ws, offsets=offsets)
        err = y.float() - want
        losses.append(float((err ** 2).mean()))
        # gradients are rounded stochastically, another seed each step
        mx.mx_linear_quantize(d, mx.MX_ROLE_GRAD, err / TOKENS, dyq, mx.MX_SR, seed=step, offsets=offsets)
        mx.mx_linear_dgrad(d, wq, dyq, dx, ws, offsets=offsets)  # for the layer before this one
        mx.mx_linear_wgrad(d, dyq, xq, dw, ws, offsets=offsets)
        mx.mx_grad_clip(grads, 0.5, norm, gws)
        w -= 2.0 * dw
        if step % 10 == 0 or step == steps - 1:
            print(f"step {step:3d}  loss {losses[-1]:.4f}  gradient norm {float(norm):.4f}", flush=True)

    # serving: the weights stay quantized, each call brings a few tokens
    few = 5
    ds = mx.linear_desc(few, OUT, IN, experts=EXPERTS)
    x = randn(few, IN)
    order, offsets, expert = route(x, router)
    served = torch.empty(few, OUT, device=device)
    mx.mx_linear_quantize(d, mx.MX_ROLE_WEIGHT, w, wq)
    mx.mx_linear_apply(ds, wq, x[order], served, offsets=offsets)
    want = torch.stack([teacher[e] @ v for e, v in zip(expert[order].tolist(), x[order])])
    off = float((served - want).norm() / want.norm())
    print(f"served {few} tokens, {off:.3f} from the teacher", flush=True)
    return losses, off


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
