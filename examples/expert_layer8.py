"""A layer of experts behind a norm, trained and served in 8 bits.

Each token's row of the residual stream is normed, goes to two of the experts
(by a router that learns too) and comes back as their sum, weighted by the
router; the experts learn to reproduce a teacher's.  A training step norms the
tokens, sorts them by expert, quantizes them, the weights and the output
gradients to 8 bits, multiplies them in the three directions, and takes the
gradients back to the router, the norm's weight and the stream.  Then single
tokens are served from weights kept in 8 bits.

    python examples/expert_layer8.py [steps]
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import microscaling_quantized_convolution_mx_amd as mx

TOKENS, EXPERTS, CHOICES, FEATURES = 1500, 8, 2, 384


class Layer:
    """The parameters and, for a number of tokens, the buffers of a layer."""

    def __init__(self, tokens, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        randn = lambda *s: torch.randn(*s, device=device, generator=g)  # noqa: E731
        self.norm = torch.ones(FEATURES, device=device)
        self.router = randn(EXPERTS, FEATURES) / FEATURES ** 0.5
        self.w = randn(EXPERTS, FEATURES, FEATURES) / FEATURES ** 0.5
        self.wq = mx.Linear8QTensor(mx.linear_desc(0, FEATURES, FEATURES, experts=EXPERTS, block=128), mx.MX_ROLE_WEIGHT, device)
        self.resize(tokens, device)
        self.quantize()

    def resize(self, tokens, device="cuda"):
        new = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device=device)  # noqa: E731
        rows = tokens * CHOICES
        self.nd = mx.norm_desc(tokens, FEATURES)
        self.rd = mx.route_desc(tokens, CHOICES, EXPERTS, FEATURES)
        # square blocks for the weights, a scale per 128 contracted elements for the others
        self.d, self.d1 = (mx.linear_desc(rows, FEATURES, FEATURES, experts=EXPERTS, block=b) for b in (128, 1))
        self.xq, self.dyq = (mx.Linear8QTensor(self.d1, r, device) for r in (mx.MX_ROLE_ACT, mx.MX_ROLE_GRAD))
        self.h, self.out, self.dh, self.dx = (new(tokens, FEATURES) for _ in range(4))
        self.hs, self.ys, self.dys, self.dhs = (new(rows, FEATURES) for _ in range(4))
        self.rstd = new(tokens, dtype=torch.float32)
        self.offsets, self.rows = new(EXPERTS + 1, dtype=torch.int32), new(tokens, CHOICES, dtype=torch.int32)
        self.dweight = new(tokens, CHOICES, dtype=torch.float32)
        self.dnorm, self.dw = torch.empty_like(self.norm), torch.empty_like(self.w)
        need = max(mx.mx_linear8_workspace_bytes(self.d), mx.mx_norm_workspace_bytes(self.nd), mx.mx_route_workspace_bytes(self.rd), 16)
        self.ws = torch.empty(need, dtype=torch.uint8, device=device)

    def quantize(self):
        mx.mx_linear8_quantize(self.d, mx.MX_ROLE_WEIGHT, self.w, self.wq)

    def route(self):
        """Experts and weights of the normed tokens, and their places by expert."""
        best, self.expert = (self.h.float() @ self.router.T).topk(CHOICES, dim=1)
        self.weight = torch.softmax(best, 1)
        mx.mx_route_sort(self.rd, self.expert.int(), self.offsets, self.rows, workspace=self.ws)
        mx.mx_route_gather(self.rd, self.h, self.rows, self.hs)

    def forward(self, x):
        self.x = x
        mx.mx_norm_fwd(self.nd, x, self.norm, self.h, rstd=self.rstd)
        self.route()
        mx.mx_linear8_quantize(self.d1, mx.MX_ROLE_ACT, self.hs, self.xq, offsets=self.offsets)
        mx.mx_linear8_fwd(self.d, self.wq, self.xq, self.ys, self.ws, offsets=self.offsets)
        mx.mx_route_combine(self.rd, self.ys, self.rows, self.weight, self.out)
        return self.out

    def backward(self, dout):
        """Gradients of the parameters, and of x in self.dx."""
        mx.mx_route_combine_bwd(self.rd, dout, self.ys, self.rows, self.weight, self.dys, self.dweight)
        mx.mx_linear8_quantize(self.d1, mx.MX_ROLE_GRAD, self.dys, self.dyq, offsets=self.offsets)
        mx.mx_linear8_dgrad(self.d, self.wq, self.dyq, self.dhs, self.ws, offsets=self.offsets)
        mx.mx_linear8_wgrad(self.d, self.dyq, self.xq, self.dw, self.ws, offsets=self.offsets)
        mx.mx_route_gather_bwd(self.rd, self.dhs, self.rows, self.dh)
        # the router's: through the softmax over the chosen ones
        d = self.weight * (self.dweight - (self.weight * self.dweight).sum(1, keepdim=True))
        logits = torch.zeros(len(d), EXPERTS, device=d.device).scatter_(1, self.expert, d)
        self.drouter = logits.T @ self.h.float()
        self.dh += (logits @ self.router).bfloat16()
        mx.mx_norm_bwd(self.nd, self.dh, self.x, self.norm, self.rstd, self.dx, self.dnorm, workspace=self.ws)

    def serve(self, x):
        """A few tokens, whose rows are quantized on the way into the product."""
        mx.mx_norm_fwd(self.nd, x, self.norm, self.h)
        self.route()
        mx.mx_linear8_apply(self.d, self.wq, self.hs, self.ys, self.ws, offsets=self.offsets)
        mx.mx_route_combine(self.rd, self.ys, self.rows, self.weight, self.out)
        return self.out


def main(steps: int = 60, device: str = "cuda"):
    g = torch.Generator(device=device).manual_seed(1)
    teacher, layer = Layer(TOKENS, 2, device), Layer(TOKENS, 3, device)
    layer.router.copy_(teacher.router)
    layer.w.mul_(0.1)
    layer.quantize()
    losses = []
    for step in range(steps):
        x = torch.randn(TOKENS, FEATURES, device=device, generator=g).bfloat16()
        err = layer.forward(x).float() - teacher.forward(x).float()
        losses.append(float((err ** 2).mean()))
        layer.backward((err * (2 / TOKENS)).bfloat16())
        layer.w -= 1.0 * layer.dw
        layer.router -= 0.1 * layer.drouter
        layer.norm -= 0.05 * layer.dnorm
        layer.quantize()
        if step % 10 == 0 or step == steps - 1:
            print(f"step {step:3d}  loss {losses[-1]:.4f}", flush=True)

    few = 5
    x = torch.randn(few, FEATURES, device=device, generator=g).bfloat16()
    for one in (layer, teacher):
        one.resize(few, device)
    served, want = layer.serve(x).float(), teacher.serve(x).float()
    off = float((served - want).norm() / want.norm())
    print(f"served {few} tokens, {off:.3f} from the teacher", flush=True)
    return losses, off


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
