"""A gated recurrent layer with 4-bit projections, run with the library's operators:

  input      block norm (residual, norm) -> 4-bit rows -> projections
  recurrence lores_scan (a prompt) or lores_decode_step (a token)
  readout    gated norm -> 4-bit rows -> output projection
  output     block norm: norm after the block, residual scale, norm of the next block
  training   both passes of the norms and the scan under torch.autograd

    python examples/gated_layer.py [--device cuda:0]

Weights and inputs are random.  Prints how far decoding lies from the prompt over
the same tokens, how far the 4-bit layer lies from the same layer in bf16, and the
gradients' sizes.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_linear_recurrence_amd as lores  # noqa: E402

EPS = 1e-6
SCALE = 0.5                                          # of a block's output in the residual stream


class BlockNorm(torch.autograd.Function):
    """(y, h) of lores_block_norm: h = residual + SCALE norm(x) weight, y = norm(h) weight_next."""

    @staticmethod
    def forward(ctx, x, residual, weight, weight_next):
        y, _, h = lores.lores_block_norm(x, residual, weight, weight_next, EPS, scale=SCALE)
        ctx.save_for_backward(x, h, weight, weight_next)
        return y, h

    @staticmethod
    def backward(ctx, dy, dh):
        x, h, weight, weight_next = ctx.saved_tensors
        dx, dres, _, dw, dwn = lores.lores_block_norm_backward(x, h, weight, weight_next, dy.contiguous(), EPS,
                                                               scale=SCALE, dh=dh.contiguous())
        return dx, dres, dw.to(weight.dtype), dwn.to(weight.dtype)


class GatedNorm(torch.autograd.Function):
    """norm(o) weight silu(z) per head."""

    @staticmethod
    def forward(ctx, o, z, weight):
        ctx.save_for_backward(o, z, weight)
        return lores.lores_gated_norm(o, z, weight, EPS)[0]

    @staticmethod
    def backward(ctx, dy):
        o, z, weight = ctx.saved_tensors
        do, dz, dw = lores.lores_gated_norm_backward(o, z, weight, dy.contiguous(), EPS)
        return do, dz, dw.to(weight.dtype)


class Scan(torch.autograd.Function):
    """o of lores_scan from the zero state (delta rule)."""

    @staticmethod
    def forward(ctx, q, k, v, alpha, beta):
        ctx.save_for_backward(q, k, v, alpha, beta)
        return lores.lores_scan(q, k, v, alpha, beta, 1)[0]

    @staticmethod
    def backward(ctx, do):
        return lores.lores_scan_backward(*ctx.saved_tensors, 1, do.contiguous())[:5]


class Layer:
    def __init__(self, device, width=256, H=4, d=64, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.H, self.d, self.width = H, d, width
        # q, k, v, the output gate and the two gates per head in one projection
        self.parts = (H * d, H * d, H * d, H * d, H, H)

        def mat(n, m):
            return (torch.randn(n, m, generator=g, device=device) / m ** 0.5).to(torch.bfloat16)

        def ones(n):
            return (1 + 0.1 * torch.randn(n, generator=g, device=device)).to(torch.bfloat16)

        self.p = {"first": ones(width), "in": mat(sum(self.parts), width), "onorm": ones(d),
                  "out": mat(width, H * d), "post": ones(width), "next": ones(width)}
        # laid out once, as a serving program keeps them
        self.mx = {n: lores.lores_mx_quant(self.p[n]) for n in ("in", "out")}

    def split(self, u):
        """q, k (unit rows), v, z [..., H, d], alpha, beta [..., H] of the projection's rows."""
        q, k, v, z, a, b = u.split(self.parts, -1)
        q, k, v, z = (x.unflatten(-1, (self.H, self.d)) for x in (q, k, v, z))

        def unit(x):
            x = x.float()
            return (x / (x.norm(dim=-1, keepdim=True) + EPS)).to(torch.bfloat16)

        return (unit(q), unit(k), v, z, torch.exp(-torch.nn.functional.softplus(a.float() - 3.0)),
                2.0 * torch.sigmoid(b.float()))

    def before(self, x, residual, exact=False):
        """The residual stream and the projection of its norm."""
        if exact:
            y, _, h = lores.lores_block_norm(x, residual, None, self.p["first"], EPS)
            return y @ self.p["in"].t(), h
        codes, scales, h = lores.lores_block_norm(x, residual, None, self.p["first"], EPS,
                                                  out_prec=lores.LORES_MXFP4)
        return lores.lores_mx_matmul(codes, scales, *self.mx["in"]), h

    def after(self, o, z, h, exact=False):
        """The next block's input and the residual stream, from the readout."""
        if exact:
            y, _ = lores.lores_gated_norm(o, z, self.p["onorm"], EPS)
            y = y.flatten(-2) @ self.p["out"].t()
        else:
            codes, scales = lores.lores_gated_norm(o, z, self.p["onorm"], EPS, out_prec=lores.LORES_MXFP4)
            y = lores.lores_mx_matmul(codes, scales, *self.mx["out"])
        y, _, h = lores.lores_block_norm(y, h, self.p["post"], self.p["next"], EPS, scale=SCALE)
        return y, h

    def prompt(self, x, residual, exact=False):
        """(next input, residual stream, state) over x [B, T, width]."""
        u, h = self.before(x, residual, exact)
        q, k, v, z, alpha, beta = self.split(u)
        o, S = lores.lores_scan(q, k, v, alpha, beta, 1)
        return (*self.after(o, z, h, exact), S)

    def step(self, st, x, residual, t):
        """One decoding step over x [B, width] on a lores state of H heads."""
        u, h = self.before(x, residual)
        q, k, v, z, alpha, beta = self.split(u)
        o = lores.lores_decode_step(st, q, k, v.contiguous(), alpha, beta, 1, 0, t)
        return self.after(o.to(torch.bfloat16), z, h)

    def loss(self, p, x, residual, target):
        """A training loss through both passes, on bf16 weights p."""
        y, h = BlockNorm.apply(x, residual, p["post"], p["first"])
        q, k, v, z, alpha, beta = self.split(y @ p["in"].t())
        o = Scan.apply(q, k, v.contiguous(), alpha, beta)
        y = GatedNorm.apply(o, z, p["onorm"]).flatten(-2) @ p["out"].t()
        y, h = BlockNorm.apply(y, h, p["post"], p["next"])
        return (y.float() - target.float()).square().mean() + h.float().square().mean()


def run(device):
    torch.manual_seed(0)
    layer = Layer(device)
    B, T, n = 3, 90, 6
    x, r = (torch.randn(B, T + n, layer.width, device=device).to(torch.bfloat16) for _ in range(2))
    want, stream, _ = layer.prompt(x, r)
    exact, _, _ = layer.prompt(x, r, exact=True)

    def off(a, b):
        return float((a.float() - b.float()).norm() / b.float().norm())

    _, _, S = layer.prompt(x[:, :T].contiguous(), r[:, :T].contiguous())
    st = lores.lores_state_alloc(B, layer.H, layer.d, layer.d, [lores.LORES_FP32] * layer.H, device=device)
    lores.lores_quant_state(st, S, 0)
    steps = [layer.step(st, x[:, T + t].contiguous(), r[:, T + t].contiguous(), t + 1) for t in range(n)]
    p = {k: v.clone().requires_grad_() for k, v in layer.p.items()}
    target = torch.randn(B, T + n, layer.width, device=device).to(torch.bfloat16)
    loss = layer.loss(p, x, r, target)
    grads = dict(zip(p, torch.autograd.grad(loss, list(p.values()))))
    return {"decode": off(torch.stack([s[0] for s in steps], 1), want[:, T:]),
            "stream": off(torch.stack([s[1] for s in steps], 1), stream[:, T:]),
            "four_bits": off(want, exact), "layer": layer, "data": (x, r, target), "grads": grads}


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--device", default="cuda:0")
    r = run(torch.device(ap.parse_args().device))
    print(f"decoding against the prompt: {r['decode']:.3g}, residual stream {r['stream']:.3g}")
    print(f"4-bit layer against bf16: {r['four_bits']:.3g}")
    print("gradients: " + ", ".join(f"{k} {float(g.float().norm()):.3g}" for k, g in r["grads"].items()))
