"""One recurrent layer with the library's operators, as a model runs it:

  prompt    residual + norm -> projections -> lores_scan -> norm of the readout,
            E4M3 for the output projection; the state, quantized, to decoding
  decoding  residual + norm -> projections -> lores_decode_step -> the same norm
  training  both passes of norm and scan under torch.autograd

    python examples/layer.py [--device cuda:0]

Weights and inputs are random; the prompt followed by decoding is compared with
the prompt over all tokens, and a few training steps bring a loss down.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_linear_recurrence_amd as lores  # noqa: E402

EPS = 1e-6


class Norm(torch.autograd.Function):
    """(y, h) of lores_rmsnorm over x + residual."""

    @staticmethod
    def forward(ctx, x, residual, weight):
        y, _, h = lores.lores_rmsnorm(x, weight, EPS, residual=residual)
        ctx.save_for_backward(h, weight)
        return y, h

    @staticmethod
    def backward(ctx, dy, dh):
        h, weight = ctx.saved_tensors
        dx, dw = lores.lores_rmsnorm_backward(h, weight, dy.contiguous(), EPS,
                                              dresidual=dh.contiguous())
        return dx, dx, dw.to(weight.dtype)


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
    def __init__(self, device, width=256, H=4, H_k=2, d_k=64, d_v=64, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.H, self.H_k, self.d_k, self.d_v = H, H_k, d_k, d_v

        def mat(n, m):
            return (torch.randn(n, m, generator=g, device=device) / n ** 0.5).to(torch.bfloat16)

        self.p = {"norm": torch.ones(width, dtype=torch.bfloat16, device=device),
                  "q": mat(width, H_k * d_k), "k": mat(width, H_k * d_k), "v": mat(width, H * d_v),
                  "gates": mat(width, 2 * H), "onorm": torch.ones(d_v, dtype=torch.bfloat16, device=device),
                  "out": mat(H * d_v, width)}

    def project(self, y):
        """q, k (unit rows), v, alpha, beta of normed rows y [..., width]."""
        p, s = self.p, y.shape[:-1]

        def unit(x):
            x = x.float().view(*s, self.H_k, self.d_k)
            return (x / (x.norm(dim=-1, keepdim=True) + EPS)).to(torch.bfloat16)

        a, b = (y @ p["gates"]).float().chunk(2, -1)
        return (unit(y @ p["q"]), unit(y @ p["k"]), (y @ p["v"]).view(*s, self.H, self.d_v),
                torch.exp(-torch.nn.functional.softplus(a - 3.0)), 2.0 * torch.sigmoid(b))

    def output(self, o):
        """The readout [..., H, d_v] normed per head, in E4M3 with one scale per
        head, through the output projection."""
        e, scales, _ = lores.lores_rmsnorm(o.reshape(-1, self.d_v), self.p["onorm"], EPS,
                                           out_prec=lores.LORES_FP8)
        y = (e.float() * scales[:, None]).to(torch.bfloat16)
        return y.view(*o.shape[:-2], self.H * self.d_v) @ self.p["out"]

    def prompt(self, x, residual, lengths=None):
        """(output, residual stream, state) over x [B, T, width]."""
        y, _, h = lores.lores_rmsnorm(x, self.p["norm"], EPS, residual=residual)
        o, S = lores.lores_scan(*self.project(y), 1, lengths=lengths)
        return self.output(o), h, S

    def step(self, st, x, residual, t):
        """One decoding step over x [B, width] on a lores state of H heads."""
        y, _, h = lores.lores_rmsnorm(x, self.p["norm"], EPS, residual=residual)
        q, k, v, alpha, beta = self.project(y)
        q, k = (z.repeat_interleave(self.H // self.H_k, 1).contiguous() for z in (q, k))
        o = lores.lores_decode_step(st, q, k, v.contiguous(), alpha, beta, 1, 0, t)
        return self.output(o.to(torch.bfloat16)), h

    def train_step(self, x, residual, target, lr):
        p = {n: w.detach().requires_grad_() for n, w in self.p.items()}
        keep, self.p = self.p, p
        y, h = Norm.apply(x, residual, p["norm"])
        o = Scan.apply(*self.project(y))
        z, _ = Norm.apply(o.reshape(-1, self.d_v), torch.zeros_like(o).reshape(-1, self.d_v), p["onorm"])
        out = z.view(*o.shape[:-2], self.H * self.d_v) @ p["out"] + h
        loss = (out.float() - target.float()).square().mean()
        grads = torch.autograd.grad(loss, list(p.values()))
        self.p = {n: (w.float() - lr * g.float()).to(w.dtype) for (n, w), g in zip(keep.items(), grads)}
        return float(loss.detach())


def run(device):
    torch.manual_seed(0)
    layer = Layer(device)
    B, T, n, width = 3, 90, 6, 256
    x, r = (torch.randn(B, T + n, width, device=device).to(torch.bfloat16) for _ in range(2))
    want, _, _ = layer.prompt(x, r)
    got, _, S = layer.prompt(x[:, :T].contiguous(), r[:, :T].contiguous())
    worst = (got.float() - want[:, :T].float()).norm() / want[:, :T].float().norm()
    st = lores.lores_state_alloc(B, layer.H, layer.d_k, layer.d_v, [lores.LORES_INT8] * layer.H, device=device)
    lores.lores_quant_state(st, S, 0)
    steps = []
    for t in range(n):
        o, _ = layer.step(st, x[:, T + t].contiguous(), r[:, T + t].contiguous(), t + 1)
        steps.append(o)
    got = torch.stack(steps, 1)
    decode = (got.float() - want[:, T:].float()).norm() / want[:, T:].float().norm()
    target = torch.randn(B, T, width, device=device).to(torch.bfloat16)
    losses = [layer.train_step(x[:, :T].contiguous(), r[:, :T].contiguous(), target, 2.0) for _ in range(5)]
    return {"prompt": float(worst), "decode": float(decode), "losses": losses}


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--device", default="cuda:0")
    r = run(torch.device(ap.parse_args().device))
    print(f"prompt against the longer prompt: {r['prompt']:.3g}")
    print(f"int8 decoding against the prompt: {r['decode']:.3g}")
    print("training losses: " + " ".join(f"{x:.4f}" for x in r["losses"]))
