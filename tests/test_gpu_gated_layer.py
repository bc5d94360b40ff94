"""The example layer of gated norm, block norms and 4-bit projections: prompt,
decoding and gradients together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
EPS, SCALE = 1e-6, 0.5
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_layer.py")


@pytest.fixture(scope="module")
def result():
    spec = importlib.util.spec_from_file_location("example_gated_layer", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module.run(torch.device("cuda:0"))


def test_decoding_follows_the_prompt(result):
    # fp32 states; the readout's bf16 roundings (2^-8) move a few of its 4-bit codes by
    # a step, a fourth to a sixth of their size, each among 256 terms of an output
    assert result["decode"] < 2.0 ** -4 and result["stream"] < 2.0 ** -4


def test_four_bits_are_near_the_layer_in_bf16(result):
    # two operands a product and two products, each rounded by a step of 1/4 to 1/12 of a
    # value, uniform: 0.1 of its size in the 2-norm or so for each of the four
    assert 0 < result["four_bits"] < 0.5


def plain_loss(layer, p, x, residual, target):
    """The training loss in fp64 by elementary operations, the recurrence token by token."""
    def norm(u, w):
        return u * (u.square().mean(-1, keepdim=True) + EPS).rsqrt() * w

    h = residual + SCALE * norm(x, p["post"])
    q, k, v, z, a, b = (norm(h, p["first"]) @ p["in"].T).split(layer.parts, -1)
    q, k, v, z = (u.unflatten(-1, (layer.H, layer.d)) for u in (q, k, v, z))
    q, k = (u / (u.norm(dim=-1, keepdim=True) + EPS) for u in (q, k))
    alpha, beta = torch.exp(-torch.nn.functional.softplus(a - 3.0)), 2.0 * torch.sigmoid(b)
    S, o = torch.zeros(x.shape[0], layer.H, layer.d, layer.d, dtype=x.dtype), []
    for t in range(x.shape[1]):
        S = S * alpha[:, t, :, None, None]
        u = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, None, :]).sum(-1))
        S = S + u[..., None] * k[:, t, :, None, :]
        o.append((S * q[:, t, :, None, :]).sum(-1))
    y = norm(torch.stack(o, 1), p["onorm"]) * torch.nn.functional.silu(z)
    h = h + SCALE * norm(y.flatten(-2) @ p["out"].T, p["post"])
    return (norm(h, p["next"]) - target).square().mean() + h.square().mean()


def test_gradients_match_the_formulas(result):
    """Every weight's gradient against autograd in fp64.  On the way forward and back some
    24 tensors are rounded to bf16, half a step of 2^-8 each: 24 2^-8 of the gradient
    together if none of it cancels; 2^-3 leaves a third for the gates' slopes."""
    layer, data = result["layer"], [t.double().cpu() for t in result["data"]]
    p = {k: v.double().cpu().requires_grad_() for k, v in layer.p.items()}
    want = torch.autograd.grad(plain_loss(layer, p, *data), list(p.values()))
    for (name, g), w in zip(result["grads"].items(), want):
        g = g.double().cpu()
        assert g.shape == w.shape
        assert float((g - w).norm()) <= 2.0 ** -3 * float(w.norm()), name
