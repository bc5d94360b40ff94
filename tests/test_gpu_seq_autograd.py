"""The sequence operators record no autograd graph, and say so to a caller whose
inputs require a gradient; under no_grad and inside an autograd.Function, which
calls the backward operator itself, they are silent."""
import warnings

import pytest
import torch

import quantized_linear_recurrence_amd as lores

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _scan(**grad):
    x = {"q": torch.ones(1, 3, 1, 32), "k": torch.ones(1, 3, 1, 32), "v": torch.ones(1, 3, 1, 4),
         "alpha": torch.ones(1, 3, 1), "beta": torch.ones(1, 3, 1), "S0": torch.ones(1, 1, 4, 32)}
    x = {n: t.to(DEV).requires_grad_(n in grad) for n, t in x.items()}
    return lores.lores_scan(x["q"], x["k"], x["v"], x["alpha"], x["beta"], 0, S0=x["S0"])


def _norm(**grad):
    x = {n: torch.ones(*s, device=DEV).requires_grad_(n in grad)
         for n, s in (("x", (2, 8)), ("weight", (8,)), ("residual", (2, 8)))}
    return lores.lores_rmsnorm(x["x"], x["weight"], 1e-6, residual=x["residual"])


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight):
        ctx.save_for_backward(x, weight)
        return lores.lores_rmsnorm(x, weight, 1e-6)[0]

    @staticmethod
    def backward(ctx, dy):
        return lores.lores_rmsnorm_backward(*ctx.saved_tensors, dy.contiguous(), 1e-6)


@pytest.mark.parametrize("call,name", [(_scan, n) for n in ("q", "k", "v", "alpha", "beta", "S0")]
                         + [(_norm, n) for n in ("x", "weight", "residual")])
def test_an_input_that_requires_a_gradient_warns(call, name):
    with pytest.warns(UserWarning, match="records no autograd graph"):
        call(**{name: True})
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        call()
        with torch.no_grad():
            call(**{name: True})


def test_a_function_is_silent_and_has_the_gradient():
    x = torch.randn(4, 64, device=DEV, requires_grad=True)
    w = torch.ones(64, device=DEV, requires_grad=True)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        _Norm.apply(x, w).sum().backward()
    want = lores.lores_rmsnorm_backward(x.detach(), w.detach(), torch.ones_like(x), 1e-6)
    assert torch.equal(x.grad, want[0]) and torch.equal(w.grad, want[1])
