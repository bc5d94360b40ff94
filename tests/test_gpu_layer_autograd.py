"""The layer operators record no autograd graph, and say so to a caller whose inputs
require a gradient; under no_grad they are silent."""
import warnings

import pytest
import torch

import quantized_linear_recurrence_amd as lores

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _ones(grad, name, *shape, dtype=torch.float32):
    return torch.ones(*shape, device=DEV).to(dtype).requires_grad_(name in grad)


def _quant(*grad):
    return lores.lores_mx_quant(_ones(grad, "x", 4, 64))


def _matmul(*grad):
    w = lores.lores_mx_quant(torch.ones(8, 64, device=DEV))
    return lores.lores_mx_matmul(_ones(grad, "a", 4, 64, dtype=torch.float8_e4m3fn), _ones(grad, "a_scales", 4), *w)


CALLS = [(_quant, "x"), (_matmul, "a_scales"), (_matmul, "a")]


@pytest.mark.parametrize("call,name", CALLS)
def test_an_input_that_requires_a_gradient_warns(call, name):
    with pytest.warns(UserWarning, match="records no autograd graph"):
        call(name)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        call()
        with torch.no_grad():
            call(name)
