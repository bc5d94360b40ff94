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


def _gated(*grad):
    return lores.lores_gated_norm(_ones(grad, "x", 4, 2, 64), _ones(grad, "gate", 4, 2, 64), _ones(grad, "weight", 64), 0.1)


def _block(*grad):
    return lores.lores_block_norm(_ones(grad, "x", 4, 64), _ones(grad, "residual", 4, 64), _ones(grad, "weight", 64),
                                  _ones(grad, "weight_next", 64), 0.1, gate=_ones(grad, "gate", 4, 64))


CALLS = [(_gated, n) for n in ("x", "gate", "weight")]
CALLS += [(_block, n) for n in ("x", "residual", "weight", "weight_next", "gate")]
CALLS += [(_quant, "x"), (_matmul, "a_scales"), (_matmul, "a")]


@pytest.mark.parametrize("call,name", CALLS)
def test_an_input_that_requires_a_gradient_warns(call, name):
    with pytest.warns(UserWarning, match="records no autograd graph"):
        call(name)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        call()
        with torch.no_grad():
            call(name)


@pytest.mark.parametrize("call,name", CALLS)
def test_the_warning_names_the_caller_s_line(call, name):
    """Else a program sees it once, from this library's own line, for all of its calls."""
    with warnings.catch_warnings(record=True) as seen:
        warnings.simplefilter("always")
        call(name)
    assert [w.filename for w in seen] == [__file__]
