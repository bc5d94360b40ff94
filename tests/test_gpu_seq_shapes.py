"""The sequence operators refuse tensors that have the right number of elements in
another order of dimensions: they would be read in the wrong order."""
import pytest
import torch

import quantized_linear_recurrence_amd as lores

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
B, T, H, HK, DK, DV = 2, 12, 4, 2, 64, 32


def _inputs():
    z = lambda *s: torch.zeros(*s, device=DEV)                       # noqa: E731
    return {"q": z(B, T, HK, DK), "k": z(B, T, HK, DK), "v": z(B, T, H, DV), "alpha": z(B, T, H),
            "beta": z(B, T, H), "S0": z(B, H, DV, DK), "lengths": torch.full((B,), T, dtype=torch.int32, device=DEV),
            "o": z(B, T, H, DV), "S": z(B, H, DV, DK), "do": z(B, T, H, DV), "dS": z(B, H, DV, DK)}


def _scan(x):
    return lores.lores_scan(x["q"], x["k"], x["v"], x["alpha"], x["beta"], 1, S0=x["S0"], lengths=x["lengths"],
                            o=x["o"], S=x["S"])


def _back(x):
    return lores.lores_scan_backward(x["q"], x["k"], x["v"], x["alpha"], x["beta"], 1, x["do"], dS=x["dS"],
                                     S0=x["S0"], lengths=x["lengths"])


ORDERS = {"alpha": [(B, H, T), (T, B, H), (B * T, H), (B * T * H,)], "beta": [(B, H, T), (B, T, H, 1)],
          "S0": [(B, H, DK, DV), (H, B, DV, DK), (B * H, DV, DK)], "lengths": [(B, 1), (1, B)],
          "o": [(B, H, T, DV), (B, T, H * DV)], "S": [(B, H, DK, DV), (B * H, DV, DK)],
          "do": [(B, H, T, DV), (B, T, DV, H)], "dS": [(B, H, DK, DV)]}


@pytest.mark.parametrize("name", list(ORDERS))
def test_scan_takes_no_other_order(name):
    x = _inputs()
    _scan(x), _back(x)
    for shape in ORDERS[name]:
        y = {**x, name: x[name].reshape(shape)}
        calls = ((_scan,) if name in ("o", "S") else (_back,) if name in ("do", "dS") else (_scan, _back))
        for call in calls:
            with pytest.raises(ValueError, match=name):
                call(y)


def test_norm_takes_no_other_order():
    x, w = torch.zeros(6, 4, 64, device=DEV), torch.ones(64, device=DEV)
    lores.lores_rmsnorm(x, w, 1e-6)
    lores.lores_rmsnorm_backward(x, w, x, 1e-6, dresidual=x)
    for bad in (w.view(1, 64), w.view(64, 1)):
        with pytest.raises(ValueError, match="weight"):
            lores.lores_rmsnorm(x, bad, 1e-6)
    for shape in ((4, 6, 64), (24, 64), (6, 64, 4)):
        with pytest.raises(ValueError, match="dy"):
            lores.lores_rmsnorm_backward(x, w, x.reshape(shape), 1e-6)
        with pytest.raises(ValueError, match="dresidual"):
            lores.lores_rmsnorm_backward(x, w, x, 1e-6, dresidual=x.reshape(shape))
