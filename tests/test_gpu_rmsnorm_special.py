"""8-bit outputs of lores_rmsnorm where a value or a weight is not a number, rows
are zero without an epsilon, or their largest value is next to nothing.

What is not finite has to show: such a row's scale is NaN and its codes are 0.
For all others scale x code is y to half a step of the code (int8), or to E4M3's
2^-4 of the value or half its smallest step, 2^-10.  Besides that half step
there are a handful of fp32 roundings: 2^-20.
"""
import numpy as np
import pytest
import torch

import quantized_linear_recurrence_amd as lores
from oracle import sequence as oseq

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
EIGHT = [lores.LORES_INT8, lores.LORES_FP8]
WIDTHS = [96, 101, 500, 1000, 2000, 4000, 8000, 16000]          # every number of threads a row takes
NAN, INF = float("nan"), float("inf")


def rows(r, n, dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(r, n, generator=g).to(dtype).to("cuda:0")


def ones(n, dtype=F32):
    return torch.ones(n, dtype=dtype, device="cuda:0")


def is_lost(y, s):
    return bool(torch.isnan(s).all() and (y.float() == 0).all())


def check_values(x, w, eps, prec):
    y, s, _ = lores.lores_rmsnorm(x, w, eps, out_prec=prec)
    want, _ = oseq.rmsnorm(x.double().cpu().numpy(), w.double().cpu().numpy(), eps)
    s = s.double().cpu().numpy()[:, None]
    assert np.isfinite(s).all()
    off = np.abs(y.double().cpu().numpy() * s - want)
    most = 0.5 * s if prec == lores.LORES_INT8 else np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * s)
    assert (off <= most * (1 + 2.0 ** -20) + 2.0 ** -20 * np.abs(want)).all()


@pytest.mark.parametrize("prec", EIGHT)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", WIDTHS)
def test_a_weight_that_is_not_finite_shows(n, dtype, prec):
    x = rows(5, n, dtype)
    x[4] = 0.0
    for bad in (NAN, INF, -INF):
        for at in (0, n // 2, n - 1):
            w = ones(n, dtype)
            w[at] = bad
            y, s, _ = lores.lores_rmsnorm(x, w, 1e-6, out_prec=prec)
            assert is_lost(y, s), (bad, at)


@pytest.mark.parametrize("prec", EIGHT)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", WIDTHS)
def test_a_row_that_is_not_finite_shows_under_any_weight(n, dtype, prec):
    for weight in (0.0, 1.0):
        for bad in (NAN, INF, -INF):
            x, w = rows(4, n, dtype), ones(n, dtype)
            w[n - 1] = weight
            x[1, n - 1] = x[2, n - 1] = bad
            y, s, _ = lores.lores_rmsnorm(x, w, 1e-6, out_prec=prec)
            assert is_lost(y[1:3], s[1:3]), (bad, weight)
            assert torch.isfinite(s[[0, 3]]).all()
            check_values(x[[0, 3]], w, 1e-6, prec)


@pytest.mark.parametrize("prec", EIGHT)
@pytest.mark.parametrize("n", WIDTHS)
def test_a_row_whose_squares_leave_fp32_shows(n, prec):
    x = rows(3, n, BF16)
    x[1] = 2.0 ** 66
    y, s, _ = lores.lores_rmsnorm(x, ones(n, BF16), 1e-6, out_prec=prec)
    assert is_lost(y[1:2], s[1:2]) and torch.isfinite(s[[0, 2]]).all()


@pytest.mark.parametrize("prec", EIGHT)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", WIDTHS)
def test_rows_of_zeros_without_an_epsilon(n, dtype, prec):
    x = rows(3, n, dtype)
    x[1] = 0.0
    y, s, _ = lores.lores_rmsnorm(x, ones(n, dtype), 0.0, out_prec=prec)
    assert float(s[1]) == 0.0 and (y[1].float() == 0).all()
    check_values(x[[0, 2]], ones(n, dtype), 0.0, prec)
    y, s, _ = lores.lores_rmsnorm(x, torch.zeros_like(ones(n, dtype)), 0.0, out_prec=prec)
    assert (s == 0).all() and (y.float() == 0).all()


@pytest.mark.parametrize("prec", EIGHT)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", WIDTHS)
def test_scale_times_code_is_the_value_for_tiny_rows(n, dtype, prec):
    e = torch.tensor([-126.0, -125.0, -123.0, -120.0, -119.5, -119.0, -118.0, -100.0]).to("cuda:0")
    x = rows(len(e), n, F32)
    x = (x / x.abs().amax(1, keepdim=True) * torch.exp2(e)[:, None]).to(dtype)
    check_values(x, ones(n, dtype), 1e-6, prec)
