"""lores_rmsnorm and lores_rmsnorm_backward on the GPU against the fp64 oracle.

Tolerances (2-norms): a row's sum of squares is reduced in fp32 by up to 16
steps per lane and 10 across lanes, its root and quotient are correctly rounded:
fewer than 64 roundings of 2^-24, 2^-18.  bf16 results add 2^-9 per element.
The codes of 8-bit outputs depend on elementwise fp32 operations alone and are
equal.  dw adds up to 2^16 products in fp32: 2^-17.
"""
import numpy as np
import pytest
import torch

import quantized_linear_recurrence_amd as lores
from oracle import sequence as oseq

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 2.0 ** -18, BF16: 2.0 ** -9 + 2.0 ** -17}
EPS = 1e-6


def _dev():
    return torch.device("cuda:0")


def _np(t):
    return t.detach().double().cpu().numpy()


def near(got, want, tol, what):
    got = _np(got)
    assert got.shape == want.shape, what
    assert np.isfinite(got).all(), what
    err, size = np.linalg.norm(got - want), np.linalg.norm(want)
    assert err <= tol * size + 1e-30, f"{what}: {err / max(size, 1e-300):.3g} > {tol:.3g}"


def rows(r, n, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(r, n, generator=g)).to(dtype).to(_dev())


def weight(n, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (1.0 + 0.2 * torch.randn(n, generator=g)).to(dtype).to(_dev())


def check(x, w, res, out_prec):
    y, scales, h = lores.lores_rmsnorm(x, w, EPS, residual=res, out_prec=out_prec)
    if res is None:
        assert h is x
    else:
        assert torch.equal(h, (x.float() + res.float()).to(x.dtype))
    yr, r = oseq.rmsnorm(_np(h), _np(w), EPS)
    if out_prec in (lores.LORES_INT8, lores.LORES_FP8):
        top = 127.0 if out_prec == lores.LORES_INT8 else 448.0
        c, m = oseq.rmsnorm_codes(h.float().cpu().numpy(), w.float().cpu().numpy(), top)
        if out_prec == lores.LORES_INT8:
            assert y.dtype == torch.int8
            np.testing.assert_array_equal(y.cpu().numpy(), np.rint(c).astype(np.int8))
        else:
            want = torch.from_numpy(np.clip(c, -448, 448)).to(torch.float8_e4m3fn)
            assert torch.equal(y.cpu().view(torch.uint8), want.view(torch.uint8))
        near(scales, m.astype(np.float64) * r / top, TOL[F32], "scales")
    else:
        assert scales is None
        near(y, yr, TOL[y.dtype], "y")
    return h


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [1, 7, 8, 64, 100, 128, 129, 512, 515, 1024, 1030, 2048, 2056, 4096,
                               4100, 8192, 8200, 16384])
def test_forward_widths(dtype, n):
    for r, res, prec in ((5, True, None), (1, False, lores.LORES_INT8), (19, True, lores.LORES_INT8),
                         (6, True, lores.LORES_FP8), (3, False, lores.LORES_FP32),
                         (3, False, lores.LORES_BF16)):
        x = rows(r, n, dtype, n)
        check(x, weight(n, dtype, 1), rows(r, n, dtype, n + 1, 3.0) if res else None, prec)


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("wt", [F32, BF16])
def test_weight_types_and_shapes(xt, wt):
    x = rows(24, 96, xt, 2).view(2, 3, 4, 96)
    y, s, h = lores.lores_rmsnorm(x, weight(96, wt, 3), EPS, out_prec=lores.LORES_INT8)
    assert y.shape == x.shape and s.shape == x.shape[:-1] and h is x
    check(x.view(24, 96), weight(96, wt, 3), None, None)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [64, 200, 4096])
def test_strides_and_alignment(dtype, n):
    wide = rows(9, 2 * n + 3, dtype, 4)
    for x, res in ((wide[:, 1:1 + n], wide[:, n + 2:2 * n + 2]), (wide[::2, :n], None)):
        w = weight(n + 1, dtype, 5)[1:]
        for prec in (None, lores.LORES_INT8, lores.LORES_FP8):
            check(x, w, res, prec)


def test_rows_that_are_zero_tiny_or_not_finite():
    x = rows(6, 256, F32, 6)
    x[0] = 0.0
    x[1] = 1e-38
    x[2, 3] = float("inf")
    x[3, 200] = float("nan")
    x[4] *= 1e15
    w = weight(256, F32, 7)
    for prec in (lores.LORES_INT8, lores.LORES_FP8):
        y, s, _ = lores.lores_rmsnorm(x, w, EPS, out_prec=prec)
        y = y.float()
        assert torch.isfinite(y).all()
        assert (y[0] == 0).all() and float(s[0]) == 0.0
        assert torch.isnan(s[2]) and torch.isnan(s[3])
        assert torch.isfinite(s[[0, 1, 4, 5]]).all()
    y, _, _ = lores.lores_rmsnorm(x, w, EPS)
    keep = [0, 4, 5]
    near(y[keep], oseq.rmsnorm(_np(x[keep]), _np(w), EPS)[0], TOL[F32], "y")
    assert torch.isnan(y[3]).all()                   # NaN in the mean
    assert torch.isfinite(y[1]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("r,n", [(1, 1), (1, 64), (7, 100), (33, 128), (5, 515), (300, 1024),
                                 (70, 2056), (2100, 4096), (9, 4100), (11, 8192), (520, 8200),
                                 (3, 16384)])
def test_backward(dtype, r, n):
    h, w = rows(r, n, dtype, r + n, 2.0), weight(n, dtype, 8)
    dy = rows(r, n, dtype, r + n + 1)
    for dres in (None, rows(r, n, dtype, r + n + 2)):
        eps = 0.5 if n == 1 else EPS                 # a row of one element has dx = eps r^3 w dy
        dx, dw = lores.lores_rmsnorm_backward(h, w, dy, eps, dresidual=dres)
        rx, rw = oseq.rmsnorm_backward(_np(h), _np(w), eps, _np(dy), None if dres is None else _np(dres))
        near(dx, rx, TOL[dtype], "dx")
        near(dw, rw, 2.0 ** -17, "dw")
        again = lores.lores_rmsnorm_backward(h, w, dy, eps, dresidual=dres)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("r,n", [(8193, 100), (9001, 128), (2050, 130), (2101, 1024), (1100, 2048)])
def test_backward_with_more_rows_than_work_groups_take_at_once(dtype, r, n):
    h, w, dy = rows(r, n, dtype, r + n, 2.0), weight(n, dtype, 8), rows(r, n, dtype, r + n + 1)
    dx, dw = lores.lores_rmsnorm_backward(h, w, dy, EPS)
    rx, rw = oseq.rmsnorm_backward(_np(h), _np(w), EPS, _np(dy), None)
    near(dx, rx, TOL[dtype], "dx")
    near(dw, rw, 2.0 ** -17, "dw")
    again = lores.lores_rmsnorm_backward(h, w, dy, EPS)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_gradient_matches_differences():
    h, w, dy = rows(5, 130, F32, 20), weight(130, F32, 21), rows(5, 130, F32, 22)
    dx, dw = lores.lores_rmsnorm_backward(h, w, dy, EPS)
    loss = lambda h, w: float((lores.lores_rmsnorm(h, w, EPS)[0].double() * dy.double()).sum())  # noqa: E731
    e = 2.0 ** -7                                    # truncation 2^-14, rounding 2^-18 / 2^-7
    for x, g, f in ((h, dx, lambda x: loss(x, w)), (w, dw, lambda x: loss(h, x))):
        d = rows(x.numel(), 1, F32, 23).view(x.shape)
        num = (f(x + e * d) - f(x - e * d)) / (2 * e)
        size = float(g.double().norm() * d.double().norm())
        assert abs(num - float((g.double() * d.double()).sum())) <= 2.0 ** -10 * size


def test_streams_and_no_rows():
    x, w = rows(64, 512, BF16, 30), weight(512, BF16, 31)
    want = lores.lores_rmsnorm(x, w, EPS, residual=x, out_prec=lores.LORES_INT8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = lores.lores_rmsnorm(x, w, EPS, residual=x, out_prec=lores.LORES_INT8, stream=s)
    grad = lores.lores_rmsnorm_backward(x, w, x, EPS, stream=s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for a, b in zip(grad, lores.lores_rmsnorm_backward(x, w, x, EPS)):
        assert torch.equal(a, b)
    y, sc, _ = lores.lores_rmsnorm(x[:0], w, EPS, out_prec=lores.LORES_INT8)
    assert y.shape == (0, 512) and sc.shape == (0,)
    dx, dw = lores.lores_rmsnorm_backward(x[:0], w, x[:0], EPS)
    assert dx.shape == (0, 512) and (dw == 0).all()


def test_refusals():
    x, w = rows(4, 64, F32, 40), weight(64, F32, 41)
    for bad in ((x.half(), w), (x, w.half()), (None, w), (x, None)):
        with pytest.raises(TypeError):
            lores.lores_rmsnorm(*bad, EPS)
    for bad in ((x.cpu(), w), (x, w[:32]), (x.t(), weight(4, F32, 1)), (x, w.cpu())):
        with pytest.raises(ValueError):
            lores.lores_rmsnorm(*bad, EPS)
    with pytest.raises(TypeError):
        lores.lores_rmsnorm(x, w, EPS, residual=x.to(BF16))
    with pytest.raises(ValueError):
        lores.lores_rmsnorm(x, w, EPS, residual=x[:2])
    with pytest.raises(ValueError):
        lores.lores_rmsnorm(x, w, EPS, out_prec=lores.LORES_INT4)
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(lores.LoresError):
            lores.lores_rmsnorm(x, w, eps)
    big = torch.zeros(1, lores.LORES_MAX_NORM + 1, device=_dev())
    with pytest.raises(lores.LoresError):
        lores.lores_rmsnorm(big, big[0], EPS)
    with pytest.raises(TypeError):
        lores.lores_rmsnorm_backward(x, w, x.to(BF16), EPS)
    with pytest.raises(ValueError):
        lores.lores_rmsnorm_backward(x, w, x[:2], EPS)
