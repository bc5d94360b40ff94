"""Values of the layer operators' rows that are not finite, tiny or far, against the fp64
oracle element by element."""
import numpy as np
import pytest
import torch

import quantized_linear_recurrence_amd as lores
from tests.layer_common import BF16, DW, EPS, F32, TOL, arr, randn, weight
from oracle import layer

pytestmark = pytest.mark.gpu
INF = float("inf")


def like(got, want, tol, what):
    """NaNs and infinities where the formula has them, and the rest near it in the 2-norm."""
    got = arr(got)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want), err_msg=what)
    lost = np.isinf(want)
    np.testing.assert_array_equal(got[lost], want[lost], err_msg=what)
    fine = np.isfinite(want)
    assert np.isfinite(got[fine]).all(), what
    err, size = np.linalg.norm(got[fine] - want[fine]), np.linalg.norm(want[fine])
    assert err <= tol * size + 1e-30, f"{what}: {err / max(size, 1e-300):.3g} > {tol:.3g}"


# Rows of whole vectors, and of those that end with a vector over part of its
# neighbour's (from n - 8 to the last multiple of 8); an element in that part, the last
# one before it, the row's last and its first.
WIDTHS = [96, 100, 130, 1030, 4100, 8204, 16380]


def places(n):
    return sorted({0, n - 9, n - 8, max(n - 8, (n - 1) // 8 * 8 - 1), n - 1})


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("first", [False, True])
def test_one_infinity_in_a_gated_row(dtype, n, first):
    z, w, dy = randn((3, 2, n), dtype, 2), weight((n,), dtype, 3), randn((3, 2, n), dtype, 4)
    for at in places(n):
        x, g = randn((3, 2, n), dtype, 1), dy.clone()
        x[1, 0, at] = INF
        g[2, 1, at] = -INF
        kw = {"act": lores.LORES_ACT_SIGMOID, "gate_first": first}
        y, _ = lores.lores_gated_norm(x, z, w, EPS, **kw)
        with np.errstate(invalid="ignore"):
            want = layer.gated_norm(arr(x), arr(z), arr(w), EPS, "sigmoid", first)
            grads = [layer.gated_norm_backward(arr(a), arr(z), arr(w), arr(b), EPS, "sigmoid", first)
                     for a, b in ((x, dy), (randn((3, 2, n), dtype, 1), g))]
        like(y, want, TOL[dtype], f"y, {at}")
        for a, b, v in ((x, dy, grads[0]), (randn((3, 2, n), dtype, 1), g, grads[1])):
            for got, ref, name, tol in zip(lores.lores_gated_norm_backward(a, z, w, b, EPS, **kw), v,
                                           ("dx", "dgate", "dw"), (TOL[dtype], TOL[dtype], DW)):
                like(got, ref, tol, f"{name}, {at}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", WIDTHS)
def test_one_infinity_in_a_block_s_row(dtype, n):
    w, wn, gate = weight((n,), dtype, 3), weight((n,), dtype, 4), randn((3, n), dtype, 5)
    dy, dh = randn((3, n), dtype, 6), randn((3, n), dtype, 7)
    kw = {"scale": 0.5, "gate": gate, "act": lores.LORES_ACT_SIGMOID}
    for at in places(n):
        def row(seed, row=None):
            t = randn((3, n), dtype, seed)
            if row is not None:
                t[row, at] = INF
            return t

        for post in (None, w):
            x, r = row(1, 1), row(2)
            y, _, h = lores.lores_block_norm(x, r, post, wn, EPS, **kw)
            with np.errstate(invalid="ignore"):
                like(h, layer.block_sum(arr(x), arr(r), arr(post), EPS, 0.5, arr(gate), "sigmoid"), TOL[dtype], f"h, {at}")
                like(y, layer.block_norm(arr(h), arr(wn), EPS), TOL[dtype], f"y, {at}")
            for a, b, c, d in ((row(1, None if post is None else 1), row(8), dy, dh), (row(1), row(8, 0), dy, dh),
                               (row(1), row(8), row(6, 2), dh), (row(1), row(8), dy, row(7, 1))):
                got = lores.lores_block_norm_backward(a, b, post, wn, c, EPS, dh=d, **kw)
                with np.errstate(invalid="ignore"):
                    want = layer.block_norm_backward(arr(a), arr(b), arr(post), arr(wn), arr(c), EPS, 0.5, arr(gate),
                                                     "sigmoid", arr(d))
                for v, name, tol in zip(got, ("dx", "dres", "dgate", "dw", "dwn"), [TOL[dtype]] * 3 + [DW] * 2):
                    if want[name] is not None:
                        like(v, want[name], tol, f"{name}, {at}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [1, 96, 100, 1030, 16380])
@pytest.mark.parametrize("value", [INF, -INF, float("nan")])
def test_a_row_that_is_not_finite_without_a_weight_has_a_gradient(dtype, n, value):
    """dx = scale a(gate) G has no x in it."""
    wn, gate, h = weight((n,), dtype, 4), randn((3, n), dtype, 5), randn((3, n), dtype, 8)
    x, dy, dh = randn((3, n), dtype, 1), randn((3, n), dtype, 6), randn((3, n), dtype, 7)
    want = lores.lores_block_norm_backward(x, h, None, wn, dy, 0.5, scale=0.5, gate=gate, act=lores.LORES_ACT_SIGMOID, dh=dh)
    x[1, n // 2] = value
    got = lores.lores_block_norm_backward(x, h, None, wn, dy, 0.5, scale=0.5, gate=gate, act=lores.LORES_ACT_SIGMOID, dh=dh)
    assert torch.isfinite(want[0]).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[4], want[4])
    ref = layer.block_norm_backward(arr(x), arr(h), None, arr(wn), arr(dy), 0.5, 0.5, arr(gate), "sigmoid", arr(dh))
    like(got[0], ref["dx"], TOL[dtype], "dx")
    like(got[2], ref["dgate"], TOL[dtype], "dgate")
