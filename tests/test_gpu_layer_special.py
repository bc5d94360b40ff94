"""Values of the layer operators' rows that are not finite, tiny or far, against the fp64
oracle element by element."""
import numpy as np
import pytest
import torch

import quantized_linear_recurrence_amd as lores
from tests.layer_common import BF16, DW, EPS, F32, TOL, arr, blocks_near, randn, weight
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


# A gate's element alone: a row of equal values whose r takes 3 roundings of 2^-24; the
# gate's exponential and reciprocal take 2 each (1 ulp), its factor and sum 3, and the
# products 4: fewer than 16, 2^-20.  Results down to 2^-126 are not subnormal for |z| <= 80.
GATE = 2.0 ** -20


def far(dtype, n):
    return torch.linspace(-80.0, 80.0, 24 * n).to(dtype).view(24, 1, n).to("cuda:0")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["silu", "sigmoid"])
def test_gates_in_fp32_results(dtype, kind):
    """fp32 results of bf16 and fp32 gates alike, element by element: y, and dw of one token."""
    n = 128
    z, act = far(dtype, n), {"silu": lores.LORES_ACT_SILU, "sigmoid": lores.LORES_ACT_SIGMOID}[kind]
    x, w = torch.ones_like(z), torch.full((n,), 0.75, dtype=dtype, device=z.device)
    y, _ = lores.lores_gated_norm(x, z, w, 1.0, act=act, out_prec=lores.LORES_FP32)
    want = layer.gated_norm(arr(x), arr(z), arr(w), 1.0, kind, False)
    assert (np.abs(arr(y) - want) <= GATE * np.abs(want)).all(), np.max(np.abs(arr(y) / want - 1))
    for t in range(24):
        _, _, dw = lores.lores_gated_norm_backward(x[t:t + 1], z[t:t + 1], w, x[t:t + 1], 1.0, act=act)
        want = layer.gated_norm_backward(arr(x[t:t + 1]), arr(z[t:t + 1]), arr(w), arr(x[t:t + 1]), 1.0, kind, False)[2]
        assert (np.abs(arr(dw) - want) <= GATE * np.abs(want)).all(), np.max(np.abs(arr(dw) / want - 1))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["silu", "sigmoid"])
def test_gates_in_a_block_s_fp32_gradient(dtype, kind):
    """dw of one row whose G is dh alone (dy 0), of x in equal values: dw = scale dh a(z) r."""
    n = 128
    z, act = far(dtype, n)[:, 0], {"silu": lores.LORES_ACT_SILU, "sigmoid": lores.LORES_ACT_SIGMOID}[kind]
    x, w = torch.ones_like(z), torch.full((n,), 0.75, dtype=dtype, device=z.device)
    for t in range(24):
        a, g, zero = x[t:t + 1], z[t:t + 1], torch.zeros_like(x[t:t + 1])
        dw = lores.lores_block_norm_backward(a, a, w, w, zero, 1.0, scale=0.5, gate=g, act=act, dh=a)[3]
        want = layer.block_norm_backward(arr(a), arr(a), arr(w), arr(w), arr(zero), 1.0, 0.5, arr(g), kind, arr(a))["dw"]
        assert (np.abs(arr(dw) - want) <= GATE * np.abs(want)).all(), np.max(np.abs(arr(dw) / want - 1))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_infinite_and_largest_gates(dtype):
    z = torch.tensor([INF, -INF, float("nan"), 3e38, -3e38, 1e6, -1e6, 160.0, -160.0], device="cuda:0").to(dtype).view(9, 1, 1)
    x, w = torch.ones_like(z), torch.ones(1, dtype=dtype, device=z.device)
    s = lores.lores_gated_norm(x, z, w, 0.0, act=lores.LORES_ACT_SIGMOID, out_prec=lores.LORES_FP32)[0].flatten().tolist()
    assert s[0] == s[3] == s[5] == s[7] == 1.0 and s[1] == s[4] == s[6] == s[8] == 0.0 and s[2] != s[2]
    y = lores.lores_gated_norm(x, z, w, 0.0, out_prec=lores.LORES_FP32)[0].flatten().tolist()
    assert y[0] == INF and y[2] != y[2] and y[3:] == [float(z[3]), 0.0, float(z[5]), 0.0, float(z[7]), 0.0]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [32, 96, 128, 1024, 4096, 16384])
@pytest.mark.parametrize("eps", [1e-6, 1e-30])
def test_4_bit_rows_of_tiny_values(dtype, n, eps):
    """Rows whose squares are below fp32 (or add up to less than eps) but not their values: r is eps^-1/2."""
    x, z, w = 1e-30 * randn((3, 2, n), F32, 1), randn((3, 2, n), dtype, 2), weight((n,), dtype, 3)
    x = x.to(dtype)
    closed = (-60.0 + randn((3, 2, n), F32, 4)).to(dtype)      # a(z) near 1e-26 (sigmoid), -6e-25 (silu)
    for kind in ("silu", "sigmoid"):
        for a, g, first in ((x, z, False), (x, z, True), (randn((3, 2, n), dtype, 5), closed, True),
                            (randn((3, 2, n), dtype, 5), closed, False)):
            act = {"silu": lores.LORES_ACT_SILU, "sigmoid": lores.LORES_ACT_SIGMOID}[kind]
            c, s = lores.lores_gated_norm(a, g, w, eps, act=act, gate_first=first, out_prec=lores.LORES_MXFP4)
            want = layer.gated_norm(arr(a), arr(g), arr(w), eps, kind, first).reshape(3, -1)
            assert (np.abs(want) > 0).all()
            blocks_near(c, s, want, f"{kind}, {first}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [32, 128, 1024, 4096, 16384])
def test_4_bit_rows_without_an_epsilon(dtype, n):
    """Zeros have codes and scales of 0; rows whose squares are below fp32 have no r and NaN scales, as fp32
    outputs there are not finite.  The block norm's answers are the same."""
    x, z, w = torch.zeros(5, 1, n, dtype=dtype, device="cuda:0"), randn((5, 1, n), dtype, 2), weight((n,), dtype, 3)
    x[1] = 1e-30
    x[2, 0, n // 2] = -1e-30
    x[3] = randn((1, n), dtype, 4)
    x[4] = -0.0
    c, s = lores.lores_gated_norm(x, z, w, 0.0, out_prec=lores.LORES_MXFP4)
    y, _ = lores.lores_gated_norm(x, z, w, 0.0, out_prec=lores.LORES_FP32)
    assert not torch.isfinite(y[1:3]).any() and torch.isfinite(y[3]).all()
    blocks = n // 32
    for c, s in ((c, s), lores.lores_block_norm(x[:, 0], None, None, w, 0.0, out_prec=lores.LORES_MXFP4)[:2]):
        assert (c[[0, 4]] & 0x77 == 0).all() and (s[[0, 4]] == 0).all()
        assert (s[1:3, :blocks] == 255).all() and (c[1:3] == 0).all() and (s[3, :blocks] < 255).all()
    z[1, 0, 1] = float("nan")                        # 0 times NaN stays
    c, s = lores.lores_gated_norm(torch.zeros_like(x), z, w, 0.0, out_prec=lores.LORES_MXFP4)
    assert s[1, 0] == 255 and (s[1, 1:] == 0).all() and (s[[0, 2, 3, 4]] == 0).all()
    c, s = lores.lores_gated_norm(x, z, w, 0.0, gate_first=True, out_prec=lores.LORES_MXFP4)
    assert (s[1, :blocks] == 255).all() and (s[0] == 0).all()
