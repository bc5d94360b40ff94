"""Pins of oracle/layer.py: gradients against central differences, the 4-bit grid
and its ties by hand, and the rule of a block's scale over many magnitudes."""
import numpy as np
import pytest

from oracle import layer


def _diff(f, x, d, eps=1e-5):
    return (f(x + eps * d) - f(x - eps * d)) / (2 * eps)


@pytest.mark.parametrize("kind", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("per_head", [False, True])
def test_gated_gradients(kind, gate_first, per_head):
    r = np.random.default_rng(1)
    x, z, dy = (r.normal(size=(3, 4, 10)) for _ in range(3))
    w = 1 + 0.1 * r.normal(size=(4, 10) if per_head else (10,))
    got = layer.gated_norm_backward(x, z, w, dy, 1e-3, kind, gate_first)

    def loss(x=x, z=z, w=w):
        return (layer.gated_norm(x, z, w, 1e-3, kind, gate_first) * dy).sum()

    for g, (name, v) in zip(got, (("x", x), ("z", z), ("w", w))):
        assert g.shape == v.shape
        for _ in range(3):
            d = r.normal(size=v.shape)
            # central differences: 1e-10 of the third derivative, 1e-16 / 1e-5 of the value
            assert abs(_diff(lambda y: loss(**{name: y}), v, d) - (g * d).sum()) < 1e-7


@pytest.mark.parametrize("kind", [None, "none", "silu", "sigmoid"])
@pytest.mark.parametrize("post", [False, True])
def test_block_gradients(kind, post):
    r = np.random.default_rng(2)
    x, res, dy, dh = (r.normal(size=(5, 12)) for _ in range(4))
    z = None if kind is None else r.normal(size=(5, 12))
    w = 1 + 0.1 * r.normal(size=12) if post else None
    wn = 1 + 0.1 * r.normal(size=12)

    def loss(x=x, res=res, z=z, w=w, wn=wn):
        h = layer.block_sum(x, res, w, 1e-3, 0.7, z, kind)
        return (layer.block_norm(h, wn, 1e-3) * dy).sum() + (h * dh).sum()

    h = layer.block_sum(x, res, w, 1e-3, 0.7, z, kind)
    got = layer.block_norm_backward(x, h, w, wn, dy, 1e-3, 0.7, z, kind, dh)
    for key, name, v in (("dx", "x", x), ("dres", "res", res), ("dgate", "z", z), ("dw", "w", w), ("dwn", "wn", wn)):
        if v is None:
            assert got[key] is None
            continue
        for _ in range(3):
            d = r.normal(size=v.shape)
            assert abs(_diff(lambda y: loss(**{name: y}), v, d) - (got[key] * d).sum()) < 1e-7


def test_block_without_gate_or_weights_is_the_plain_norm():
    from oracle import sequence
    r = np.random.default_rng(3)
    x, res, w = r.normal(size=(4, 9)), r.normal(size=(4, 9)), r.normal(size=9)
    h = layer.block_sum(x, res, None, 1e-6, 1.0, None, None)
    np.testing.assert_array_equal(h, x + res)
    np.testing.assert_allclose(layer.block_norm(h, w, 1e-6), sequence.rmsnorm(h, w, 1e-6)[0], rtol=1e-14)


def test_grid_and_ties():
    x = np.zeros(32)
    x[:16] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -5, 0.2500001, 0.74, 5.0001, 0.1, 2.51, -6]
    c, e = layer.mx_quant(x[None])
    assert e[0, 0] == 127
    assert c[0, :16].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8, 14, 1, 1, 7, 0, 5, 15]


@pytest.mark.parametrize("top,e", [(6.0, 0), (6.99, 0), (7.0, 1), (8.0, 1), (13.9, 1), (14.0, 2), (3.5, 0), (3.49, -1),
                                   (2.0 ** -126, -127), (2.0 ** -130, -127), (0.0, -127), (3.0e38, 126)])
def test_scale_rule(top, e):
    x = np.zeros(32, np.float32)
    x[5] = -top
    c, got = layer.mx_quant(x[None])
    assert int(got[0, 0]) - 127 == e


def test_largest_is_rounded_not_cut():
    """Every value q (in units of 2^e) is within a fifth of its block's largest
    magnitude m of its place on the grid.  m is at least 3.5 units.  Below 4 units a
    step is at most 1, so the error is at most 0.5 <= m / 7.  From 4 to 6 it is at most
    min(q - 4, 6 - q), at most 1 at q = 5, where m >= 5; from 6 to 7 at most q - 6 < 1 <= m / 6."""
    r = np.random.default_rng(4)
    x = (r.normal(size=(500, 64)) * np.exp(4 * r.normal(size=(500, 1)))).astype(np.float32).astype(np.float64)
    v = layer.mx_values(*layer.mx_pack(*layer.mx_quant(x)))
    b, q = x.reshape(-1, 32), v.reshape(-1, 32)
    assert (np.abs(b - q).max(-1) <= np.abs(b).max(-1) / 5).all()


def test_not_finite():
    x = np.ones((2, 64), np.float32)
    x[0, 3], x[1, 40] = np.nan, -np.inf
    c, e = layer.mx_quant(x)
    assert e.tolist() == [[255, 125], [125, 255]]
    assert (c[0, :32] == 0).all() and (c[1, 32:] == 0).all()
    v = layer.mx_values(*layer.mx_pack(c, e))
    assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 1).all()
