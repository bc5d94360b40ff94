"""lores_gated_norm and its gradient against the fp64 oracle (tolerances: layer_common)."""
import pytest
import torch

import quantized_linear_recurrence_amd as lores
from tests.layer_common import BF16, DW, EPS, F32, TOL, arr, blocks_near, dev, near, randn, weight
from oracle import layer

pytestmark = pytest.mark.gpu
ACTS = {"none": lores.LORES_ACT_NONE, "silu": lores.LORES_ACT_SILU, "sigmoid": lores.LORES_ACT_SIGMOID}


def forward(x, z, w, kind, first, prec=None, eps=EPS):
    y, s = lores.lores_gated_norm(x, z, w, eps, act=ACTS[kind], gate_first=first, out_prec=prec)
    want = layer.gated_norm(arr(x), arr(z), arr(w), eps, kind, first)
    if prec == lores.LORES_MXFP4:
        lead = x.shape[:-2]
        blocks_near(y, s, want.reshape(*lead, -1), "codes")
    else:
        assert s is None
        near(y, want, TOL[y.dtype], "y")


def backward(x, z, w, kind, first, eps=EPS, seed=9):
    dy = randn(x.shape, x.dtype, seed)
    got = lores.lores_gated_norm_backward(x, z, w, dy, eps, act=ACTS[kind], gate_first=first)
    want = layer.gated_norm_backward(arr(x), arr(z), arr(w), arr(dy), eps, kind, first)
    for g, v, name, tol in zip(got, want, ("dx", "dgate", "dw"), (TOL[x.dtype], TOL[x.dtype], DW)):
        near(g, v, tol, name)
    again = lores.lores_gated_norm_backward(x, z, w, dy, eps, act=ACTS[kind], gate_first=first)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [1, 7, 8, 64, 100, 128, 129, 512, 515, 1024, 1030, 2048, 2056, 4096, 4100, 8192, 8200,
                               16384])
def test_widths(dtype, n):
    eps = 0.5 if n == 1 else EPS                     # a row of one element has dx = eps r^3 e
    for tokens, heads, kind, first, per in ((3, 2, "silu", False, False), (1, 1, "sigmoid", True, False),
                                            (5, 3, "silu", True, True), (2, 5, "none", False, True)):
        x, z = randn((tokens, heads, n), dtype, n), randn((tokens, heads, n), dtype, n + 1, 1.5)
        w = weight((heads, n) if per else (n,), dtype, n + 2)
        forward(x, z, w, kind, first, eps=eps)
        backward(x, z, w, kind, first, eps=eps)


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("wt", [F32, BF16])
def test_types(xt, wt):
    x, z, w = randn((2, 3, 4, 96), xt, 1), randn((2, 3, 4, 96), xt, 2), weight((96,), wt, 3)
    for prec, dt in ((lores.LORES_FP32, F32), (lores.LORES_BF16, BF16), (None, xt)):
        y, _ = lores.lores_gated_norm(x, z, w, EPS, out_prec=prec)
        assert y.dtype is dt and y.shape == x.shape
        forward(x, z, w, "silu", False, prec)
    backward(x, z, w, "silu", True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("heads,n", [(1, 32), (3, 32), (4, 128), (5, 96), (2, 1024), (1, 4096), (3, 160)])
def test_blocks(dtype, heads, n):
    """A token's heads are one row of blocks; zeros stand behind the last of them."""
    x, z = randn((2, 7, heads, n), dtype, 11), randn((2, 7, heads, n), dtype, 12)
    for first, per in ((False, False), (True, True)):
        forward(x, z, weight((heads, n) if per else (n,), dtype, 13), "silu", first, lores.LORES_MXFP4)
    wide = randn((14, 2 * heads * n + 3), dtype, 14)
    odd = wide[:, 1:1 + heads * n].view(14, heads, n)
    forward(odd, wide[:, -heads * n:].view(14, heads, n), weight((n + 1,), dtype, 15)[1:], "sigmoid", False,
            lores.LORES_MXFP4)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [64, 100, 4096])
def test_strides(dtype, n):
    """Slices of a projection's rows, odd offsets, heads first, and broadcast gates."""
    wide = randn((6, 5 * n + 3), dtype, 21)
    w = weight((n + 1,), dtype, 22)[1:]
    x, z = wide[:, 1:1 + 2 * n].view(6, 2, n), wide[:, 2 * n + 2:4 * n + 2].view(6, 2, n)
    turned = randn((2, 6, n), dtype, 23).transpose(0, 1)
    for a, b in ((x, z), (turned, z), (x, randn((1, 1, n), dtype, 24).expand(6, 2, n)),
                 (x[::2], turned[::2]), (x[:, :1], z[:, 1:])):
        forward(a, b, w, "silu", False)
        backward(a, b, w, "silu", True)


def test_weights_per_head_are_their_own():
    x, z = randn((40, 6, 128), BF16, 31), randn((40, 6, 128), BF16, 32)
    w = weight((6, 128), BF16, 33)
    y, _ = lores.lores_gated_norm(x, z, w, EPS)
    for h in range(6):
        one, _ = lores.lores_gated_norm(x[:, h:h + 1], z[:, h:h + 1], w[h], EPS)
        assert torch.equal(one[:, 0], y[:, h])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,heads,n,per", [(4099, 5, 64, False), (1031, 33, 128, True), (2050, 3, 130, True),
                                                (2101, 2, 1024, False), (1100, 1, 2048, True)])
def test_gradients_of_more_rows_than_run_at_once(dtype, tokens, heads, n, per):
    x, z = randn((tokens, heads, n), dtype, 41), randn((tokens, heads, n), dtype, 42)
    backward(x, z, weight((heads, n) if per else (n,), dtype, 43), "silu", False)


@pytest.mark.parametrize("kind", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("first", [False, True])
def test_gradients_match_differences(kind, first):
    x, z, w = randn((3, 2, 130), F32, 51), randn((3, 2, 130), F32, 52), weight((2, 130), F32, 53)
    dy = randn((3, 2, 130), F32, 54)
    grads = lores.lores_gated_norm_backward(x, z, w, dy, EPS, act=ACTS[kind], gate_first=first)

    def loss(x=x, z=z, w=w):
        y, _ = lores.lores_gated_norm(x, z, w, EPS, act=ACTS[kind], gate_first=first)
        return float((y.double() * dy.double()).sum())

    e = 2.0 ** -7                                    # truncation 2^-14, rounding 2^-18 / 2^-7
    for name, v, g in (("x", x, grads[0]), ("z", z, grads[1]), ("w", w, grads[2])):
        d = randn(v.shape, F32, 55)
        num = (loss(**{name: v + e * d}) - loss(**{name: v - e * d})) / (2 * e)
        size = float(g.double().norm() * d.double().norm())
        assert abs(num - float((g.double() * d.double()).sum())) <= 2.0 ** -10 * size


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_far_gates(dtype):
    """Gates where the exponential over- or underflows, and small ones."""
    z = torch.tensor([0.0, -0.0, 1e-8, -1e-8, 20.0, -20.0, 80.0, -80.0, 100.0, -100.0, 3e4, -3e4, 1e30, -1e30, 0.5, -3.0],
                     device=dev()).to(dtype).repeat(2, 1, 2)
    x, w = randn((2, 1, 32), dtype, 61), weight((32,), dtype, 62)
    for kind in ("silu", "sigmoid"):
        y, _ = lores.lores_gated_norm(x, z, w, EPS, act=ACTS[kind])
        want = layer.gated_norm(arr(x), arr(z), arr(w), EPS, kind, False)
        # every element for itself; results below 2^-100 may be 0
        assert ((torch.from_numpy(want) - y.double().cpu()).abs()
                <= TOL[dtype] * torch.from_numpy(abs(want)) + 2.0 ** -100).all()
        dy = randn((2, 1, 32), dtype, 63)
        _, dz, _ = lores.lores_gated_norm_backward(x, z, w, dy, EPS, act=ACTS[kind])
        rz = torch.from_numpy(layer.gated_norm_backward(arr(x), arr(z), arr(w), arr(dy), EPS, kind, False)[1])
        # s (1 + z (1 - s)) near its zero at z = -1.28, and 1 - s beside 1, keep 2^-24 of their terms
        assert ((rz - dz.double().cpu()).abs() <= TOL[dtype] * rz.abs() + 2.0 ** -20).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_every_gate_has_a_value(dtype):
    """Gates on both sides of where the exponential leaves fp32's range (88.7), densely."""
    z = torch.linspace(-160.0, 160.0, 8192, device=dev()).to(dtype).view(64, 1, 128)
    x, w, dy = randn((64, 1, 128), dtype, 64), weight((128,), dtype, 65), randn((64, 1, 128), dtype, 66)
    for kind in ("silu", "sigmoid"):
        for first in (False, True):
            args = arr(x), arr(z), arr(w)
            y, _ = lores.lores_gated_norm(x, z, w, EPS, act=ACTS[kind], gate_first=first, out_prec=lores.LORES_FP32)
            want = torch.from_numpy(layer.gated_norm(*args, EPS, kind, first))
            # gated first, a row of gates of 2^-100 is one that is scaled up by 2^10 (eps 2^-20)
            assert ((want - y.double().cpu()).abs() <= TOL[dtype] * want.abs() + 2.0 ** -90).all()
            dx, dz, _ = lores.lores_gated_norm_backward(x, z, w, dy, EPS, act=ACTS[kind], gate_first=first)
            assert torch.isfinite(dx).all() and torch.isfinite(dz).all()


def test_a_gate_without_a_value_in_a_row_of_zeros():
    x, z, w = torch.zeros(2, 2, 64, device=dev()), randn((2, 2, 64), F32, 74), weight((64,), F32, 75)
    z[1, 1, 40] = float("nan")                       # 0 times NaN
    for eps in (EPS, 0.0):
        c, s = lores.lores_gated_norm(x, z, w, eps, out_prec=lores.LORES_MXFP4)
        assert s[1, 3] == 255 and (c & 0x77 == 0).all()
        s[1, 3] = 0
        assert (s == 0).all()


def test_values_that_are_not_finite():
    x, z, w = randn((6, 1, 64), F32, 71), randn((6, 1, 64), F32, 72), weight((64,), F32, 73)
    z[0, 0, 3] = float("inf")                        # s = 1
    z[1, 0, 3] = float("-inf")
    z[2, 0, 3] = float("nan")
    x[3, 0, 5] = float("nan")
    x[4] = 0.0
    for kind in ("silu", "sigmoid"):
        y, _ = lores.lores_gated_norm(x, z, w, EPS, act=ACTS[kind])
        assert torch.isfinite(y[5]).all() and (y[4] == 0).all() and torch.isnan(y[3]).all()
        assert torch.isnan(y[2, 0, 3]) and int(torch.isnan(y[2]).sum()) == 1
        other = torch.arange(64, device=dev()) != 3
        assert torch.isfinite(y[:2, 0, other]).all()
        if kind == "sigmoid":
            assert torch.isfinite(y[:2]).all() and y[1, 0, 3] == 0
        c, s = lores.lores_gated_norm(x, z, w, EPS, act=ACTS[kind], out_prec=lores.LORES_MXFP4)
        assert (s[3, :2] == 255).all() and s[2, 0] == 255 and s[2, 1] < 255 and (s[5, :2] < 255).all()
        assert (c[4] & 0x77 == 0).all() and (s[4, :2] == 0).all() and (s[:, 2:] == 0).all()
    y, _ = lores.lores_gated_norm(x[4:5], z[4:5], w, 0.0)
    assert torch.isnan(y).all()                      # 0 times an infinite r
    c, s = lores.lores_gated_norm(x[4:5], z[4:5], w, 0.0, out_prec=lores.LORES_MXFP4)
    assert (c & 0x77 == 0).all() and (s == 0).all()
    big, _ = lores.lores_gated_norm(x[5:] * 1e30, z[5:], w, EPS, out_prec=lores.LORES_MXFP4), None
    assert (big[1][0, :2] == 255).all()              # squares beyond fp32


def test_streams_empty_calls_and_inputs_left_alone():
    x, z, w = randn((64, 4, 128), BF16, 81), randn((64, 4, 128), BF16, 82), weight((128,), BF16, 83)
    keep = [t.clone() for t in (x, z, w)]
    want = lores.lores_gated_norm(x, z, w, EPS)[0], *lores.lores_gated_norm_backward(x, z, w, x, EPS)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = lores.lores_gated_norm(x, z, w, EPS, stream=s)[0], *lores.lores_gated_norm_backward(x, z, w, x, EPS, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(keep, (x, z, w)))
    for per in (False, True):
        w0 = weight((4, 128) if per else (128,), BF16, 84)
        y, sc = lores.lores_gated_norm(x[:0], z[:0], w0, EPS, out_prec=lores.LORES_MXFP4)
        assert y.shape == (0, 256) and sc.shape == (0, 16)
        dx, dz, dw = lores.lores_gated_norm_backward(x[:0], z[:0], w0, x[:0], EPS)
        assert dx.shape == dz.shape == (0, 4, 128) and dw.shape == w0.shape and (dw == 0).all()
    for shape in ((3, 0, 4, 128), (0, 3, 4, 128), (2, 3, 0, 4, 128)):
        e = x.new_empty(shape)
        assert lores.lores_gated_norm(e, e, w, EPS)[0].shape == shape
        assert lores.lores_gated_norm_backward(e, e, w, e, EPS)[0].shape == shape


def test_replayed_graph():
    x, z, w = randn((300, 4, 128), BF16, 91), randn((300, 4, 128), BF16, 92), weight((4, 128), BF16, 93)
    dy = randn((300, 4, 128), BF16, 94)

    def step():
        return (*lores.lores_gated_norm(x, z, w, EPS, out_prec=lores.LORES_MXFP4),
                *lores.lores_gated_norm_backward(x, z, w, dy, EPS))

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        for t, seed in ((x, 95), (z, 96), (dy, 97)):
            t.copy_(randn(t.shape, BF16, seed + 10 * i))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_refusals():
    x, z, w = randn((4, 2, 64), F32, 1), randn((4, 2, 64), F32, 2), weight((64,), F32, 3)
    for bad in ((x.half(), z, w), (x, z, w.half()), (None, z, w), (x, None, w), (x, z, None), (x, z.to(BF16), w)):
        with pytest.raises(TypeError):
            lores.lores_gated_norm(*bad, EPS)
    for bad in ((x.cpu(), z, w), (x, z.cpu(), w), (x, z, w.cpu()), (x, z, w[:32]), (x, z[:2], w), (x[0, 0], z[0, 0], w),
                (x.transpose(1, 2), z.transpose(1, 2), weight((2,), F32, 1)), (x, z, weight((3, 64), F32, 1)),
                (randn((4, 3, 2, 64), F32, 1).transpose(0, 1), randn((3, 4, 2, 64), F32, 1), w)):
        with pytest.raises(ValueError):
            lores.lores_gated_norm(*bad, EPS)
    for prec in (lores.LORES_INT8, lores.LORES_FP8, lores.LORES_INT4, 99):
        with pytest.raises(ValueError):
            lores.lores_gated_norm(x, z, w, EPS, out_prec=prec)
    for kw in ({"act": 3}, {"act": -1}, {"eps": -1.0}, {"eps": float("nan")}):
        with pytest.raises(lores.LoresError):
            lores.lores_gated_norm(x, z, w, **{"eps": EPS, **kw})
    with pytest.raises(lores.LoresError):
        lores.lores_gated_norm(x[..., :40], z[..., :40], w[:40], EPS, out_prec=lores.LORES_MXFP4)
    big = torch.zeros(1, 1, lores.LORES_MAX_NORM + 1, device=dev())
    with pytest.raises(lores.LoresError):
        lores.lores_gated_norm(big, big, big[0, 0], EPS)
    with pytest.raises(TypeError):
        lores.lores_gated_norm_backward(x, z, w, x.to(BF16), EPS)
    for dy in (x[:2], x.transpose(0, 1).contiguous().transpose(0, 1)):
        with pytest.raises(ValueError):
            lores.lores_gated_norm_backward(x, z, w, dy, EPS)
    with pytest.warns(UserWarning, match="records no autograd graph"):
        lores.lores_gated_norm(x, z.clone().requires_grad_(), w, EPS)
