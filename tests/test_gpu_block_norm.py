"""lores_block_norm and its gradient against the fp64 oracle (tolerances: layer_common)."""
import numpy as np
import pytest
import torch

import quantized_linear_recurrence_amd as lores
from tests.layer_common import BF16, DW, EPS, F32, TOL, arr, blocks_near, dev, near, randn, weight
from oracle import layer
from oracle import sequence as oseq

pytestmark = pytest.mark.gpu
ACTS = {None: lores.LORES_ACT_NONE, "none": lores.LORES_ACT_NONE, "silu": lores.LORES_ACT_SILU,
        "sigmoid": lores.LORES_ACT_SIGMOID}


def forward(x, res, w, wn, scale, gate, kind, prec=None, eps=EPS):
    y, s, h = lores.lores_block_norm(x, res, w, wn, eps, scale=scale, gate=gate, act=ACTS[kind], out_prec=prec)
    assert h.dtype is x.dtype and h.shape == x.shape
    near(h, layer.block_sum(arr(x), arr(res), arr(w), eps, scale, arr(gate), kind), TOL[x.dtype], "h")
    want = layer.block_norm(arr(h), arr(wn), eps)
    if prec in (lores.LORES_INT8, lores.LORES_FP8):
        top = 127.0 if prec == lores.LORES_INT8 else 448.0
        c, m = oseq.rmsnorm_codes(h.float().cpu().numpy(), wn.float().cpu().numpy(), top)
        if prec == lores.LORES_INT8:
            np.testing.assert_array_equal(y.cpu().numpy(), np.rint(c).astype(np.int8))
        else:
            c = torch.from_numpy(np.clip(c, -448, 448)).to(torch.float8_e4m3fn)
            assert torch.equal(y.cpu().view(torch.uint8), c.view(torch.uint8))
        near(s, m.astype(np.float64) * oseq.rmsnorm(arr(h), arr(wn), eps)[1] / top, TOL[F32], "scales")
    elif prec == lores.LORES_MXFP4:
        blocks_near(y, s, want, "codes")
    else:
        assert s is None
        near(y, want, TOL[y.dtype], "y")
    return h


def backward(x, h, w, wn, scale, gate, kind, with_dh, eps=EPS, seed=7):
    dy = randn(x.shape, x.dtype, seed)
    dh = randn(x.shape, x.dtype, seed + 1) if with_dh else None

    def call():
        return lores.lores_block_norm_backward(x, h, w, wn, dy, eps, scale=scale, gate=gate, act=ACTS[kind], dh=dh)

    got = call()
    want = layer.block_norm_backward(arr(x), arr(h), arr(w), arr(wn), arr(dy), eps, scale, arr(gate), kind, arr(dh))
    for g, name, tol in zip(got, ("dx", "dres", "dgate", "dw", "dwn"), [TOL[x.dtype]] * 3 + [DW] * 2):
        if want[name] is None:
            assert g is None
        else:
            near(g, want[name], tol, name)
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, call()))


FORMS = ((True, True, None, 1.0, True), (True, True, "sigmoid", 0.5, True), (False, True, "silu", 0.3, False),
         (True, False, "none", 1.0, True), (False, False, None, 1.0, False), (True, False, None, -2.0, True))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [1, 7, 8, 64, 100, 128, 129, 512, 515, 1024, 1030, 2048, 2056, 4096, 4100, 8192, 8200,
                               16384])
def test_widths(dtype, n):
    eps = 0.5 if n == 1 else EPS                     # a row of one element has dx = eps r^3 e
    for i, (res, post, kind, scale, dh) in enumerate(FORMS):
        x = randn((5, n), dtype, n + i)
        r = randn((5, n), dtype, n + i + 1, 3.0) if res else None
        g = None if kind is None else randn((5, n), dtype, n + i + 2)
        w = weight((n,), dtype, 3) if post else None
        wn = weight((n,), dtype, 4)
        prec = (None, lores.LORES_INT8, lores.LORES_FP8, lores.LORES_FP32, lores.LORES_BF16, None)[i]
        h = forward(x, r, w, wn, scale, g, kind, prec, eps)
        backward(x, h, w, wn, scale, g, kind, dh, eps)


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("wt", [F32, BF16])
@pytest.mark.parametrize("n", [32, 96, 160, 1024, 4096, 8224])
def test_blocks(xt, wt, n):
    x, r, g = (randn((2, 3, n), xt, n + i) for i in range(3))
    forward(x, r, weight((n,), wt, 1), weight((n,), wt, 2), 0.5, g, "silu", lores.LORES_MXFP4)
    forward(x, r, None, weight((n,), wt, 2), 1.0, None, None, lores.LORES_MXFP4)
    wide = randn((6, 3 * n + 5), xt, n)
    forward(wide[:, 1:n + 1], wide[:, n + 2:2 * n + 2], None, weight((n + 1,), wt, 2)[1:], 1.0, None, None,
            lores.LORES_MXFP4)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [64, 200, 4096])
def test_strides(dtype, n):
    wide = randn((9, 3 * n + 5), dtype, 4)
    w, wn = weight((n + 1,), dtype, 5)[1:], weight((n + 3,), dtype, 6)[3:]
    x, r, g = wide[:, 1:1 + n], wide[:, n + 2:2 * n + 2], wide[:, 2 * n + 3:3 * n + 3]
    for a, b, c in ((x, r, g), (x[::2], r[::2], g[::2]), (x, r, randn((1, n), dtype, 8).expand(9, n)),
                    (x, randn((1, n), dtype, 9).expand(9, n), None)):
        for prec in (None, lores.LORES_INT8):
            h = forward(a, b, w, wn, 0.5, c, "sigmoid" if c is not None else None, prec)
        backward(a, h, w, wn, 0.5, c, "sigmoid" if c is not None else None, True)


def test_it_is_the_plain_norm_without_weight_and_gate():
    x, r, wn = randn((33, 1024), BF16, 1), randn((33, 1024), BF16, 2, 3.0), weight((1024,), BF16, 3)
    for prec in (None, lores.LORES_INT8, lores.LORES_FP8):
        for a, b in zip(lores.lores_block_norm(x, r, None, wn, EPS, out_prec=prec),
                        lores.lores_rmsnorm(x, wn, EPS, residual=r, out_prec=prec)):
            assert a is b or torch.equal(a.float(), b.float())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("r,n", [(8193, 100), (9001, 128), (2050, 130), (2101, 1024), (1100, 2048), (2100, 4096),
                                 (520, 8200)])
def test_gradients_of_more_rows_than_run_at_once(dtype, r, n):
    x, h, g = randn((r, n), dtype, 1), randn((r, n), dtype, 2, 2.0), randn((r, n), dtype, 3)
    backward(x, h, weight((n,), dtype, 4), weight((n,), dtype, 5), 0.7, g, "silu", True)
    backward(x, h, None, weight((n,), dtype, 5), 0.7, None, None, False)


@pytest.mark.parametrize("kind", [None, "none", "silu", "sigmoid"])
@pytest.mark.parametrize("post", [False, True])
def test_gradients_match_differences(kind, post):
    x, r = randn((5, 130), F32, 20), randn((5, 130), F32, 21, 2.0)
    g = None if kind is None else randn((5, 130), F32, 22)
    w, wn = weight((130,), F32, 23) if post else None, weight((130,), F32, 24)
    dy, dh = randn((5, 130), F32, 25), randn((5, 130), F32, 26)
    kw = {"scale": 0.6, "act": ACTS[kind]}
    _, _, h = lores.lores_block_norm(x, r, w, wn, EPS, gate=g, **kw)
    grads = lores.lores_block_norm_backward(x, h, w, wn, dy, EPS, gate=g, dh=dh, **kw)

    def loss(x=x, r=r, g=g, w=w, wn=wn):
        y, _, h = lores.lores_block_norm(x, r, w, wn, EPS, gate=g, **kw)
        return float((y.double() * dy.double()).sum() + (h.double() * dh.double()).sum())

    e = 2.0 ** -7                                    # truncation 2^-14, rounding 2^-18 / 2^-7
    for (name, v), d in zip((("x", x), ("r", r), ("g", g), ("w", w), ("wn", wn)), grads):
        if v is None:
            assert d is None
            continue
        u = randn(v.shape, F32, 27)
        num = (loss(**{name: v + e * u}) - loss(**{name: v - e * u})) / (2 * e)
        size = float(d.double().norm() * u.double().norm())
        assert abs(num - float((d.double() * u.double()).sum())) <= 2.0 ** -10 * size


def test_rows_that_are_zero_tiny_or_not_finite():
    x, r = randn((6, 256), F32, 6), torch.zeros(6, 256, device=dev())
    x[0] = 0.0
    x[1] = 1e-38
    x[2, 3] = float("inf")
    x[3, 200] = float("nan")
    x[4] *= 1e30
    wn = weight((256,), F32, 7)
    c, s, _ = lores.lores_block_norm(x, r, None, wn, EPS, out_prec=lores.LORES_MXFP4)
    assert (c[0] & 0x77 == 0).all() and (s[0] == 0).all()
    assert (s[2:5] == 255).all() and (c[2:5] == 0).all()
    assert (s[[1, 5]] < 255).all()
    c, s, _ = lores.lores_block_norm(x[:1], r[:1], None, wn, 0.0, out_prec=lores.LORES_MXFP4)
    assert (c & 0x77 == 0).all() and (s == 0).all()
    for prec in (lores.LORES_INT8, lores.LORES_FP8):
        _, s, _ = lores.lores_block_norm(x, r, None, wn, EPS, out_prec=prec)
        assert float(s[0]) == 0 and torch.isnan(s[2:5]).all() and torch.isfinite(s[[0, 1, 5]]).all()
    _, _, h = lores.lores_block_norm(x, r, wn, wn, EPS)
    assert (h[0] == 0).all() and torch.isnan(h[3]).all() and torch.isfinite(h[[0, 1, 5]]).all()


def test_streams_empty_calls_and_graph():
    x, r, g = (randn((64, 512), BF16, 30 + i) for i in range(3))
    w, wn, dy = weight((512,), BF16, 33), weight((512,), BF16, 34), randn((64, 512), BF16, 35)

    def step(stream=None):
        kw = {"scale": 0.5, "gate": g, "act": lores.LORES_ACT_SILU, "stream": stream}
        y, s, h = lores.lores_block_norm(x, r, w, wn, EPS, out_prec=lores.LORES_MXFP4, **kw)
        return (y, s, h, *lores.lores_block_norm_backward(x, h, w, wn, dy, EPS, dh=dy, **kw))

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        x.copy_(randn((64, 512), BF16, 40 + i))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))
    y, s, h = lores.lores_block_norm(x[:0], r[:0], w, wn, EPS, out_prec=lores.LORES_INT8)
    assert y.shape == h.shape == (0, 512) and s.shape == (0,)
    dx, dres, dg, dw, dwn = lores.lores_block_norm_backward(x[:0], h, w, wn, dy[:0], EPS, gate=g[:0])
    assert dx.shape == dres.shape == dg.shape == (0, 512) and (dw == 0).all() and (dwn == 0).all()


def test_batches_of_no_rows():
    w = weight((96,), BF16, 1)
    for shape in ((3, 0, 96), (0, 3, 96), (0, 96), (2, 3, 0, 96)):
        e = torch.empty(shape, dtype=BF16, device=dev())
        y, _, h = lores.lores_block_norm(e, e, w, w, EPS, gate=e)
        assert y.shape == h.shape == shape
        dx, dres, dgate, dw, dwn = lores.lores_block_norm_backward(e, e, w, w, e, EPS, gate=e)
        assert dx.shape == dgate.shape == shape and (dw == 0).all() and (dwn == 0).all()


def test_refusals():
    x, w = randn((4, 64), F32, 40), weight((64,), F32, 41)
    for bad in ((x.half(), None, w, w), (x, None, w.half(), w), (x, None, w, w.half()), (None, x, w, w), (x, x, w, None),
                (x, x.to(BF16), w, w), (x, x, w.to(BF16), w)):
        with pytest.raises(TypeError):
            lores.lores_block_norm(*bad, EPS)
    for bad in ((x.cpu(), None, w, w), (x, x[:2], w, w), (x, x, w[:32], w), (x, x, w, w[:32]), (x.t(), None, w, w),
                (x, x.cpu(), w, w)):
        with pytest.raises(ValueError):
            lores.lores_block_norm(*bad, EPS)
    with pytest.raises(ValueError):
        lores.lores_block_norm(x, x, w, w, EPS, out_prec=lores.LORES_INT4)
    with pytest.raises(ValueError):
        lores.lores_block_norm(x, x, w, w, EPS, gate=x[:2])
    for kw in ({"eps": -1.0}, {"eps": float("inf")}, {"scale": float("nan")}, {"act": 7}):
        with pytest.raises(lores.LoresError):
            lores.lores_block_norm(x, x, w, w, **{"eps": EPS, **kw})
    with pytest.raises(lores.LoresError):
        lores.lores_block_norm(x[:, :40], None, None, w[:40], EPS, out_prec=lores.LORES_MXFP4)
    with pytest.raises(lores.LoresError):            # rows that overlap
        lores.lores_block_norm(x.view(-1).as_strided((4, 64), (32, 1)), None, w, w, EPS)
    big = torch.zeros(1, lores.LORES_MAX_NORM + 1, device=dev())
    with pytest.raises(lores.LoresError):
        lores.lores_block_norm(big, None, None, big[0], EPS)
    with pytest.raises(TypeError):
        lores.lores_block_norm_backward(x, x, w, w, x.to(BF16), EPS)
    for kw in ({"h": x[:2]}, {"dh": x[:2]}, {"dy": x.t().contiguous().t()}):
        with pytest.raises(ValueError):
            lores.lores_block_norm_backward(**{"x": x, "h": x, "weight": w, "weight_next": w, "dy": x, "eps": EPS, **kw})
    with pytest.warns(UserWarning, match="records no autograd graph"):
        lores.lores_block_norm(x, x, w.clone().requires_grad_(), w, EPS)
