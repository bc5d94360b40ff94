"""lores_scan and lores_scan_backward on the GPU against the fp64 oracle.

Tolerances (2-norm of the difference over the 2-norm of the result): sums run
in fp32 over at most 256 keys and a few chunks' products, each leaving out less
than 2^-24 of a term, so a result's error is a random walk of some hundred
roundings of 2^-25: 2^-19 covers it by an order of magnitude.  bf16 results
add one rounding of at most 2^-9 to each element, and 2^-17 for the two planes
that carry them.
"""
import numpy as np
import pytest
import torch

import quantized_linear_recurrence_amd as lores
from oracle import sequence as oseq

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 2.0 ** -19, BF16: 2.0 ** -9 + 2.0 ** -16}


def _dev():
    return torch.device("cuda:0")


def make(B, T, H, Hk, dk, dv, dtype, seed=0, state=True, lengths=None, alpha=None):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)                    # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)                # noqa: E731
    x = {"q": unit(rnd(B, T, Hk, dk)).to(dtype), "k": unit(rnd(B, T, Hk, dk)).to(dtype),
         "v": rnd(B, T, H, dv).to(dtype),
         "alpha": torch.exp(-torch.nn.functional.softplus(rnd(B, T, H) - 3.0)),
         "beta": 2.0 * torch.sigmoid(rnd(B, T, H)), "S0": 0.3 * rnd(B, H, dv, dk) if state else None,
         "lengths": None if lengths is None else torch.tensor(lengths, dtype=torch.int32),
         "do": rnd(B, T, H, dv).to(dtype), "dS": 0.3 * rnd(B, H, dv, dk) if state else None}
    if alpha is not None:
        x["alpha"] = alpha(x["alpha"])
    return {n: None if t is None else t.to(_dev()) for n, t in x.items()}


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy() if t.is_floating_point() \
        else t.cpu().numpy()


def near(got, want, tol, what):
    got = _np(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.isfinite(got).all(), what
    err, size = np.linalg.norm(got - want), np.linalg.norm(want)
    assert err <= tol * size + 1e-30, f"{what}: {err / max(size, 1e-300):.3g} > {tol:.3g}"


def _args(x, delta):
    return (x["q"], x["k"], x["v"], x["alpha"], x["beta"], delta)


def check(x, delta, backward=True):
    dt = x["q"].dtype
    n = {k: _np(t) for k, t in x.items()}
    o, S = lores.lores_scan(*_args(x, delta), S0=x["S0"], lengths=x["lengths"])
    base = [n[k] for k in ("q", "k", "v", "alpha", "beta")]
    o_ref, S_ref = oseq.scan(*base, delta, n["S0"], n["lengths"])
    near(o, o_ref, TOL[dt], "o")
    near(S, S_ref, TOL[F32], "S")
    if not backward:
        return
    got = dict(zip(("dq", "dk", "dv", "dalpha", "dbeta", "dS0"),
                   lores.lores_scan_backward(*_args(x, delta), x["do"], dS=x["dS"], S0=x["S0"],
                                             lengths=x["lengths"])))
    want = oseq.scan_backward(*base, delta, n["do"], n["dS"], n["S0"], n["lengths"])
    for name, w in want.items():
        near(got[name], w, TOL[dt if name in ("dq", "dk", "dv") else F32], name)


# lengths around the chunks of 32 and 64 tokens, and the kernel for few tokens
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 2, 8, 9, 31, 32, 33, 63, 64, 65, 127, 129, 200])
def test_lengths(dtype, T):
    for delta in (0, 1):
        check(make(2, T, 2, 2, 64, 48, dtype, seed=T), delta)


# every width: padded keys, value columns that end inside a tile and a block
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(32, 1), (32, 33), (64, 16), (96, 100), (128, 8), (128, 129),
                                   (160, 40), (192, 65), (224, 256), (256, 250)])
def test_widths(dtype, dk, dv):
    check(make(1, 75, 2, 1, dk, dv, dtype, seed=dk + dv), 1)


# shared q and k: gradients are sums over the heads of a group
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,Hk,dk", [(4, 1, 128), (6, 3, 64), (8, 2, 256), (3, 1, 32)])
@pytest.mark.parametrize("delta", [0, 1])
def test_shared_heads(dtype, H, Hk, dk, delta):
    check(make(2, 70, H, Hk, dk, 24, dtype, seed=H), delta)


# sequences of 0, 1 and all tokens, and lengths that are out of range; what
# stands behind an end is not a number
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [5, 70, 130])
def test_ragged(dtype, T):
    n = [T, 0, 1, T // 2, -3, T + 5]
    for delta, state in ((1, True), (0, False)):
        x = make(6, T, 2, 2, 96, 40, dtype, seed=T, state=state, lengths=n)
        for b, m in enumerate(n):
            for name in ("q", "k", "v", "alpha", "beta", "do"):
                x[name][b, max(0, m):] = float("nan")
        check(x, delta)
        o, _ = lores.lores_scan(*_args(x, delta), S0=x["S0"], lengths=x["lengths"])
        for b, m in enumerate(n):
            assert (o[b, max(0, m):] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["zeros", "ones", "tiny"])
def test_gates_at_their_ends(dtype, kind):
    """alpha of exactly 0 (everything is forgotten, its gradient is not), of 1
    and of the smallest numbers."""
    def gate(a):
        g = torch.Generator().manual_seed(9)
        pick = torch.rand(a.shape, generator=g) < 0.15
        return {"zeros": torch.where(pick, torch.zeros(()), a), "ones": torch.ones_like(a),
                "tiny": torch.where(pick, torch.tensor(1.5e-38), a)}[kind]
    for delta in (0, 1):
        x = make(2, 100, 2, 2, 64, 32, dtype, seed=4, alpha=gate)
        x["beta"][:, ::7] = 0.0                      # tokens that write nothing
        check(x, delta)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [3, 70])
def test_strides_and_alignment(dtype, T):
    """q, k and v as slices of one projection at odd addresses, with heads and
    tokens in another order, and broadcast over heads."""
    B, H, dk, dv = 2, 2, 64, 40
    x = make(B, T, H, H, dk, dv, dtype, seed=11)
    want = lores.lores_scan(*_args(x, 1), S0=x["S0"])
    wide = torch.empty(B, T, 1 + H * (2 * dk + dv), dtype=dtype, device=_dev())
    parts, at = {}, 1                                # one element off any alignment
    for name, w in (("q", dk), ("k", dk), ("v", dv)):
        wide[:, :, at:at + H * w] = x[name].reshape(B, T, H * w)
        parts[name] = wide[:, :, at:at + H * w].view(B, T, H, w)
        at += H * w
    turned = {n: x[n].permute(2, 1, 0, 3).contiguous().permute(2, 1, 0, 3) for n in ("q", "k", "v")}
    for y in (parts, turned):
        y = {**x, **y}
        assert not y["q"].is_contiguous()
        got = lores.lores_scan(*_args(y, 1), S0=y["S0"])
        for a, b in zip(got, want):
            assert torch.equal(a, b)                 # the same sums in the same order
        check(y, 1)
    for n in ("q", "k"):
        x[n] = x[n][:, :, :1].expand(B, T, H, dk)    # a stride of 0
    check(x, 1)


def test_offsets_past_32_bits():
    """Sequences 2^31 + 8 elements apart, and tokens 2^24 + 8 apart."""
    B, T, H, dk, dv = 2, 20, 1, 32, 16
    x = make(B, T, H, H, dk, dv, BF16, seed=12)
    want = lores.lores_scan(*_args(x, 1))
    for name, shape, stride in (("q", (B, T, H, dk), (2 ** 31 + 8, dk, dk, 1)),
                                ("v", (B, T, H, dv), (2 ** 24 + 8, 2 ** 25 + 16, dv, 1))):
        size = sum((s - 1) * d for s, d in zip(shape, stride)) + 1
        far = torch.empty(size, dtype=BF16, device=_dev()).as_strided(shape, stride)
        far.copy_(x[name])
        got = lores.lores_scan(*_args({**x, name: far}, 1))
        for a, b in zip(got, want):
            near(a, _np(b), TOL[a.dtype], name)
        del far


@pytest.mark.parametrize("T", [1, 70])
def test_buffers_and_streams(T):
    """Caller's buffers, the state in place, and a stream of its own."""
    x = make(2, T, 2, 2, 64, 64, BF16, seed=13)
    want_o, want_S = lores.lores_scan(*_args(x, 1), S0=x["S0"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    n = lores.lores_scan_workspace(x["q"], x["v"], 1)
    assert (n == 0) == (T <= 8)
    with torch.cuda.stream(s):
        o, S = torch.full_like(want_o, 7.0), x["S0"].clone()
        work = torch.empty(n, dtype=torch.uint8, device=_dev()) if n else None
        got = lores.lores_scan(*_args(x, 1), S0=S, o=o, S=S, workspace=work)
    assert got[0] is o and got[1] is S
    s.synchronize()
    assert torch.equal(o, want_o) and torch.equal(S, want_S)
    other = lores.lores_scan(*_args(x, 1), S0=x["S0"], stream=s)
    grads = lores.lores_scan_backward(*_args(x, 1), x["do"], dS=x["dS"], S0=x["S0"], stream=s)
    s.synchronize()
    assert torch.equal(other[0], want_o) and torch.equal(other[1], want_S)
    again = lores.lores_scan_backward(*_args(x, 1), x["do"], dS=x["dS"], S0=x["S0"])
    for a, b in zip(grads, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_same_bits_every_time(dtype):
    x = make(3, 150, 4, 2, 128, 72, dtype, seed=14, lengths=[150, 77, 149])
    runs = []
    for _ in range(3):
        runs.append(lores.lores_scan(*_args(x, 1), S0=x["S0"], lengths=x["lengths"])
                    + lores.lores_scan_backward(*_args(x, 1), x["do"], dS=x["dS"], S0=x["S0"],
                                                lengths=x["lengths"]))
    for r in runs[1:]:
        for a, b in zip(r, runs[0]):
            assert torch.equal(a, b)


def test_many_units():
    """Enough units for eight wavefronts in a work-group, with value rows that
    leave some of them without any."""
    for dv in (72, 128):
        x = make(16, 66, 16, 16, 64, dv, BF16, seed=15, state=False)
        check(x, 1, backward=False)


def test_gradient_matches_differences():
    """Directional differences of the kernel itself: a step of 2^-7 leaves about
    2^-14 of the third derivative, and 2^-19 / 2^-7 of rounding."""
    x = make(1, 70, 2, 2, 32, 16, F32, seed=16)
    g = torch.Generator(device=_dev()).manual_seed(17)

    def loss(y):
        o, S = lores.lores_scan(*_args(y, 1), S0=y["S0"])
        return float((o.double() * x["do"].double()).sum() + (S.double() * x["dS"].double()).sum())

    got = dict(zip(("q", "k", "v", "alpha", "beta", "S0"),
                   lores.lores_scan_backward(*_args(x, 1), x["do"], dS=x["dS"], S0=x["S0"])))
    for name in got:
        d = torch.randn(x[name].shape, generator=g, device=_dev())
        if name in ("q", "k", "alpha", "beta"):
            d = 0.1 * d
        e = 2.0 ** -7
        num = (loss({**x, name: x[name] + e * d}) - loss({**x, name: x[name] - e * d})) / (2 * e)
        ref = float((got[name].double() * d.double()).sum())
        size = float(got[name].double().norm() * d.double().norm())
        assert abs(num - ref) <= 2.0 ** -10 * size, (name, num, ref, size)


@pytest.mark.parametrize("T", [4, 70])
def test_continuing_is_the_same(T):
    """Two calls over the halves of a sequence are one call over it."""
    x = make(2, 2 * T, 2, 1, 96, 48, F32, seed=18)
    o, S = lores.lores_scan(*_args(x, 1), S0=x["S0"])
    first = {n: t[:, :T] if n != "S0" and n != "dS" and t is not None else t for n, t in x.items()}
    second = {n: t[:, T:] if n != "S0" and n != "dS" and t is not None else t for n, t in x.items()}
    for y in (first, second):
        y["alpha"], y["beta"] = y["alpha"].contiguous(), y["beta"].contiguous()
    o1, S1 = lores.lores_scan(*_args(first, 1), S0=x["S0"])
    o2, S2 = lores.lores_scan(*_args(second, 1), S0=S1)
    near(torch.cat([o1, o2], 1), _np(o), TOL[F32], "o")
    near(S2, _np(S), TOL[F32], "S")


def test_no_tokens():
    x = make(2, 0, 2, 2, 64, 32, F32, seed=19)
    o, S = lores.lores_scan(*_args(x, 1), S0=x["S0"])
    assert o.shape == (2, 0, 2, 32) and torch.equal(S, x["S0"])
    g = lores.lores_scan_backward(*_args(x, 1), x["do"], dS=x["dS"], S0=x["S0"])
    assert torch.equal(g[5], x["dS"]) and g[0].numel() == 0


def test_prompt_hands_over_to_decoding():
    """The state after a prompt, quantized as it is, decodes like the sequence."""
    B, T, H, d = 2, 40, 2, 64
    x = make(B, T + 1, H, H, d, d, F32, seed=20, state=False)
    o_ref, _ = oseq.scan(*(_np(x[n]) for n in ("q", "k", "v", "alpha", "beta")), 1)
    head = {n: x[n][:, :T].contiguous() for n in ("q", "k", "v", "alpha", "beta")}
    _, S = lores.lores_scan(*_args(head, 1))
    st = lores.lores_state_alloc(B, H, d, d, [lores.LORES_FP32] * H, device=_dev())
    lores.lores_quant_state(st, S, 0)
    last = [x[n][:, T].contiguous() for n in ("q", "k", "v", "alpha", "beta")]
    o = lores.lores_decode_step(st, *last, 1, 0, 1)
    near(o, o_ref[:, T], TOL[F32], "o")


@pytest.mark.parametrize("T", [1, 70])
def test_replayed_graph(T):
    x = make(2, T, 2, 2, 64, 64, BF16, seed=21)
    buf = {n: x[n].clone() for n in ("q", "k", "v", "alpha", "beta", "S0", "do", "dS")}
    o, S = torch.empty_like(x["v"]), torch.empty_like(x["S0"])
    n = lores.lores_scan_workspace(x["q"], x["v"], 1)
    work = torch.empty(max(n, 1), dtype=torch.uint8, device=_dev())
    wb = torch.empty(lores.lores_scan_workspace(x["q"], x["v"], 1, True), dtype=torch.uint8, device=_dev())
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        lores.lores_scan(*_args(buf, 1), S0=buf["S0"], o=o, S=S, workspace=work)
        lores.lores_scan_backward(*_args(buf, 1), buf["do"], dS=buf["dS"], S0=buf["S0"], workspace=wb)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lores.lores_scan(*_args(buf, 1), S0=buf["S0"], o=o, S=S, workspace=work)
        grads = lores.lores_scan_backward(*_args(buf, 1), buf["do"], dS=buf["dS"], S0=buf["S0"], workspace=wb)
    for seed in (22, 23, 24):
        y = make(2, T, 2, 2, 64, 64, BF16, seed=seed)
        for name in buf:
            buf[name].copy_(y[name])
        graph.replay()
        torch.cuda.synchronize()
        want = lores.lores_scan(*_args(y, 1), S0=y["S0"])
        want_g = lores.lores_scan_backward(*_args(y, 1), y["do"], dS=y["dS"], S0=y["S0"])
        assert torch.equal(o, want[0]) and torch.equal(S, want[1])
        for a, b in zip(grads, want_g):
            assert torch.equal(a, b)


def test_refusals():
    x = make(2, 12, 2, 2, 64, 32, F32, seed=25)

    def bad(error, **kw):
        y = {**x, **{n: t for n, t in kw.items() if n in x}}
        more = {n: t for n, t in kw.items() if n not in x}
        with pytest.raises(error):
            lores.lores_scan(*_args(y, 1), S0=y["S0"], lengths=y["lengths"], **more)

    bad(TypeError, q=None)
    bad(TypeError, q=x["q"].half())
    bad(TypeError, k=x["k"].to(BF16))
    bad(TypeError, alpha=x["alpha"].double())
    bad(TypeError, beta=None)
    bad(TypeError, lengths=torch.zeros(2, dtype=torch.int64, device=_dev()))
    bad(ValueError, q=x["q"].cpu())
    bad(ValueError, v=x["v"].cpu())
    bad(ValueError, q=x["q"][:, :5])
    bad(ValueError, k=x["k"][..., :32])
    bad(ValueError, v=x["v"].transpose(2, 3).contiguous().transpose(2, 3))
    bad(ValueError, alpha=x["alpha"][:, :5])
    bad(ValueError, S0=x["S0"][:1])
    bad(ValueError, lengths=torch.zeros(3, dtype=torch.int32, device=_dev()))
    bad(ValueError, o=torch.empty(5, device=_dev()))
    bad(lores.LoresError, workspace=torch.empty(256, dtype=torch.uint8, device=_dev()))
    for dk in (48, 288):
        z = torch.zeros(1, 12, 1, dk, device=_dev())
        g = torch.zeros(1, 12, 1, device=_dev())
        with pytest.raises(lores.LoresError):
            lores.lores_scan(z, z, z[..., :16], g, g, 1)
    with pytest.raises(lores.LoresError):            # H_k does not divide H
        lores.lores_scan(x["q"], x["k"], x["v"][:, :, :1].contiguous().expand(2, 12, 3, 32),
                         torch.zeros(2, 12, 3, device=_dev()), torch.zeros(2, 12, 3, device=_dev()), 1)
    with pytest.raises(lores.LoresError):
        lores.lores_scan(*_args(x, 2))
    with pytest.raises(TypeError):
        lores.lores_scan_backward(*_args(x, 1), None)
    with pytest.raises(TypeError):
        lores.lores_scan_backward(*_args(x, 1), x["do"].to(BF16))
    with pytest.raises(ValueError):
        lores.lores_scan_backward(*_args(x, 1), x["do"], dS=x["dS"][:1])
