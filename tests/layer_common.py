"""What the tests of the layer operators share: inputs, comparison in 2-norms, tolerances.

fp32 results: a row's sum of squares takes at most 16 steps per lane and 10 across
lanes, halved by the root; a gate adds an exponential and a reciprocal of 2^-23 each
and a handful of products: fewer than 64 roundings of 2^-24, 2^-18.  bf16 results add
half a step, 2^-8.  A weight's gradient adds up to 2^16 products in fp32: 2^-17.
"""
import numpy as np
import torch

F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 2.0 ** -18, BF16: 2.0 ** -8 + 2.0 ** -17}
DW = 2.0 ** -17
EPS = 1e-6


def dev():
    return torch.device("cuda:0")


def arr(t):
    return None if t is None else t.detach().double().cpu().numpy()


def near(got, want, tol, what):
    got = arr(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.isfinite(got).all(), what
    err, size = np.linalg.norm(got - want), np.linalg.norm(want)
    assert err <= tol * size + 1e-30, f"{what}: {err / max(size, 1e-300):.3g} > {tol:.3g}"


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(dtype).to(dev())


def weight(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (1.0 + 0.2 * torch.randn(*shape, generator=g)).to(dtype).to(dev())


def blocks_near(codes, scales, y, what):
    """4-bit rows of values that fp32 roundings set apart from y by up to 2^-17:
    each is a nearest value of the grid to that, and a block's scale is the rule's
    or, where its largest is that near 7 units, the next one."""
    from oracle import layer
    codes, scales, y = codes.cpu().numpy(), scales.cpu().numpy(), np.asarray(y, np.float64)
    n = y.shape[-1]
    _, want = layer.mx_quant(y)
    got = scales[..., :n // 32]
    assert (scales[..., n // 32:] == 0).all(), what
    m = np.abs(y.reshape(*y.shape[:-1], -1, 32)).max(-1)
    f = np.frexp(m)[0]
    border = np.abs(f / 0.875 - 1) < 2.0 ** -17
    assert (np.where(border, np.abs(got.astype(int) - want) <= 1, got == want)).all(), what
    q = np.abs(y.reshape(*y.shape[:-1], -1, 32)) * np.exp2(127.0 - got)[..., None]
    v = layer.mx_values(codes, scales).reshape(q.shape) * np.exp2(127.0 - got)[..., None]
    v = np.abs(v)
    best = np.abs(q[..., None] - layer.GRID).min(-1)
    assert (np.abs(v - q) <= best + 2.0 ** -16 * q).all(), what
    sign = np.sign(layer.mx_values(codes, scales)) * np.sign(y)
    assert (sign >= 0).all(), what
