"""The operators around the recurrence in fp64: the gated norm, the norms around
a block, their gradients, and microscaled 4-bit rows.

A gate's activations: "none" z, "silu" z / (1 + e^-z), "sigmoid" 1 / (1 + e^-z).
"""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def act(kind, z):
    """(a(z), a'(z))."""
    z = np.asarray(z, np.float64)
    if kind == "none":
        return z, np.ones_like(z)
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-z))
    if kind == "sigmoid":
        return s, s * (1.0 - s)
    return z * s, s * (1.0 + z * (1.0 - s))


def _norm(u, eps):
    r = 1.0 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    return u * r, r


def _norm_back(e, n, r):
    """The gradient of u from that of n = u r."""
    return r * (e - n * (e * n).mean(-1, keepdims=True))


def gated_norm(x, gate, weight, eps, kind, gate_first):
    x, w = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    a, _ = act(kind, gate)
    if gate_first:
        return _norm(x * a, eps)[0] * w
    return _norm(x, eps)[0] * w * a


def gated_norm_backward(x, gate, weight, dy, eps, kind, gate_first):
    """(dx, dgate, dw) of sum(dy y); dw of the weight's shape."""
    x, w, dy = (np.asarray(v, np.float64) for v in (x, weight, dy))
    a, slope = act(kind, gate)
    if gate_first:
        n, r = _norm(x * a, eps)
        du = _norm_back(dy * w, n, r)
        dx, dgate, rows = du * a, du * x * slope, dy * n
    else:
        n, r = _norm(x, eps)
        dx, dgate, rows = _norm_back(dy * w * a, n, r), dy * w * n * slope, dy * a * n
    return dx, dgate, rows.reshape(-1, *w.shape).sum(0) if w.ndim == 2 else rows.reshape(-1, w.size).sum(0)


def block_sum(x, residual, weight, eps, scale, gate, kind):
    """h before its rounding."""
    x = np.asarray(x, np.float64)
    p = x if weight is None else _norm(x, eps)[0] * np.asarray(weight, np.float64)
    p = scale * p if gate is None else scale * p * act(kind, gate)[0]
    return p if residual is None else np.asarray(residual, np.float64) + p


def block_norm(h, weight_next, eps):
    return _norm(np.asarray(h, np.float64), eps)[0] * np.asarray(weight_next, np.float64)


def block_norm_backward(x, h, weight, weight_next, dy, eps, scale, gate, kind, dh):
    """A dict with dx, dres, dgate, dw and dwn of sum(dy y) + sum(dh h)."""
    x, h, wn, dy = (np.asarray(v, np.float64) for v in (x, h, weight_next, dy))
    size = wn.size
    n2, r2 = _norm(h, eps)
    G = _norm_back(dy * wn, n2, r2)
    if dh is not None:
        G = G + np.asarray(dh, np.float64)
    a, slope = (1.0, None) if gate is None else act(kind, gate)
    n1, r1, w = (x, None, 1.0) if weight is None else (*_norm(x, eps), np.asarray(weight, np.float64))
    e = scale * G * a * w
    out = {"dres": G, "dwn": (dy * n2).reshape(-1, size).sum(0), "dx": e, "dgate": None, "dw": None}
    if gate is not None:
        out["dgate"] = scale * G * n1 * w * slope
    if weight is not None:
        out["dx"] = _norm_back(e, n1, r1)
        out["dw"] = (scale * G * a * n1).reshape(-1, size).sum(0)
    return out


# ------------------------------------------------------------ 4-bit blocks

def mx_quant(x):
    """(codes [..., n], biased exponents [..., n / 32]) of rows of fp32 values."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    m = np.abs(b).max(-1)
    fine = np.isfinite(b).all(-1)
    f, k = np.frexp(np.where(fine, m, 1.0))          # m = f 2^k, f in [0.5, 1)
    e = np.clip(np.where(f < 0.875, k - 3, k - 2), -127, None)
    e = np.where(m == 0.0, -127, e)
    with np.errstate(invalid="ignore"):
        q = np.abs(np.where(fine[..., None], b, 0.0)) * np.exp2(-e.astype(np.float64))[..., None]
    d = np.abs(q[..., None] - GRID)                  # ties: the even one of the two nearest codes
    c = np.argmin(d, -1)
    up = np.minimum(c + 1, 7)
    tie = np.take_along_axis(d, up[..., None], -1)[..., 0] == np.take_along_axis(d, c[..., None], -1)[..., 0]
    c = np.where(tie & (c % 2 == 1), up, c)
    c = np.where(np.signbit(b) & fine[..., None], c + 8, c)
    return c.reshape(x.shape).astype(np.uint8), np.where(fine, e + 127, 255).astype(np.uint8)


def mx_pack(codes, exps):
    """The bytes of codes [..., n / 2] and of scales [..., 4 ceil(n / 128)]."""
    n = codes.shape[-1]
    s = np.zeros((*exps.shape[:-1], (n + 127) // 128 * 4), np.uint8)
    s[..., :exps.shape[-1]] = exps
    return codes[..., 0::2] | (codes[..., 1::2] << 4), s


def mx_values(codes, scales):
    """The values [..., n] of packed bytes."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = np.where(c >= 8, -1.0, 1.0) * GRID[c & 7]
    s = scales[..., :c.shape[-1] // 32].astype(np.float64)
    f = np.where(s == 255, np.nan, np.exp2(s - 127.0))
    return (v.reshape(*c.shape[:-1], -1, 32) * f[..., None]).reshape(c.shape)
