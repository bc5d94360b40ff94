"""Whole sequences in fp64: the unquantized recurrence token by token, its
gradient, and the root-mean-square norm with its gradient.

  S_t = S_{t-1} alpha_t (I - delta beta_t k_t k_t^T) + beta_t v_t k_t^T,
  o_t = S_t q_t

Arrays carry a leading [B, T] (sequence, token); q and k have H_k heads, value
head h reading q / k head h // (H / H_k).  Tokens from lengths[b] on do not
exist: nothing of theirs is read, their outputs and gradients are 0.
"""
import numpy as np


def _live(T, B, lengths):
    n = np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)
    return np.arange(T)[None, :] < n[:, None]


def _clean(x, live, fill):
    x = np.asarray(x, np.float64)
    return np.where(live.reshape(live.shape + (1,) * (x.ndim - 2)), x, fill)


def _inputs(q, k, v, alpha, beta, lengths):
    B, T, H = np.asarray(alpha).shape
    live = _live(T, B, lengths)
    G = H // q.shape[2]
    q, k = (np.repeat(_clean(x, live, 0.0), G, axis=2) for x in (q, k))
    return q, k, _clean(v, live, 0.0), _clean(alpha, live, 1.0), _clean(beta, live, 0.0), live, G


def _step(S, k, v, al, be, delta):
    """S_t, the decayed state S_{t-1} alpha_t and w_t (the write is beta_t w_t k_t^T)."""
    Sd = S * al[..., None, None]
    w = v - delta * np.einsum("bhvk,bhk->bhv", Sd, k)
    return Sd + np.einsum("bh,bhv,bhk->bhvk", be, w, k), Sd, w


def scan(q, k, v, alpha, beta, delta, S0=None, lengths=None):
    """(o [B, T, H, d_v], S_T [B, H, d_v, d_k])."""
    q, k, v, alpha, beta, _, _ = _inputs(q, k, v, alpha, beta, lengths)
    B, T, H, dk = k.shape
    S = np.zeros((B, H, v.shape[3], dk)) if S0 is None else np.asarray(S0, np.float64)
    o = np.zeros(v.shape)
    for t in range(T):
        S, _, _ = _step(S, k[:, t], v[:, t], alpha[:, t], beta[:, t], delta)
        o[:, t] = np.einsum("bhvk,bhk->bhv", S, q[:, t])
    return o, S


def scan_backward(q, k, v, alpha, beta, delta, do, dS=None, S0=None, lengths=None):
    """Gradients of sum(do o) + sum(dS S_T): a dict with dq, dk, dv, dalpha, dbeta, dS0."""
    Hk = q.shape[2]
    q, k, v, alpha, beta, live, G = _inputs(q, k, v, alpha, beta, lengths)
    do = _clean(do, live, 0.0)
    B, T, H, dk = k.shape
    S = np.zeros((B, H, v.shape[3], dk)) if S0 is None else np.asarray(S0, np.float64)
    before = []
    for t in range(T):
        before.append(S)
        S, _, _ = _step(S, k[:, t], v[:, t], alpha[:, t], beta[:, t], delta)
    g = np.zeros(S.shape) if dS is None else np.asarray(dS, np.float64)
    dq, dk_, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    da, db = np.zeros(alpha.shape), np.zeros(beta.shape)
    for t in reversed(range(T)):
        S, Sd, w = _step(before[t], k[:, t], v[:, t], alpha[:, t], beta[:, t], delta)
        dq[:, t] = np.einsum("bhvk,bhv->bhk", S, do[:, t])
        g = g + np.einsum("bhv,bhk->bhvk", do[:, t], q[:, t])
        gk = np.einsum("bhvk,bhk->bhv", g, k[:, t])             # gradient of beta w
        be = beta[:, t][..., None]
        db[:, t] = (gk * w).sum(-1)
        dv[:, t] = be * gk
        dk_[:, t] = be * np.einsum("bhvk,bhv->bhk", g, w) - delta * np.einsum("bhvk,bhv->bhk", Sd, be * gk)
        g = g - delta * np.einsum("bhv,bhk->bhvk", be * gk, k[:, t])
        da[:, t] = (g * before[t]).sum((-1, -2))
        g = g * alpha[:, t][..., None, None]

    def heads(x):
        return x.reshape(B, T, Hk, G, dk).sum(3)

    m = live[..., None]
    return {"dq": heads(dq) * m[..., None], "dk": heads(dk_) * m[..., None], "dv": dv * m[..., None],
            "dalpha": da * m, "dbeta": db * m, "dS0": g}


def rmsnorm(h, weight, eps):
    """y = h r w with r = (mean h^2 + eps)^(-1/2); returns (y, r)."""
    h, w = np.asarray(h, np.float64), np.asarray(weight, np.float64)
    r = 1.0 / np.sqrt((h * h).mean(-1) + eps)
    return h * r[..., None] * w, r


def rmsnorm_backward(h, weight, eps, dy, dresidual=None):
    """(dx, dw) of sum(dy y) plus the gradient dresidual of h itself."""
    h, w, dy = (np.asarray(x, np.float64) for x in (h, weight, dy))
    n = h.shape[-1]
    r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    g = w * dy
    dx = r * g - h * r ** 3 * (g * h).sum(-1, keepdims=True) / n
    if dresidual is not None:
        dx = dx + np.asarray(dresidual, np.float64)
    return dx, (dy * h * r).reshape(-1, n).sum(0)


def rmsnorm_codes(h, weight, top):
    """The codes of an 8-bit output, before their own rounding: z fl(top fl(1 / m))
    in fp32, with z = fl(h w) and m its largest magnitude (at least 2^-119); and the
    m of the scale, which is 0 for a row of zeros."""
    z = np.asarray(h, np.float32) * np.asarray(weight, np.float32)
    most = np.abs(z).max(-1, keepdims=True)
    m = np.maximum(most, np.float32(2.0 ** -119))
    return z * (np.float32(top) * (np.float32(1.0) / m)), np.where(most > 0, m, most)[..., 0]
