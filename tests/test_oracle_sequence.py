"""The fp64 sequence oracle: its recurrence against the closed form of a chunk,
its gradients against central differences, the norm's likewise."""
import numpy as np
import pytest

from oracle import sequence as seq


def _case(seed, B=2, T=7, H=4, Hk=2, dk=5, dv=3):
    g = np.random.default_rng(seed)
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)   # noqa: E731
    return {"q": unit(g.normal(size=(B, T, Hk, dk))), "k": unit(g.normal(size=(B, T, Hk, dk))),
            "v": g.normal(size=(B, T, H, dv)), "alpha": g.uniform(0.3, 1, (B, T, H)),
            "beta": g.uniform(0.1, 1.9, (B, T, H)), "S0": g.normal(size=(B, H, dv, dk))}


@pytest.mark.parametrize("delta", [0, 1])
def test_state_is_the_product_of_the_transitions(delta):
    """S_T = S_0 A_1 .. A_T + sum_j beta_j v_j k_j^T A_{j+1} .. A_T."""
    c = _case(1)
    o, S = seq.scan(**c, delta=delta)
    B, T, H, dv = c["v"].shape
    dk = c["q"].shape[3]
    for b in range(B):
        for h in range(H):
            A = [c["alpha"][b, t, h] * (np.eye(dk) - delta * c["beta"][b, t, h]
                 * np.outer(c["k"][b, t, h // 2], c["k"][b, t, h // 2])) for t in range(T)]
            want = c["S0"][b, h]
            for t in range(T):
                want = want @ A[t] + c["beta"][b, t, h] * np.outer(c["v"][b, t, h], c["k"][b, t, h // 2])
                np.testing.assert_allclose(o[b, t, h], want @ c["q"][b, t, h // 2], rtol=1e-12, atol=1e-13)
            np.testing.assert_allclose(S[b, h], want, rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("delta", [0, 1])
@pytest.mark.parametrize("lengths", [None, [7, 0], [1, 5]])
def test_gradient_matches_differences(delta, lengths):
    c = _case(2)
    c["alpha"][0, 3, 1] = 0.0                        # a gate that forgets everything
    g = np.random.default_rng(3)
    do, dS = g.normal(size=c["v"].shape), g.normal(size=c["S0"].shape)
    live = seq._live(7, 2, lengths)[..., None, None]

    def loss(**x):
        o, S = seq.scan(**x, delta=delta, lengths=lengths)
        return (do * o * live).sum() + (dS * S).sum()

    got = seq.scan_backward(**c, delta=delta, do=do, dS=dS, lengths=lengths)
    for name in ("q", "k", "v", "alpha", "beta", "S0"):
        d = g.normal(size=c[name].shape)
        e = 1e-5
        num = (loss(**{**c, name: c[name] + e * d}) - loss(**{**c, name: c[name] - e * d})) / (2 * e)
        # truncation e^2 and cancellation 2^-53 / e, both under 1e-9 of the terms' size
        assert abs(num - (got["d" + name] * d).sum()) < 1e-7 * max(1.0, abs(num)), name


def test_nothing_behind_the_end_counts():
    c = _case(4)
    o, S = seq.scan(**c, delta=1, lengths=[3, 0])
    for x in ("q", "k", "v", "alpha", "beta"):
        c[x][0, 3:] = np.nan
        c[x][1] = np.nan
    o2, S2 = seq.scan(**c, delta=1, lengths=[3, 0])
    np.testing.assert_array_equal(o, o2)
    np.testing.assert_array_equal(S, S2)
    assert (o[0, 3:] == 0).all() and (o[1] == 0).all()
    np.testing.assert_array_equal(S[1], c["S0"][1])


def test_norm_gradient_matches_differences():
    g = np.random.default_rng(5)
    h, w, dy, dr = g.normal(size=(4, 9)), g.normal(size=9), g.normal(size=(4, 9)), g.normal(size=(4, 9))
    dx, dw = seq.rmsnorm_backward(h, w, 1e-3, dy, dr)
    loss = lambda h, w: (dy * seq.rmsnorm(h, w, 1e-3)[0]).sum() + (dr * h).sum()   # noqa: E731
    for x, got, f in ((h, dx, lambda x: loss(x, w)), (w, dw, lambda x: loss(h, x))):
        d, e = g.normal(size=x.shape), 1e-5
        num = (f(x + e * d) - f(x - e * d)) / (2 * e)
        assert abs(num - (got * d).sum()) < 1e-7 * max(1.0, abs(num))
