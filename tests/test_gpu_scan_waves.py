"""The scan's passes by eight wavefronts a work-group (from 256 work-groups of up to
128 value rows on), forward and backward: against the fp64 oracle on some of the
sequences, and bit by bit against the same sequences by four wavefronts, which
add in the same order.  Nothing may depend on what the workspace holds before.

Tolerances: sums run in fp32 over at most 256 keys and a few chunks' products, a
random walk of some hundred roundings of 2^-25, which 2^-19 of the 2-norm covers by
an order of magnitude.  A bf16 result is such a sum rounded once: every element
may be half a step of bf16 off (2^-8 of its power of two, bf16 having 8
significant bits), and what is off beyond that has to be fp32's.
"""
import numpy as np
import pytest
import torch

import quantized_linear_recurrence_amd as lores
from oracle import sequence as oseq

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TOL = 2.0 ** -19
DEV = "cuda:0"
GRADS = ("dq", "dk", "dv", "dalpha", "dbeta", "dS0")


def make(B, T, H, Hk, dk, dv, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)        # noqa: E731
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dtype)    # noqa: E731
    x = {"q": unit(rnd(B, T, Hk, dk)), "k": unit(rnd(B, T, Hk, dk)), "v": rnd(B, T, H, dv).to(dtype),
         "alpha": torch.exp(-torch.nn.functional.softplus(rnd(B, T, H) - 3.0)),
         "beta": 2.0 * torch.sigmoid(rnd(B, T, H)), "S0": 0.3 * rnd(B, H, dv, dk),
         "lengths": torch.randint(0, T + 1, (B,), generator=g, device=DEV, dtype=torch.int32),
         "do": rnd(B, T, H, dv).to(dtype), "dS": 0.3 * rnd(B, H, dv, dk)}
    x["lengths"][:4] = torch.tensor([T, 0, 1, T - 1])
    x["lengths"][-1] = T
    pad = torch.arange(T, device=DEV)[None] >= x["lengths"][:, None]
    for n in ("q", "k", "v", "alpha", "beta", "do"):
        x[n][pad] = float("nan")
    return x


def run(x, delta):
    args = (x["q"], x["k"], x["v"], x["alpha"], x["beta"], delta)

    def work(backward):                              # not a number, whatever type it is read as
        n = lores.lores_scan_workspace(x["q"], x["v"], delta, backward)
        return torch.full((n,), 255, dtype=torch.uint8, device=DEV)

    out = dict(zip(("o", "S"), lores.lores_scan(
        *args, S0=x["S0"], lengths=x["lengths"], workspace=work(False),
        o=torch.full_like(x["v"], float("nan")), S=torch.full_like(x["S0"], float("nan")))))
    out.update(zip(GRADS, lores.lores_scan_backward(*args, x["do"], dS=x["dS"], S0=x["S0"], lengths=x["lengths"],
                                                    workspace=work(True))))
    return out


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("delta", [0, 1])
@pytest.mark.parametrize("T", [40, 130])
@pytest.mark.parametrize("H,Hk,dk,dv", [(8, 8, 64, 72), (8, 2, 96, 40), (8, 8, 128, 128), (8, 4, 128, 136),
                                        (8, 8, 32, 16)])
def test_eight_wavefronts(dtype, delta, T, H, Hk, dk, dv):
    B = 33                                           # 264 units, and 248 without the last two sequences
    x = make(B, T, H, Hk, dk, dv, dtype, seed=T + dk + dv)
    got = run(x, delta)
    n = {k: t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy() for k, t in x.items()}
    for b in (0, 1, 2, 17, B - 1):
        s = slice(b, b + 1)
        base = [n[k][s] for k in ("q", "k", "v", "alpha", "beta")]
        want = dict(zip(("o", "S"), oseq.scan(*base, delta, n["S0"][s], n["lengths"][s])))
        want.update(oseq.scan_backward(*base, delta, n["do"][s], n["dS"][s], n["S0"][s], n["lengths"][s]))
        for name, w in want.items():
            y = got[name][s].double().cpu().numpy()
            assert np.isfinite(y).all(), (name, b)
            off = np.abs(y - w)
            if got[name].dtype == BF16:
                off = np.maximum(off - 2.0 ** -8 * np.exp2(np.floor(np.log2(np.maximum(np.abs(w), 1e-30)))), 0.0)
            assert np.linalg.norm(off) <= TOL * np.linalg.norm(w) + 1e-30, (name, b)
    if dv <= 128:                                    # with more value rows 124 units are still enough for eight
        for part in (slice(0, B - 2), slice(2, B)):
            few = run({k: t[part].contiguous() for k, t in x.items()}, delta)
            for name in got:
                assert torch.equal(few[name], got[name][part]), name
