"""bf16 scans whose large terms cancel: the sums are held to fp32 accuracy before
the one rounding to bf16, so what is left of a cancellation is right too.

Every case has terms of size about 1 whose sum is 2^-17 or 2^-19: it stands in
bits that two bf16 planes (16 bits) of a term do not hold and fp32 does.  Keys and
queries are unit vectors and most factors powers of two, so an fp32 sum makes a
handful of roundings of 2^-24: 2^-21 covers them, and a lost third plane is off
by 2^-17 or 2^-19.  The bf16 result's own rounding is at most 2^-8 of the result.
"""
import numpy as np
import pytest
import torch

import quantized_linear_recurrence_amd as lores
from oracle import sequence as oseq

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
DK, DV = 64, 3
TWO = 1.0 - 2.0 ** -8 + 2.0 ** -10                   # two planes hold it
THREE = TWO + 2.0 ** -19                             # and three this


def _case(T):
    """Gates of 1 and rows of zeros, for a case to fill in."""
    z = {"q": torch.zeros(1, T, 1, DK), "k": torch.zeros(1, T, 1, DK), "v": torch.zeros(1, T, 1, DV),
         "alpha": torch.ones(1, T, 1), "beta": torch.ones(1, T, 1), "S0": torch.zeros(1, 1, DV, DK),
         "do": torch.zeros(1, T, 1, DV)}
    z["k"][:, :, :, 5] = 1.0                         # tokens that are not part of the case write zeros there
    return z


def _state(T):
    """The entering state is read by a difference of two columns."""
    z = _case(T)
    z["S0"][..., 0], z["S0"][..., 1] = 1 + 2.0 ** -8 + 2.0 ** -17, 1 + 2.0 ** -8
    z["q"][..., 0], z["q"][..., 1] = 1.0, -1.0
    return z


def _writes(T):
    """Two writes at opposite keys; later tokens read their difference."""
    z = _case(T)
    z["k"][:, :2] = 0.0
    z["k"][0, 0, 0, 0], z["k"][0, 1, 0, 0] = 1.0, -1.0
    z["v"][:, :2] = 1.0
    z["beta"][0, 0, 0], z["beta"][0, 1, 0] = 1 + 2.0 ** -8 + 2.0 ** -17, 1 + 2.0 ** -8
    z["q"][:, 2:, :, 0] = 1.0
    return z


def _decay(T):
    """A write that has decayed by THREE, and one of -TWO on top of it: outputs,
    and the gradients of the queries that read them."""
    z = _case(T)
    z["k"][:, :2] = 0.0
    z["k"][:, :2, :, 0] = 1.0
    z["v"][0, 0], z["v"][0, 1] = 1.0, -1.0
    z["alpha"][0, 1, 0], z["beta"][0, 1, 0] = THREE, TWO
    z["q"][..., 0] = 1.0
    z["q"][:, 0] = 0.0
    z["do"][:, 1:, :, 0] = 1.0
    return z


def _key(T):
    """A key that two outputs read, one of them through a decay of THREE."""
    z = _case(T)
    z["k"][:, 0] = 0.0
    z["k"][0, 0, 0, 0] = 1.0
    z["v"][0, 0, 0] = 1.0
    z["alpha"][0, 1, 0] = THREE
    z["q"][:, :2, :, 1] = 1.0
    z["do"][0, 0, 0, 0], z["do"][0, 0, 0, 1] = 1.0 - 2.0 ** -8, 2.0 ** -10
    z["do"][0, 1, 0, 0] = -1.0
    return z


def _correction(T):
    """delta: a key whose correction by an earlier write of THREE cancels what
    a later output reads of it."""
    z = _case(T)
    z["k"][:, :2] = 0.0
    z["k"][0, 0, 0, 0], z["k"][0, 1, 0, 1] = 1.0, 1.0
    z["v"][0, 0, 0] = torch.tensor([1.0, 0.0, 0.0])
    z["v"][0, 1, 0] = torch.tensor([0.0, 1.0, 1.0])
    z["beta"][0, 0, 0] = THREE
    z["q"][0, 1, 0, 1], z["q"][0, 2, 0, 0] = 1.0, 1.0
    z["do"][0, 1, 0] = torch.tensor([1.0, 0.0, 0.0])
    z["do"][0, 2, 0] = torch.tensor([0.0, 1.0 - 2.0 ** -8, 2.0 ** -10])
    return z


def _near(got, want, what):
    got = got.double().cpu().numpy()
    bad = np.abs(got - want) > 2.0 ** -8 * np.abs(want) + 2.0 ** -21
    assert not bad.any(), (what, got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("T", [9, 40, 70])
@pytest.mark.parametrize("case,delta,small", [(_state, 0, "o"), (_writes, 0, "o"), (_decay, 0, "o"),
                                              (_decay, 0, "dq"), (_key, 0, "dk"), (_correction, 1, "dk")])
def test_what_is_left_of_a_cancellation(case, delta, small, T):
    z = case(T)
    dev = {n: x.to("cuda:0", BF16 if n in ("q", "k", "v", "do") else F32) for n, x in z.items()}
    for n in z:                                      # bf16 holds the case
        assert torch.equal(dev[n].float().cpu(), z[n]), n
    names = ("q", "k", "v", "alpha", "beta")
    ref = {n: x.double().numpy() for n, x in z.items()}
    args = (*(dev[n] for n in names), delta)
    o, _ = lores.lores_scan(*args, S0=dev["S0"])
    o_ref, _ = oseq.scan(*(ref[n] for n in names), delta, ref["S0"])
    got = dict(zip(("dq", "dk", "dv"), lores.lores_scan_backward(*args, dev["do"], S0=dev["S0"])))
    want = oseq.scan_backward(*(ref[n] for n in names), delta, ref["do"], None, ref["S0"])
    got["o"], want["o"] = o, o_ref
    size = np.abs(want[small])
    assert ((size > 2.0 ** -20) & (size < 2.0 ** -16)).any()     # the case is what it says
    for n in ("o", "dq", "dk", "dv"):
        _near(got[n], want[n], n)
