"""The weights' gradients over calls whose places pass 2^32, in whole numbers that fp32 adds
exactly: every row counts once.  Rows are of ones and signs, so that their norms are 1 at
eps 0, and their other inputs differ from row to row and on both sides of the places 2^31
and 2^32.  And rows of a product, whose bits do not depend on the rows beside them."""
import pytest
import torch

import quantized_linear_recurrence_amd as lores
from tests.layer_common import F32, randn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
N = 16384


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


def _needs(gib):
    torch.cuda.empty_cache()
    free, _ = torch.cuda.mem_get_info()
    if free < gib << 30:
        pytest.skip(f"needs {gib} GiB of GPU memory")


def _times(a, b):
    """The outer product [len(a), len(b)] in bf16."""
    return a.to(BF16)[:, None] * b.to(BF16)[None]


def test_block_norm_s_weights():
    _needs(80)
    rows = (1 << 18) + 5
    i, j = torch.arange(rows, device=DEV), torch.arange(N, device=DEV)
    part = (i >= 1 << 17).long() + (i >= 1 << 18)     # of the places below 2^31, below 2^32 and behind
    sign, alt = 1 - 2 * (j // 3 % 2), 1 - 2 * (j % 2)
    one, u = torch.ones(N, dtype=BF16, device=DEV), torch.ones(rows, device=DEV)
    x, h = _times(u, sign), _times(u, torch.ones(N, device=DEV))
    f, d = i % 3 + 1, 2 * part + i % 2 + 1
    # sum_j dy_j h_j = 0, so that G = dh + dy; the sums stay below 2^18 9 < 2^24
    dy, dh = _times(f, alt), _times(d, torch.ones(N, device=DEV))
    dx, dres, _, dw, dwn = lores.lores_block_norm_backward(x, h, one, one, dy, 0.0, dh=dh)
    assert torch.equal(dwn, (int(f.sum()) * alt).float())
    assert torch.equal(dw, (sign * (int(d.sum()) + int(f.sum()) * alt)).float())
    for at in (0, (1 << 17) - 2, (1 << 18) - 2):
        assert torch.equal(dres[at:at + 5], dy[at:at + 5] + dh[at:at + 5])


@pytest.mark.parametrize("per_head", [False, True])
def test_gated_norm_s_weights(per_head):
    _needs(70)
    tokens, heads = (1 << 16) + 3, 4
    rows = tokens * heads
    i, j = torch.arange(rows, device=DEV), torch.arange(N, device=DEV)
    part = (i >= 1 << 17).long() + (i >= 1 << 18)
    sign, alt = 1 - 2 * (j // 3 % 2), 1 - 2 * (j % 2)
    f, d = i % 3 + 1, part + i % 2 + 1                # sums below 2^18 12 < 2^24
    x, z, dy = (t.view(tokens, heads, N) for t in (_times(torch.ones(rows, device=DEV), sign), _times(d, alt),
                                                   _times(f, torch.ones(N, device=DEV))))
    w = torch.ones(*((heads, N) if per_head else (N,)), dtype=BF16, device=DEV)
    dx, dz, dw = lores.lores_gated_norm_backward(x, z, w, dy, 0.0, act=lores.LORES_ACT_NONE)
    s = (f * d).view(tokens, heads).sum(0)
    want = s[:, None] * (sign * alt)[None] if per_head else int(s.sum()) * sign * alt
    assert torch.equal(dw, want.float())
    for t in (0, (1 << 15) - 1, tokens - 2):
        assert torch.equal(dz[t:t + 2], dy[t:t + 2] * x[t:t + 2])


@pytest.mark.parametrize("M,N,K,parts", [(600, 300, 1056, (1, 5, 40, 300)), (64, 8192, 4096, (33, 50)),
                                         (200, 4096, 1056, (130, 150)), (250, 3900, 2080, (130, 201)),
                                         (250, 3900, 8224, (130, 201)), (700, 4096, 1056, (600, 530)),
                                         (2600, 4096, 544, (2304, 2100))])
def test_a_row_has_the_same_bits_in_every_batch_of_a_variant(M, N, K, parts):
    w, ws = lores.lores_mx_quant(randn((N, K), F32, 1))
    x = randn((M, K), F32, 2)
    a, as_ = lores.lores_mx_quant(x)
    top = x.abs().amax(-1) / 448.0
    e = (x / top[:, None]).to(torch.float8_e4m3fn)
    full = lores.lores_mx_matmul(a, as_, w, ws, out_prec=lores.LORES_FP32), lores.lores_mx_matmul(e, top, w, ws)
    for m in parts:
        got = (lores.lores_mx_matmul(a[:m], as_[:m], w, ws, out_prec=lores.LORES_FP32),
               lores.lores_mx_matmul(e[:m], top[:m], w, ws))
        assert all(torch.equal(g, v[:m]) for g, v in zip(got, full)), m
