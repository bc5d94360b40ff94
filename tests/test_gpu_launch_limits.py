"""Calls with more work-groups than a row of the grid holds: 2^32 work-items along x
are more than a launch takes, and every size that the entry points allow has to
run whole."""
import pytest
import torch

import quantized_linear_recurrence_amd as lores

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


def _needs(gib):
    torch.cuda.empty_cache()
    free, _ = torch.cuda.mem_get_info()
    if free < gib << 30:
        pytest.skip(f"needs {gib} GiB of GPU memory")


def test_norm_of_more_than_2_28_rows():
    """2^24 work-groups of 16 rows and 256 threads, and three more."""
    _needs(8)
    rows = (1 << 28) + 37
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(rows, 1, generator=g, device=DEV, dtype=BF16)
    w = torch.full((1,), 1.5, device=DEV)
    y, s, _ = lores.lores_rmsnorm(x, w, 0.25, out_prec=lores.LORES_INT8)
    assert (y[x == 0] == 0).all()
    for at in range(0, rows, 1 << 26):                               # a single value's code is its sign times 127
        xc, yc, sc = x[at:at + (1 << 26), 0].float(), y[at:at + (1 << 26), 0], s[at:at + (1 << 26)]
        assert torch.equal(yc, (torch.sign(xc) * 127).to(torch.int8))
        want = xc.abs() * 1.5 / torch.sqrt(xc * xc + 0.25)
        # a dozen fp32 roundings of 2^-24
        assert ((sc * 127 - want).abs() <= 2.0 ** -20 * want).all()


def test_one_token_of_the_largest_batch():
    """65535 x 512 units by the token's kernel: 2^25 work-groups of 256 threads."""
    _needs(24)
    B, H, dk = 65535, 512, 32
    g = torch.Generator(device=DEV).manual_seed(2)
    k = torch.nn.functional.normalize(torch.randn(1, 1, H, dk, generator=g, device=DEV), dim=-1)
    q = torch.nn.functional.normalize(torch.randn(1, 1, H, dk, generator=g, device=DEV), dim=-1)
    v = torch.randn(B, 1, H, 1, generator=g, device=DEV)
    beta = torch.rand(B, 1, H, generator=g, device=DEV)
    o, S = lores.lores_scan(q.expand(B, 1, H, dk), k.expand(B, 1, H, dk), v, torch.ones_like(beta), beta, 1)
    write = v[:, 0, :, 0] * beta[:, 0]
    want = write * (q * k).sum(-1)[0]
    # 32 products and sums of 2^-24 of terms below 1
    assert ((o[:, 0, :, 0] - want).abs() <= 2.0 ** -18 * write.abs()).all()
    for at in range(0, B, 8192):
        Sc = write[at:at + 8192, :, None] * k[0]
        assert ((S[at:at + 8192, :, 0] - Sc).abs() <= 2.0 ** -22 * write[at:at + 8192, :, None].abs()).all()


def test_chunks_of_more_than_2_23_units():
    """16385 x 512 units by the passes over the chunks, forward and backward: 2^23
    work-groups of 512 threads, and 512 more."""
    _needs(220)
    B, H, T, dk, dv = 16385, 512, 9, 32, 4
    g = torch.Generator(device=DEV).manual_seed(3)
    k = torch.nn.functional.normalize(torch.randn(1, T, H, dk, generator=g, device=DEV), dim=-1)
    q = torch.nn.functional.normalize(torch.randn(1, T, H, dk, generator=g, device=DEV), dim=-1)
    v = torch.randn(B, T, H, dv, generator=g, device=DEV)
    alpha = 0.5 + 0.5 * torch.rand(B, T, H, generator=g, device=DEV)
    beta = torch.rand(B, T, H, generator=g, device=DEV)
    args = (q.expand(B, T, H, dk), k.expand(B, T, H, dk))

    def near(a, b):                                  # sums of some hundred terms in fp32
        assert float((a.double() - b.double()).norm()) <= 2.0 ** -19 * float(b.double().norm()) + 1e-30

    got = lores.lores_scan(*args, v, alpha, beta, 0)
    parts = (slice(0, 40), slice(8000, 8040), slice(B - 40, B))
    for s in parts:                                  # 40 sequences alone: a launch of 20480 units
        want = lores.lores_scan(args[0][s], args[1][s], v[s], alpha[s].contiguous(), beta[s].contiguous(), 0)
        for x, y in zip(got, want):
            near(x[s], y)
    del got, want
    torch.cuda.empty_cache()
    do = v.flip(1)
    grads = lores.lores_scan_backward(*args, v, alpha, beta, 0, do)
    for s in parts:
        want = lores.lores_scan_backward(args[0][s], args[1][s], v[s], alpha[s].contiguous(), beta[s].contiguous(), 0,
                                         do[s].contiguous())
        for x, y in zip(grads, want):
            near(x[s], y)
