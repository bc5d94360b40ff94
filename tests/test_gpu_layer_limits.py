"""The layer operators at sizes where a launch has more work-groups than a row of the
grid holds, or where places pass 32 bits."""
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


def _randn(*shape, seed=1):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV, dtype=BF16)


def test_gated_rows_of_more_than_2_21_groups():
    """2^23 work-groups of 32 rows, and one more; y = x r w s(z) of one column."""
    _needs(8)
    tokens = (1 << 26) + 9
    x, z, w = _randn(tokens, 4, 1), _randn(tokens, 4, 1, seed=2), torch.full((1,), 1.5, device=DEV)
    y, _ = lores.lores_gated_norm(x, z, w, 0.25, act=lores.LORES_ACT_SIGMOID, out_prec=lores.LORES_FP32)
    for at in range(0, tokens, 1 << 24):
        xc, zc = x[at:at + (1 << 24)].float(), z[at:at + (1 << 24)].float()
        want = xc * 1.5 / torch.sqrt(xc * xc + 0.25) / (1.0 + torch.exp(-zc))
        # some 20 roundings of 2^-24 on either side, and -z log2 e off by 2^-24 of at most 2^3
        assert ((y[at:at + (1 << 24)] - want).abs() <= 2.0 ** -18 * want.abs()).all()


def test_block_norm_of_more_than_2_32_elements():
    """The last rows of a large call are those of a small one, forward and backward."""
    _needs(100)
    rows, n = (1 << 18) + 5, 16384
    x, w = _randn(1, n).expand(rows, n), 1.0 + 0.125 * _randn(n, seed=3)
    res = torch.empty(rows, n, dtype=BF16, device=DEV)
    res[:-8] = 1.0
    res[-8:] = _randn(8, n, seed=4)
    y, _, h = lores.lores_block_norm(x, res, w, w, 1e-6)
    last = lores.lores_block_norm(x[-8:], res[-8:], w, w, 1e-6)
    assert torch.equal(y[-8:], last[0]) and torch.equal(h[-8:], last[2])
    assert torch.equal(y[:1].expand(1024, n), y[(1 << 18) - 1027:][:1024])
    dx, dres, _, dw, dwn = lores.lores_block_norm_backward(x, h, w, w, res, 1e-6, dh=y)
    part = lores.lores_block_norm_backward(x[-8:], h[-8:], w, w, res[-8:], 1e-6, dh=y[-8:])
    assert torch.equal(dx[-8:], part[0]) and torch.equal(dres[-8:], part[1])
    assert torch.isfinite(dw).all() and torch.isfinite(dwn).all()


def test_4_bit_rows_of_more_than_2_21_groups():
    """2^21 work-groups of 256 rows, and one more, of one row that stands there 2^29 times."""
    _needs(64)
    rows = (1 << 29) + 37
    x = _randn(1, 32)
    codes, scales = lores.lores_mx_quant(x.expand(rows, 32))
    one = lores.lores_mx_quant(x)
    value = lores.lores_mx_dequant(*one)
    back = lores.lores_mx_dequant(codes, scales)
    for at in range(0, rows, 1 << 25):
        assert (codes[at:at + (1 << 25)] == one[0]).all() and (scales[at:at + (1 << 25)] == one[1]).all()
        assert (back[at:at + (1 << 25)] == value).all()


@pytest.mark.parametrize("M,N,K", [(70001, 32776, 32), (70001, 32771, 64), (3, 40, 1 << 24), (270, 264, 1 << 24),
                                   (270, 1700, 1 << 24)])
@pytest.mark.parametrize("fp8", [False, True])
def test_products_beyond_32_bits(M, N, K, fp8):
    """Outputs, or places in the operands, behind 2^31; each sum has three terms, the last
    ones of the row among them."""
    _needs(48)
    i, j = torch.arange(M, device=DEV), torch.arange(N, device=DEV)
    u, v = (i % 5 + 1).float(), (j % 3 + 1).float()
    w = torch.zeros(N, K // 2, dtype=torch.uint8, device=DEV)
    ws = torch.zeros(N, (K + 127) // 128 * 4, dtype=torch.uint8, device=DEV)
    ws[:, :K // 32] = 127
    at = (0, K // 2 - 16, K - 2)                     # columns, all even
    code = torch.tensor([0, 2, 4, 5], dtype=torch.uint8, device=DEV)[v.long()]      # of 1, 2, 3
    for c in at:
        w[:, c // 2] = code
    if fp8:
        a, as_ = torch.zeros(M, K, dtype=torch.float8_e4m3fn, device=DEV), torch.ones(M, device=DEV)
        for c in at:
            a[:, c] = u.to(torch.float8_e4m3fn)
    else:
        u = torch.where(u > 4, 6.0, u)
        a = torch.zeros(M, K // 2, dtype=torch.uint8, device=DEV)
        as_ = torch.zeros(M, (K + 127) // 128 * 4, dtype=torch.uint8, device=DEV)
        as_[:, :K // 32] = 127
        row = torch.tensor([0, 2, 4, 5, 6, 0, 7], dtype=torch.uint8, device=DEV)[u.long()]
        for c in at:
            a[:, c // 2] = row
    out = lores.lores_mx_matmul(a, as_, w, ws)       # 3 u v, at most 54: exact in bf16
    times = len(set(at))
    for m in range(0, M, 8192):
        assert torch.equal(out[m:m + 8192], (times * u[m:m + 8192, None] * v).to(BF16))
