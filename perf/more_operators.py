"""Cases and plain forms of the operators around the recurrence: the gated norm
behind it and the norms around a block (forward, and forward with backward), and
microscaled 4-bit rows (blocks of 32 E2M1 values with a power-of-two scale):
their quantisation and their matrix product.

With `own` false, run() computes the operators with elementary torch operations
in fp32; with `own` true it calls the package's kernels.  exact() computes the
same outputs in fp64.
"""
import math

import torch

own = False

_BF16, _F32 = "bf16", "fp32"
_EPS = 1e-6


# ------------------------------------------------------------------ cases

def _gated(name, op, tokens, heads, n, dtype, act, gate_first=False, per_head=False, wide=True):
    return {"name": name, "op": op, "tokens": tokens, "heads": heads, "n": n, "dtype": dtype,
            "act": act, "gate_first": gate_first, "per_head": per_head, "wide": wide}


def _block(name, op, rows, n, dtype, gate, post, scale):
    return {"name": name, "op": op, "rows": rows, "n": n, "dtype": dtype, "gate": gate,
            "post": post, "scale": scale}


def _quant(name, rows, K, dtype):
    return {"name": name, "op": "quant", "rows": rows, "K": K, "dtype": dtype}


def _product(name, M, N, K, a, out):
    return {"name": name, "op": "product", "M": M, "N": N, "K": K, "a": a, "out": out}


def listed():
    return [
        # the readout of a decode batch, 32 heads, gated before the output projection: latency
        _gated("gated_token", "gated", 64, 32, 128, _BF16, "silu"),
        # a training step's gated norm: four sequences of 2048 tokens
        _gated("gated_train", "gated_train", 8192, 32, 128, _BF16, "silu"),
        # gate before a norm over groups with their own weights, odd width, fp32, uneven tokens
        _gated("gated_odd", "gated_train", 777, 5, 100, _F32, "silu", True, True, False),
        # norm after a block and before the next one, a decode batch: latency
        _block("block_token", "block", 64, 4096, _BF16, "", True, 0.5),
        # the same around a gated block in a training step, forward and backward
        _block("block_train", "block_train", 16384, 4096, _BF16, "sigmoid", True, 0.5),
        # a decode batch's rows to 4 bits and back
        _quant("quant_rows", 64, 4096, _BF16),
        # a projection's weights to 4 bits and back (a checkpoint that is loaded)
        _quant("quant_weight", 8192, 4096, _BF16),
        # one token through a projection: the weights' bytes and latency
        _product("product_token", 1, 8192, 4096, "mx", _BF16),
        # a decode batch: residual and norm to 4-bit rows, then the projection
        {"name": "norm_product", "op": "norm_product", "M": 64, "N": 8192, "K": 4096,
         "dtype": _BF16},
        # prompts of 8192 tokens in all through the projection
        _product("product_prompt", 8192, 8192, 4096, "mx", _BF16),
        # the same projection on E4M3 rows with one factor per row
        _product("product_fp8", 4096, 8192, 4096, "fp8", _BF16),
        # uneven prompt, odd widths, a last block inside a tile, fp32 out
        _product("product_odd", 777, 1000, 1056, "mx", _F32),
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "gated_train", "block", "block_train", "quant", "product", "product",
                     "norm_product"])
    dtype = rng.choice([_BF16, _BF16, _F32])
    size = 2 if dtype == _BF16 else 4
    if op.startswith("gated"):
        n = rng.choice([64, 128, 128, 256, _between(rng, 16, 4096)])
        heads = _between(rng, 1, max(1, min(64, 8192 // n)))
        tokens = _between(rng, 1, min(32768, (1 << 25) * 2 // size // (heads * n)))
        return {"op": op, "tokens": tokens, "heads": heads, "n": n, "dtype": dtype,
                "act": rng.choice(["silu", "silu", "sigmoid"]), "gate_first": rng.random() < 0.4,
                "per_head": rng.random() < 0.4, "wide": rng.random() < 0.6}
    if op.startswith("block"):
        n = rng.choice([8 * _between(rng, 8, 1024), _between(rng, 64, 8192)])
        rows = _between(rng, 1, min(16384, (1 << 25) * 2 // size // n))
        return {"op": op, "rows": rows, "n": n, "dtype": dtype,
                "gate": rng.choice(["", "", "sigmoid", "silu", "none"]),
                "post": rng.random() < 0.7, "scale": rng.choice([1.0, 0.5, 0.22])}
    K = 32 * _between(rng, 1, 256)
    if op == "quant":
        return {"op": op, "rows": _between(rng, 1, min(16384, (1 << 25) // K)), "K": K,
                "dtype": dtype}
    N = rng.choice([64 * _between(rng, 1, 128), _between(rng, 16, 8192)])
    if op == "norm_product":
        return {"op": op, "M": _between(rng, 1, min(2048, (1 << 30) // (N * K) * 16 + 1)), "N": N,
                "K": K, "dtype": dtype}
    # at most half the operations of the largest listed case
    most = 8192 * 8192 * 4096 // 2
    a = rng.choice(["mx", "mx", "fp8"])                  # E4M3 rows give bf16
    return {"op": op, "M": _between(rng, 1, max(1, min(8192, most // (N * K)))), "N": N, "K": K,
            "a": a, "out": rng.choice([_BF16, _BF16, _F32]) if a == "mx" else _BF16}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    return g


def _type(name):
    return torch.bfloat16 if name == _BF16 else torch.float32


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    dt = _type(case.get("dtype", _BF16))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": case}
    if op.startswith("gated"):
        T, H, n = case["tokens"], case["heads"], case["n"]
        # a readout's heads differ in size with their decay
        s["x"] = (randn(T, H, n) * torch.exp(randn(H, 1))).to(dt)
        z = randn(T, (2 if case["wide"] else 1) * H * n).to(dt)
        # the gate is the second half of a wider projection's rows, or stands alone
        s["gate"] = z[:, -H * n:].view(T, H, n)
        s["w"] = (1.0 + 0.1 * randn(*((H, n) if case["per_head"] else (n,)))).to(dt)
        if op == "gated_train":
            s["dy"] = randn(T, H, n).to(dt)
        return s
    if op.startswith("block"):
        rows, n = case["rows"], case["n"]
        s["x"] = (0.2 * randn(rows, n)).to(dt)       # a block's output before its norm
        s["res"] = (3.0 * randn(rows, n)).to(dt)     # the residual stream
        s["w1"] = (1.0 + 0.1 * randn(n)).to(dt) if case["post"] else None
        s["w2"] = (1.0 + 0.1 * randn(n)).to(dt)
        s["gate"] = randn(rows, n).to(dt) if case["gate"] else None
        if op == "block_train":
            s["dy"] = randn(rows, n).to(dt)
            s["dh"] = randn(rows, n).to(dt)
        return s
    if op == "quant":
        # rows whose blocks differ in size, some blocks of zeros, and large single values
        rows, K = case["rows"], case["K"]
        x = randn(rows, K // 32, 32) * torch.exp(2.0 * randn(rows, K // 32, 1))
        x = x * (torch.rand(rows, K // 32, 1, generator=g, device="cuda") > 0.02)
        x = torch.where(torch.rand(x.shape, generator=g, device="cuda") < 0.005, 20.0 * x, x)
        s["x"] = x.view(rows, K).to(dt)
        return s
    M, N, K = case["M"], case["N"], case["K"]
    # the weights as such a program keeps them: 4-bit codes and their scales
    s["w"], s["w_scales"] = _pack(randn(N, K) / math.sqrt(K))
    if op == "norm_product":
        s["x"], s["res"] = randn(M, K).to(dt), (3.0 * randn(M, K)).to(dt)
        s["norm"] = (1.0 + 0.1 * randn(K)).to(dt)
    elif case["a"] == "mx":
        s["a"], s["a_scales"] = _pack(randn(M, K))
    else:
        a = randn(M, K)
        top = a.abs().amax(-1, keepdim=True) / 448.0
        s["a"], s["a_scales"] = (a / top).to(torch.float8_e4m3fn), top[:, 0].contiguous()
    return s


# ------------------------------------------------------------------ 4-bit blocks, plain

def _blocks(x):
    """Codes 0..15 and biased exponents of fp32 rows [R, K] in blocks of 32."""
    b = x.view(x.shape[0], -1, 32)
    m = b.abs().amax(-1)
    # the exponent carries where the mantissa is at least 1.75: the largest value
    # is then below 7 units, and rounds to 6 at most
    e = ((m.view(torch.int32) + (1 << 21)) >> 23) - 129
    e = e.clamp(-127, 127)
    q = torch.ldexp(b, -e[..., None]).abs()
    c = (q > 0.25).int() + (q >= 0.75) + (q > 1.25) + (q >= 1.75) + (q > 2.5) + (q >= 3.5) + (q > 5.0)
    return (c + 8 * torch.signbit(b)).view(x.shape), e + 127


def _pack(x):
    """Rows [R, K] as codes [R, K / 2] (the even column in the low half of a byte)
    and scales [R, 4 ceil(K / 128)], 0 behind the last block."""
    c, e = _blocks(x.contiguous())
    codes = (c[:, 0::2] + 16 * c[:, 1::2]).to(torch.uint8)
    scales = torch.zeros(x.shape[0], (x.shape[1] + 127) // 128 * 4, dtype=torch.uint8, device=x.device)
    scales[:, :e.shape[1]] = e.to(torch.uint8)
    return codes, scales


_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _stand_for(c, e):
    """The values of codes [R, K] and biased exponents [R, K / 32]."""
    grid = torch.tensor(_GRID + tuple(-v for v in _GRID), device=c.device)
    return torch.ldexp(grid[c].view(c.shape[0], -1, 32), (e - 127)[..., None]).view(c.shape)


def _unpack(codes, scales):
    c = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1).long()
    return _stand_for(c, scales[:, :c.shape[1] // 32].int())


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        import quantized_linear_recurrence_amd as lores
        return _own(lores, op, s)
    if op.startswith("gated"):
        return _gated_plain(s)
    if op.startswith("block"):
        return _block_plain(s)
    if op == "quant":
        return _stand_for(*_whole_codes(s["x"])).to(s["x"].dtype)
    out = {}
    if op == "norm_product":
        h = (s["x"].float() + s["res"].float()).to(s["x"].dtype)
        hf = h.float()
        y = hf / torch.sqrt((hf * hf).mean(-1, keepdim=True) + _EPS) * s["norm"].float()
        out["h"] = h
        a = _stand_for(*_whole_codes(y))
    elif s["case"]["a"] == "mx":
        a = _unpack(s["a"], s["a_scales"])
    else:
        a = s["a"].float() * s["a_scales"][:, None]
    out["out"] = (a @ _unpack(s["w"], s["w_scales"]).T).to(_type(s["case"].get("out", _BF16)))
    return out


def _whole_codes(x):
    c, e = _blocks(x.float())
    return c.long(), e


def _own(lores, op, s):
    case = s["case"]
    acts = {"": lores.LORES_ACT_NONE, "none": lores.LORES_ACT_NONE, "silu": lores.LORES_ACT_SILU,
            "sigmoid": lores.LORES_ACT_SIGMOID}
    if op.startswith("gated"):
        kw = {"act": acts[case["act"]], "gate_first": case["gate_first"]}
        out = {"y": lores.lores_gated_norm(s["x"], s["gate"], s["w"], _EPS, **kw)[0]}
        if op == "gated_train":
            out["dx"], out["dgate"], out["dw"] = lores.lores_gated_norm_backward(
                s["x"], s["gate"], s["w"], s["dy"], _EPS, **kw)
        return out
    if op.startswith("block"):
        kw = {"scale": case["scale"], "gate": s["gate"], "act": acts[case["gate"]]}
        y, _, h = lores.lores_block_norm(s["x"], s["res"], s["w1"], s["w2"], _EPS, **kw)
        out = {"y": y, "h": h}
        if op == "block_train":
            out["dx"], out["dres"], dgate, dw1, out["dw2"] = lores.lores_block_norm_backward(
                s["x"], h, s["w1"], s["w2"], s["dy"], _EPS, dh=s["dh"], **kw)
            out.update({} if s["gate"] is None else {"dgate": dgate})
            out.update({} if s["w1"] is None else {"dw1": dw1})
        return out
    if op == "quant":
        return lores.lores_mx_dequant(*lores.lores_mx_quant(s["x"]), dtype=s["x"].dtype)
    if op == "norm_product":
        codes, scales, h = lores.lores_block_norm(s["x"], s["res"], None, s["norm"], _EPS,
                                                  out_prec=lores.LORES_MXFP4)
        return {"h": h, "out": lores.lores_mx_matmul(codes, scales, s["w"], s["w_scales"])}
    prec = lores.LORES_BF16 if case["out"] == _BF16 else lores.LORES_FP32
    return {"out": lores.lores_mx_matmul(s["a"], s["a_scales"], s["w"], s["w_scales"], out_prec=prec)}


# ------------------------------------------------------------------ the norms, plain

def _act(kind, z):
    """A gate's activation and its slope."""
    if kind == "none":
        return z, torch.ones_like(z)
    sg = 1.0 / (1.0 + torch.exp(-z))
    if kind == "sigmoid":
        return sg, sg * (1.0 - sg)
    return z * sg, sg * (1.0 + z * (1.0 - sg))


def _unit(x):
    """1 / root mean square of the rows."""
    return 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + _EPS)


def _through(e, n, r):
    """The gradient that passes a norm n = x r, from that of n."""
    return r * (e - n * (e * n).mean(-1, keepdim=True))


def _gated_plain(s):
    case, dt = s["case"], s["x"].dtype
    x, z, w = s["x"].float(), s["gate"].float(), s["w"].float()
    a, slope = _act(case["act"], z)
    u = x * a if case["gate_first"] else x
    r = _unit(u)
    n = u * r
    b = 1.0 if case["gate_first"] else a                 # what multiplies the weighted norm
    out = {"y": (n * w * b).to(dt)}
    if case["op"] == "gated_train":
        dy = s["dy"].float()
        du = _through(dy * w * b, n, r)
        if case["gate_first"]:
            out["dx"], out["dgate"] = (du * a).to(dt), (du * x * slope).to(dt)
        else:
            out["dx"], out["dgate"] = du.to(dt), (dy * w * n * slope).to(dt)
        over = (0,) if case["per_head"] else (0, 1)
        out["dw"] = (dy * n * b).sum(over, dtype=torch.float64).float()
    return out


def _block_plain(s):
    case, dt, sc = s["case"], s["x"].dtype, s["case"]["scale"]
    x, w2 = s["x"].float(), s["w2"].float()
    a, slope = (1.0, None) if s["gate"] is None else _act(case["gate"], s["gate"].float())
    w1 = 1.0 if s["w1"] is None else s["w1"].float()
    r1 = None if s["w1"] is None else _unit(x)
    n1 = x if r1 is None else x * r1
    h = (s["res"].float() + sc * a * n1 * w1).to(dt)
    hf = h.float()
    r2 = _unit(hf)
    n2 = hf * r2
    out = {"y": (n2 * w2).to(dt), "h": h}
    if case["op"] == "block_train":
        dy = s["dy"].float()
        G = s["dh"].float() + _through(dy * w2, n2, r2)
        e = sc * G * a * w1
        out["dx"] = (e if r1 is None else _through(e, n1, r1)).to(dt)
        out["dres"] = G.to(dt)
        out["dw2"] = (dy * n2).sum(0, dtype=torch.float64).float()
        if slope is not None:
            out["dgate"] = (sc * G * n1 * w1 * slope).to(dt)
        if r1 is not None:
            out["dw1"] = (sc * G * a * n1).sum(0, dtype=torch.float64).float()
    return out


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("gated"):
        return _gated_exact(s)
    if case["op"].startswith("block"):
        return _block_exact(s)
    if case["op"] == "quant":
        return _nearest(s["x"].double())
    w = _read(s["w"], s["w_scales"])
    if case["op"] == "norm_product":
        h = s["x"].double() + s["res"].double()
        k = h.to(s["x"].dtype).double()              # the stream is kept in the inputs' type
        y = k * s["norm"].double() * (k.square().mean(-1, keepdim=True) + _EPS).rsqrt()
        return {"h": h, "out": torch.matmul(_nearest(y), w.t())}
    if case["a"] == "mx":
        a = _read(s["a"], s["a_scales"])
    else:
        a = s["a"].float().double() * s["a_scales"].double().unsqueeze(1)
    return {"out": torch.matmul(a, w.t())}


def _nearest(x):
    """Rows as the nearest values of their blocks: the grid's neighbours on both
    sides are found by search, ties go to the even code."""
    R, K = x.shape
    b = x.reshape(R, K // 32, 32)
    f, k = torch.frexp(b.abs().max(-1).values)
    e = torch.where(f < 0.875, k - 3, k - 2).clamp(-127, 127).double()
    e = torch.where(f == 0.0, -127.0, e).unsqueeze(-1)
    q = b.abs() * torch.exp2(-e)
    grid = torch.tensor(_GRID, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(grid, q.contiguous()).clamp(1, 7)
    lo = hi - 1
    up, down = grid[hi] - q, q - grid[lo]
    v = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), grid[hi], grid[lo])
    return (v * torch.exp2(e) * b.sign()).reshape(R, K)


def _read(codes, scales):
    """Codes byte by byte: exponent and fraction fields of each half."""
    R, half = codes.shape
    v = torch.empty(R, half, 2, dtype=torch.float64, device=codes.device)
    for i in range(2):
        c = (codes.int() >> (4 * i)) & 15
        ex, fr = (c >> 1) & 3, (c & 1).double()
        size = torch.where(ex == 0, 0.5 * fr, torch.exp2((ex - 1).double()) * (1.0 + 0.5 * fr))
        v[..., i] = torch.where(c >= 8, -size, size)
    unit = torch.exp2(scales[:, :half // 16].double() - 127.0)
    return (v.reshape(R, half // 16, 32) * unit.unsqueeze(-1)).reshape(R, 2 * half)


def _gate64(kind, z):
    if kind == "none":
        return z, torch.ones_like(z)
    sg = torch.sigmoid(z)
    if kind == "sigmoid":
        return sg, sg - sg * sg
    return z * sg, sg + z * sg - z * sg * sg


def _norm64(u, w, g):
    """norm(u) w, and the gradients of u and (row by row) of w from g."""
    r = (u.pow(2).mean(-1, keepdim=True) + _EPS).rsqrt()
    y = u * w * r
    if g is None:
        return y, None, None
    t = (g * w * u).mean(-1, keepdim=True)
    return y, g * w * r - u * t * r.pow(3), g * u * r


def _gated_exact(s):
    case = s["case"]
    x, z, w = (s[k].double() for k in ("x", "gate", "w"))
    dy = s["dy"].double() if "dy" in s else None
    a, slope = _gate64(case["act"], z)
    if case["gate_first"]:
        y, du, rows = _norm64(x * a, w, dy)
        grads = None if dy is None else (du * a, du * x * slope)
    else:
        n, du, rows = _norm64(x, w, None if dy is None else dy * a)
        y = n * a
        grads = None if dy is None else (du, dy * n * slope)
    out = {"y": y}
    if dy is not None:
        out["dx"], out["dgate"] = grads
        out["dw"] = rows.sum(0) if case["per_head"] else rows.sum((0, 1))
    return out


def _block_exact(s):
    case, dt = s["case"], s["x"].dtype
    x, w2 = s["x"].double(), s["w2"].double()
    gate = None if s["gate"] is None else _gate64(case["gate"], s["gate"].double())
    a = torch.ones_like(x) if gate is None else gate[0]
    w1 = None if s["w1"] is None else s["w1"].double()
    p = x if w1 is None else _norm64(x, w1, None)[0]
    h = s["res"].double() + case["scale"] * a * p
    dy = s["dy"].double() if "dy" in s else None
    y, dh, rows = _norm64(h.to(dt).double(), w2, dy)     # the norm is of what is kept
    out = {"y": y, "h": h}
    if dy is not None:
        G = dh + s["dh"].double()
        out["dres"], out["dw2"] = G, rows.sum(0)
        out["dx"] = case["scale"] * G * a
        if gate is not None:
            out["dgate"] = case["scale"] * G * p * gate[1]
        if w1 is not None:
            _, out["dx"], rows = _norm64(x, w1, out["dx"])
            out["dw1"] = rows.sum(0)
    return out


# ------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    size = 2 if case.get("dtype", _BF16) == _BF16 else 4
    if op.startswith("gated"):
        rows, n = case["tokens"] * case["heads"], case["n"]
        nw = n * (case["heads"] if case["per_head"] else 1)
        b = 3 * rows * n * size + nw * size                  # x, gate read, y written
        if op == "gated_train":
            b += 3 * rows * n * size + 4 * nw                # dy read, dx, dgate and dw written
        return {"bytes": b, "flops": rows * n * (10 if op == "gated" else 30)}
    if op.startswith("block"):
        rows, n = case["rows"], case["n"]
        gate, nw = 1 if case["gate"] else 0, n * (2 if case["post"] else 1)
        b = (4 + gate) * rows * n * size + nw * size         # x, res, gate read, h, y written
        if op == "block_train":
            b += (4 + gate) * rows * n * size + 4 * nw       # dy, dh read, dx, dres, dgate written
        return {"bytes": b, "flops": rows * n * (12 if op == "block" else 40)}
    mx = 17.0 / 32.0                                         # bytes a 4-bit value takes
    if op == "quant":                                        # codes written and read on the way
        return {"bytes": case["rows"] * case["K"] * (2 * size + 2 * mx),
                "flops": 4 * case["rows"] * case["K"]}
    M, N, K = case["M"], case["N"], case["K"]
    out = 4 if case.get("out") == _F32 else 2
    b = N * K * mx + M * N * out
    if op == "norm_product":
        b += 3 * M * K * size                                # x, residual read, their sum written
    else:
        b += M * K * mx if case["a"] == "mx" else M * K + 4 * M
    return {"bytes": b, "flops": 2 * M * N * K}
