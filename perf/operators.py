"""Cases and plain forms of the sequence operators: the gated linear recurrence
over whole sequences (forward, and forward with backward), and the
root-mean-square norm with residual and 8-bit outputs (forward, and backward).

With `own` false, run() computes the operators with elementary torch operations
in fp32; with `own` true it calls the package's kernels.  exact() computes the
same outputs token by token (the recurrence) or row by row (the norm) in fp64.
"""
import math

import torch

own = False

_CHUNK = 64
_BF16, _F32 = "bf16", "fp32"


# ------------------------------------------------------------------ cases

def _scan(name, op, B, T, H, Hk, dk, dv, dtype, delta, decay, state, ragged=False):
    return {"name": name, "op": op, "B": B, "T": T, "H": H, "Hk": Hk, "dk": dk, "dv": dv,
            "dtype": dtype, "delta": delta, "decay": decay, "state": state, "ragged": ragged}


def _norm(name, op, rows, n, dtype, out, residual):
    return {"name": name, "op": op, "rows": rows, "n": n, "dtype": dtype, "out": out,
            "residual": residual}


def listed():
    return [
        # one more token for a batch that decodes at fp32 state: latency and the state's bytes
        _scan("scan_token", "scan", 64, 1, 32, 32, 128, 128, _BF16, 1, "head", True),
        # a short prompt of the smallest layer: launches and latency
        _scan("scan_short", "scan", 1, 128, 2, 2, 64, 64, _F32, 1, "step", False),
        # one user's prompt through a gated delta layer: few heads, a long axis
        _scan("scan_prompt", "scan", 1, 4096, 32, 32, 128, 128, _BF16, 1, "head", False),
        # a batch of long prompts through the same layer: throughput
        _scan("scan_prompts", "scan", 8, 4096, 32, 32, 128, 128, _BF16, 1, "head", False),
        # prompts of uneven lengths (0 and 1 among them) continued from a state, odd sizes, fp32
        _scan("scan_ragged", "scan", 8, 777, 5, 5, 96, 100, _F32, 1, "step", True, True),
        # a layer without the delta correction whose heads share q and k: prompt
        _scan("scan_shared", "scan", 4, 2048, 128, 8, 128, 64, _BF16, 0, "ssd", False),
        # a training step of the gated delta layer
        _scan("train_delta", "train", 4, 2048, 32, 32, 128, 128, _BF16, 1, "head", False),
        # a training step of the layer without correction, shared q and k
        _scan("train_shared", "train", 2, 2048, 64, 4, 128, 64, _BF16, 0, "ssd", False),
        # a small fp32 step over uneven lengths with a state at both ends
        _scan("train_ragged", "train", 3, 333, 3, 3, 96, 100, _F32, 1, "step", True, True),
        # the layer norm of a decode batch, in 8 bits for the projection behind it
        _norm("norm_token", "norm", 64, 4096, _BF16, "int8", True),
        # the norm of the readout's heads at a large batch, E4M3 out
        _norm("norm_heads", "norm", 65536, 128, _F32, "fp8", False),
        # the layer norm of a training step, forward and backward
        _norm("norm_train", "norm_train", 16384, 4096, _BF16, "same", True),
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan", "train", "train", "norm", "norm", "norm_train"])
    dtype = rng.choice([_BF16, _BF16, _F32])
    if op.startswith("norm"):
        n = _between(rng, 64, 8192)
        rows = _between(rng, 1, min(65536, (1 << 26) // n))
        out = "same" if op == "norm_train" else rng.choice(["same", "int8", "fp8"])
        return {"op": op, "rows": rows, "n": n, "dtype": dtype, "out": out,
                "residual": rng.random() < 0.7}
    dk = 32 * rng.choice([1, 2, 2, 3, 4, 4, 4, 5, 6, 7, 8])
    dv = rng.choice([rng.randint(1, 256), 64, 128, 128])
    G = rng.choice([1, 1, 2, 4])
    Hk = _between(rng, 1, 32)
    B = _between(rng, 1, 16)
    # at most half the tokens x heads x widths of the largest listed cases
    most = (8 * 4096 * 32 * 256 // 2) if op == "scan" else (4 * 2048 * 32 * 256 // 2)
    T = _between(rng, 1, max(1, min(4096, most // (B * Hk * G * (dk + dv)))))
    decay = rng.choice(["head", "step", "ssd"])
    return {"op": op, "B": B, "T": T, "H": Hk * G, "Hk": Hk, "dk": dk, "dv": dv, "dtype": dtype,
            "delta": 0 if decay == "ssd" else rng.choice([0, 1, 1]), "decay": decay,
            "state": rng.random() < 0.5, "ragged": rng.random() < 0.4}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    return g


def _torch_dtype(case):
    return torch.bfloat16 if case["dtype"] == _BF16 else torch.float32


def prepare(case, seed):
    g, dt = _gen(seed), _torch_dtype(case)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"].startswith("norm"):
        rows, n = case["rows"], case["n"]
        s = {"case": case, "eps": 1e-6, "x": randn(rows, n).to(dt),
             "w": (1.0 + 0.1 * randn(n)).to(dt)}
        # the residual stream is wider than what one layer adds to it
        s["res"] = (3.0 * randn(rows, n)).to(dt) if case["residual"] else None
        if case["op"] == "norm_train":
            s["dy"] = randn(rows, n).to(dt)
            s["dres"] = randn(rows, n).to(dt) if case["residual"] else None
        return s
    B, T, H, Hk, dk, dv = (case[x] for x in ("B", "T", "H", "Hk", "dk", "dv"))
    s = {"case": case}
    for name in ("q", "k"):                      # unit rows, as the layer normalises them
        x = randn(B, T, Hk, dk)
        s[name] = (x / x.norm(dim=-1, keepdim=True)).to(dt)
    s["v"] = randn(B, T, H, dv).to(dt)
    s["beta"] = 2.0 * torch.sigmoid(randn(B, T, H))
    if case["decay"] == "head":                  # one decay per head
        a = 0.85 + 0.15 * torch.rand(H, generator=g, device="cuda")
        s["alpha"] = a.expand(B, T, H).contiguous()
    elif case["decay"] == "step":                # one per token and head, slow
        s["alpha"] = torch.exp(-torch.nn.functional.softplus(randn(B, T, H) - 3.0))
    else:                                        # exp(-dt A) and write gate dt
        A = 1.0 + 15.0 * torch.rand(H, generator=g, device="cuda")
        step = torch.nn.functional.softplus(randn(B, T, H) - 2.0)
        s["alpha"] = torch.exp(-step * A)
        s["beta"] = step
    s["S0"] = randn(B, H, dv, dk) * 0.3 if case["state"] else None
    s["lengths"] = None
    if case["ragged"]:
        n = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        n[0] = T                                 # the batch is as long as its longest
        if B > 1:
            n[1] = min(1, T)
        if B > 2:
            n[2] = 0
        s["lengths"] = n
    if case["op"] == "train":
        s["do"] = randn(B, T, H, dv).to(dt)
        s["dS"] = randn(B, H, dv, dk) * 0.3 if case["state"] else None
    if case["ragged"]:                           # nothing behind a sequence's end is a number
        pad = torch.arange(T, device="cuda")[None, :] >= s["lengths"][:, None]
        for name in ("q", "k", "v", "alpha", "beta", "do"):
            if name in s:
                s[name][pad] = float("nan")
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        import quantized_linear_recurrence_amd as lores
        return _own(lores, op, s)
    if op == "norm":
        return _norm_plain(s)
    if op == "norm_train":
        return _norm_train_plain(s)
    return _scan_plain(s, op == "train")


def _own(lores, op, s):
    if op in ("norm", "norm_train"):
        prec = {"int8": lores.LORES_INT8, "fp8": lores.LORES_FP8, "same": None}[s["case"]["out"]]
        y, scales, h = lores.lores_rmsnorm(s["x"], s["w"], s["eps"], residual=s["res"],
                                           out_prec=prec)
        out = {"y": y, "scales": scales, "h": h if s["res"] is not None else None}
        if op == "norm_train":
            out["dx"], out["dw"] = lores.lores_rmsnorm_backward(h, s["w"], s["dy"], s["eps"],
                                                                dresidual=s["dres"])
        return out
    delta = s["case"]["delta"]
    x = (s["q"], s["k"], s["v"], s["alpha"], s["beta"], delta)
    o, S = lores.lores_scan(*x, S0=s["S0"], lengths=s["lengths"])
    out = {"o": o, "S": S}
    if op == "train":
        dq, dk, dv, da, db, dS0 = lores.lores_scan_backward(*x, s["do"], dS=s["dS"], S0=s["S0"],
                                                            lengths=s["lengths"])
        out.update(dq=dq, dk=dk, dv=dv, dalpha=da, dbeta=db, dS0=dS0)
    return out


# ------------------------------------------------------------------ the norm

def _norm_plain(s):
    dt, kind = s["x"].dtype, s["case"]["out"]
    h = s["x"]
    if s["res"] is not None:
        h = (h.float() + s["res"].float()).to(dt)
    hf = h.float()
    z = hf * s["w"].float()
    rstd = 1.0 / torch.sqrt((hf * hf).mean(-1) + s["eps"])
    out = {"h": h if s["res"] is not None else None, "scales": None}
    if kind == "same":
        out["y"] = (z * rstd[:, None]).to(dt)
        return out
    top = 127.0 if kind == "int8" else 448.0
    m = z.abs().amax(-1)
    c = z * (top / m.clamp_min(2.0 ** -119))[:, None]
    out["y"] = torch.round(c).to(torch.int8) if kind == "int8" else c.to(torch.float8_e4m3fn)
    out["scales"] = m / top * rstd
    return out


def _norm_train_plain(s):
    out = _norm_plain(s)
    h = s["x"] if out["h"] is None else out["h"]
    hf, w, dy = h.float(), s["w"].float(), s["dy"].float()
    rstd = 1.0 / torch.sqrt((hf * hf).mean(-1, keepdim=True) + s["eps"])
    n = hf * rstd
    g = w * dy
    dx = rstd * (g - n * (g * n).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    out["dx"] = dx.to(h.dtype)
    out["dw"] = (dy * n).sum(0)
    return out


# ------------------------------------------------------------------ the recurrence

def _chunks(x, n, C, fill=0.0):
    """[B, T, H, ...] -> [B, H, n, C, ...], `fill` behind T."""
    B, T = x.shape[:2]
    if n * C != T:
        x = torch.cat([x, x.new_full((B, n * C - T, *x.shape[2:]), fill)], 1)
    return x.reshape(B, n, C, *x.shape[2:]).transpose(2, 3).transpose(1, 2)


def _tokens(x, T):
    """[B, H, n, C, ...] -> [B, T, H, ...]."""
    B, H, n, C = x.shape[:4]
    x = x.permute(0, 2, 3, 1, *range(4, x.dim())).reshape(B, n * C, H, *x.shape[4:])
    return x[:, :T]


def _scan_plain(s, train):
    """Chunks of C tokens: products within a chunk for all chunks at once, one
    pass over the chunks for the state, and one back for its gradient."""
    case = s["case"]
    B, T, H, Hk, dk, dv = (case[x] for x in ("B", "T", "H", "Hk", "dk", "dv"))
    delta, dt, G, C = case["delta"], s["q"].dtype, H // Hk, min(_CHUNK, T)
    n = -(-T // C)
    f = {x: s[x].float() for x in ("q", "k", "v", "alpha", "beta", "do") if x in s}
    if s["lengths"] is not None:
        pad = torch.arange(T, device="cuda")[None, :] >= s["lengths"][:, None]
        for x in f:
            f[x] = f[x].masked_fill(pad.view(B, T, *([1] * (f[x].dim() - 2))),
                                    1.0 if x == "alpha" else 0.0)
    if G > 1:
        f["q"], f["k"] = (f[x].repeat_interleave(G, 2) for x in "qk")
    q, k, v, b = (_chunks(f[x], n, C) for x in ("q", "k", "v", "beta"))
    a = _chunks(f["alpha"], n, C, 1.0)                  # padded tokens do not decay
    i = torch.arange(C, device="cuda")
    low, strict = i[:, None] >= i[None, :], i[:, None] > i[None, :]
    # D[i, j] = prod of alpha over j < l <= i
    D = torch.cumprod(torch.where(strict, a[..., :, None], 1.0), -2).masked_fill(~low, 0.0)
    gam = torch.cumprod(a, -1)
    end = D[..., -1, :]                                 # decay from j to the chunk's end
    kT = k.transpose(-1, -2).contiguous()
    qk, P = q @ kT, None
    P = qk * D
    if delta:
        kk = k @ kT
        M = (kk * D).masked_fill(~strict, 0.0)
        N = -b[..., :, None] * M                        # (I - N)^-1: N is nilpotent
        X, e = torch.eye(C, device="cuda") + N, 1
        while 2 * e < C:
            N = N @ N
            X, e = X + X @ N, 2 * e
    S = torch.zeros(B, H, dv, dk, device="cuda") if s["S0"] is None else s["S0"]
    St = S.transpose(-1, -2).contiguous()               # [dk, dv]
    starts, us = [], []
    gk, gq, ek = gam[..., None] * k, gam[..., None] * q, (end[..., None] * k).transpose(-1, -2).contiguous()
    bv = b[..., None] * v
    Xbv = X @ bv if delta else bv
    Xbk = X @ (b[..., None] * gk) if delta else None
    for c in range(n):
        starts.append(St)
        u = Xbv[:, :, c] - Xbk[:, :, c] @ St if delta else Xbv[:, :, c]
        us.append(u)
        St = gam[:, :, c, -1, None, None] * St + ek[:, :, c] @ u
    S0t, U = torch.stack(starts, 2), torch.stack(us, 2)
    out = {"o": _tokens(gq @ S0t + P @ U, T).to(dt), "S": St.transpose(-1, -2).contiguous()}
    if not train:
        return out
    do = _chunks(f["do"], n, C)
    dS = torch.zeros(B, H, dv, dk, device="cuda") if s["dS"] is None else s["dS"]
    dSt = dS.transpose(-1, -2).contiguous()             # [dk, dv]
    Pdo = P.transpose(-1, -2).contiguous() @ do
    XT = X.transpose(-1, -2).contiguous() if delta else None
    ends, hs, ekt = [None] * n, [None] * n, end[..., None] * k
    qTdo = gq.transpose(-1, -2).contiguous() @ do
    bgkT = (b[..., None] * gk).transpose(-1, -2).contiguous()
    for c in reversed(range(n)):
        ends[c] = dSt
        h = Pdo[:, :, c] + ekt[:, :, c] @ dSt
        if delta:
            h = XT[:, :, c] @ h
        hs[c] = h
        dSt = gam[:, :, c, -1, None, None] * dSt + qTdo[:, :, c]
        if delta:
            dSt = dSt - bgkT[:, :, c] @ h
    dSe, h = torch.stack(ends, 2), torch.stack(hs, 2)
    bh = b[..., None] * h
    S0d, UT = S0t.transpose(-1, -2).contiguous(), U.transpose(-1, -2).contiguous()
    dP = (do @ UT).masked_fill(~low, 0.0)
    sdo = do @ S0d
    dsu = U @ dSe.transpose(-1, -2).contiguous()
    PD = dP * D
    dq = gam[..., None] * sdo + PD @ k
    dkk = PD.transpose(-1, -2).contiguous() @ q + end[..., None] * dsu
    A = dP * qk
    a0 = (q * sdo).sum(-1)
    db = (h * v).sum(-1)
    if delta:
        Z = (h @ UT).masked_fill(~strict, 0.0)
        sh = h @ S0d
        MD = -b[..., None] * Z * D
        dkk = dkk + MD @ k + MD.transpose(-1, -2).contiguous() @ k - (b * gam)[..., None] * sh
        A = A - b[..., None] * Z * kk
        a0 = a0 - b * (k * sh).sum(-1)
        db = db - gam * (k * sh).sum(-1) - (M * Z).sum(-1)
    # W[i, j] = A[i, j] D[i, j], bordered by the entering state (column 0) and
    # the leaving one (last row); alpha_t's gradient sums the block i >= t > j
    W = torch.cat([torch.cat([(gam * a0)[..., None], A * D], -1),
                   torch.cat([(gam[..., -1] * (S0t * dSe).sum((-1, -2)))[..., None],
                              end * (k * dsu).sum(-1)], -1)[..., None, :]], -2)
    cw = torch.cumsum(W, -1)[..., :-1]                  # columns below t = 1..C
    keep = torch.arange(C + 1, device="cuda")[:, None] >= i[None, :]
    da = cw.masked_fill(~keep, 0.0).sum(-2) / a
    dq, dkk = _tokens(dq, T), _tokens(dkk, T)
    if G > 1:
        dq, dkk = (x.reshape(B, T, Hk, G, dk).sum(3) for x in (dq, dkk))
    da, db = _tokens(da, T), _tokens(db, T)
    if s["lengths"] is not None:
        da = da.masked_fill(pad[..., None], 0.0)
    out.update(dq=dq.to(dt), dk=dkk.to(dt), dv=_tokens(bh, T).to(dt), dalpha=da.contiguous(),
               dbeta=db.contiguous(), dS0=dSt.transpose(-1, -2).contiguous())
    return out


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _norm_exact(s)
    return _scan_exact(s)


def _norm_exact(s):
    case, dt = s["case"], s["x"].dtype
    x = s["x"].double()
    out = {"h": None, "scales": None, "y": None}
    if s["res"] is not None:
        # the stream is kept in the inputs' type, and the norm is of what is kept
        h = x + s["res"].double()
        out["h"], x = h, h.to(dt).double()
    w = s["w"].double()
    r = (x.square().mean(-1) + s["eps"]).rsqrt()
    if case["out"] == "same":
        out["y"] = x * w * r[:, None]
    else:
        top = 127.0 if case["out"] == "int8" else 448.0
        out["scales"] = (x * w).abs().amax(-1) * r / top
    if case["op"] == "norm_train":
        g = s["dy"].double() * w
        t = (g * x).mean(-1) * r.pow(3)
        dx = g * r[:, None] - x * t[:, None]
        out["dx"] = dx if s["dres"] is None else dx + s["dres"].double()
        out["dw"] = torch.einsum("rn,rn,r->n", s["dy"].double(), x, r)
    return out


def _scan_exact(s):
    """Token by token; the gradient walks back over states that are rebuilt
    from those kept at every 64th token."""
    case = s["case"]
    B, T, H, Hk, dk, dv = (case[x] for x in ("B", "T", "H", "Hk", "dk", "dv"))
    G, delta = H // Hk, case["delta"]
    if B * H * dk * dv * T > 3e10:
        return None
    live = torch.ones(B, T, dtype=torch.bool, device="cuda")
    if s["lengths"] is not None:
        live = torch.arange(T, device="cuda")[None] < s["lengths"][:, None]
    x = {n: torch.where(live.view(B, T, *([1] * (s[n].dim() - 2))), s[n].double(),
                        1.0 if n == "alpha" else 0.0)
         for n in ("q", "k", "v", "alpha", "beta", "do") if n in s}

    def at(n, t):
        y = x[n][:, t]
        if n in "qk" and G > 1:
            y = y.repeat_interleave(G, 1)
        return y

    def step(S, t):
        """S_t, the decayed state and what the token writes per unit of beta."""
        Sd = S * at("alpha", t)[..., None, None]
        k = at("k", t)
        w = at("v", t)
        if delta:
            w = w - (Sd * k[..., None, :]).sum(-1)
        return Sd + (at("beta", t)[..., None] * w)[..., None] * k[..., None, :], Sd, w

    S = torch.zeros(B, H, dv, dk, dtype=torch.float64, device="cuda") if s["S0"] is None \
        else s["S0"].double()
    kept, o = [], torch.empty(B, T, H, dv, dtype=torch.float64, device="cuda")
    for t in range(T):
        if t % 64 == 0:
            kept.append(S)
        S = step(S, t)[0]
        o[:, t] = (S * at("q", t)[..., None, :]).sum(-1)
    out = {"o": o, "S": S}
    if case["op"] != "train":
        return out
    like = {n: torch.zeros(B, T, H, *z, dtype=torch.float64, device="cuda")
            for n, z in (("q", (dk,)), ("k", (dk,)), ("v", (dv,)), ("alpha", ()), ("beta", ()))}
    g = torch.zeros_like(S) if s["dS"] is None else s["dS"].double()
    for c in reversed(range(len(kept))):
        S, states = kept[c], []
        for t in range(64 * c, min(T, 64 * c + 64)):
            states.append(S)
            S = step(S, t)[0]
        for t in reversed(range(64 * c, min(T, 64 * c + 64))):
            S, Sd, w = step(states[t - 64 * c], t)
            q, k, do, b = at("q", t), at("k", t), at("do", t), at("beta", t)
            like["q"][:, t] = (S * do[..., None]).sum(-2)
            g = g + do[..., None] * q[..., None, :]
            gk = (g * k[..., None, :]).sum(-1)          # gradient of beta w
            like["beta"][:, t] = (gk * w).sum(-1)
            like["v"][:, t] = b[..., None] * gk
            like["k"][:, t] = b[..., None] * (g * w[..., None]).sum(-2)
            if delta:
                dw = b[..., None] * gk
                like["k"][:, t] -= (Sd * dw[..., None]).sum(-2)
                g = g - dw[..., None] * k[..., None, :]
            like["alpha"][:, t] = (g * states[t - 64 * c]).sum((-1, -2))
            g = g * at("alpha", t)[..., None, None]
    for n in like:
        like[n] = like[n] * live.view(B, T, *([1] * (like[n].dim() - 2)))
    for n in "qk":
        like[n] = like[n].reshape(B, T, Hk, G, dk).sum(3)
    out.update(dq=like["q"], dk=like["k"], dv=like["v"], dalpha=like["alpha"],
               dbeta=like["beta"], dS0=g)
    return out


# ------------------------------------------------------------------ work

def work(case):
    size = 2 if case["dtype"] == _BF16 else 4
    if case["op"].startswith("norm"):
        rows, n = case["rows"], case["n"]
        res = 2 if case["residual"] else 0               # the residual read, the sum written
        y = size if case["out"] == "same" else 1
        b = rows * n * (size * (1 + res) + y) + n * size
        b += 0 if case["out"] == "same" else 4 * rows
        if case["op"] == "norm_train":                   # h, dy, dres read, dx written
            b += rows * n * size * (3 + bool(case["residual"])) + 4 * n
        return {"bytes": b, "flops": rows * n * (5 if case["op"] == "norm" else 15)}
    B, T, H, Hk, dk, dv = (case[x] for x in ("B", "T", "H", "Hk", "dk", "dv"))
    qk, v, gate = 2 * B * T * Hk * dk * size, B * T * H * dv * size, 2 * B * T * H * 4
    state = 4 * B * H * dk * dv * (2 if case["state"] else 1)
    b, fl = qk + 2 * v + gate + state, 2 * B * T * H * dk * dv * (2 + case["delta"])
    if case["op"] == "train":                            # inputs and do again, five gradients
        b += 2 * qk + 3 * v + 2 * gate + state + 4 * B * H * dk * dv * (1 if case["state"] else 0)
        # the states again, and two products a state or its gradient enters per forward one
        fl += 2 * B * T * H * dk * dv * (2 + case["delta"]) * 2
    return {"bytes": b, "flops": fl}
