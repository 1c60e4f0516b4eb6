"""Cases of the fused feed-forward operators: the matrix product with scales, bias, activation and
residual in its epilogue, its backward pass, the root-mean-square norm with the residual's addition
(16-bit result, or 8 bits with row or block scales) and its backward pass.

`run` computes them in plain torch operations, in 32 bits; with `own` set it calls
tile_level_gemm_amd.  `exact` gives the same outputs in 64 bits.
"""

import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32,
         "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
QMAX = {"e4m3": 448.0, "e5m2": 57344.0}
EPS = 1e-5
AMAX_FLOOR = 2.0 ** -100   # largest magnitude below which a row or block is scaled as if it had this one


# ------------------------------------------------------------------------------ cases ----

def _product(name, M, N, K, dtype, act, ta=0, tb=1, bias=True, residual=False, keep_z=False, pad=0):
    """pad: elements between the rows of A and B beyond their length (a slice of a wider tensor)."""
    c = {"op": "product", "M": M, "N": N, "K": K, "dtype": dtype, "act": act, "ta": ta, "tb": tb,
         "bias": bias, "residual": residual, "keep_z": keep_z, "pad": pad}
    return dict(c, name=name) if name else c


def _product_bwd(name, M, N, K, dtype, act, ta=0, tb=1):
    c = {"op": "product_bwd", "M": M, "N": N, "K": K, "dtype": dtype, "act": act, "ta": ta, "tb": tb}
    return dict(c, name=name) if name else c


def _norm(name, rows, cols, dtype, out, residual=True, pad=0):
    c = {"op": "norm", "rows": rows, "cols": cols, "dtype": dtype, "out": out, "residual": residual,
         "pad": pad}
    return dict(c, name=name) if name else c


def _norm_bwd(name, rows, cols, dtype, stream):
    c = {"op": "norm_bwd", "rows": rows, "cols": cols, "dtype": dtype, "stream": stream}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token through a projection: the weights are read once, latency counts
        _product("product 1 token bf16", 1, 4096, 4096, "bf16", "silu"),
        # a small batch of tokens against 8-bit weights with row and column scales, onto the residual stream
        _product("product 16 tokens e4m3", 16, 8192, 4096, "e4m3", "none", bias=False, residual=True),
        # a short prompt, odd sizes, operands that are slices of wider tensors
        _product("product odd f16", 333, 1003, 2057, "f16", "gelu_tanh", residual=True, pad=5),
        # a prompt of a few hundred tokens: few output tiles, a long sum
        _product("product prompt bf16", 256, 4096, 8192, "bf16", "gelu", residual=True),
        # training forward at the benchmark's size, pre-activation kept for the backward pass
        _product("product training bf16", 8192, 8192, 8192, "bf16", "gelu_tanh", keep_z=True),
        # a long prompt with 8-bit operands
        _product("product long e4m3", 8192, 8192, 4096, "e4m3", "silu", bias=True),
        # gradients of a feed-forward product over a training batch
        _product_bwd("product gradients bf16", 4096, 8192, 2048, "bf16", "gelu_tanh"),
        # gradients of a small ragged batch, weights stored [K][N]
        _product_bwd("product gradients ragged f16", 200, 520, 264, "f16", "silu", tb=0),
        # one token's norm, quantised for the product that follows
        _norm("norm 1 token e4m3", 1, 4096, "bf16", "e4m3_row"),
        # a long batch, quantised in blocks of 32 for the block-scaled product
        _norm("norm long e4m3 blocks", 16384, 8192, "bf16", "e4m3_block"),
        # odd row length, 16-bit result
        _norm("norm odd f16", 1003, 2057, "f16", "same"),
        # training backward over a batch, with the gradient that arrives by the residual stream
        _norm_bwd("norm gradients bf16", 8192, 8192, "bf16", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """Spread over the logarithm; half of them whole multiples of 16, the others as they fall."""
    n = _log(rng, lo, hi)
    return max(lo, n // 16 * 16) if n >= 16 and rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["product", "product", "product_bwd", "norm", "norm_bwd"])
    acts = ["none", "relu", "gelu", "gelu_tanh", "silu"]
    if op == "product":
        dtype = rng.choice(["bf16", "f16", "e4m3", "e5m2"])
        eight = dtype in QMAX
        return _product(None, _size(rng, 1, 8192), _size(rng, 16, 8192), _size(rng, 16, 8192), dtype,
                        rng.choice(acts), 0 if eight else rng.randrange(2),
                        1 if eight else rng.randrange(2), rng.random() < 0.7, rng.random() < 0.5,
                        rng.random() < 0.3, rng.choice([0, 0, 5, 16]))
    if op == "product_bwd":
        return _product_bwd(None, _size(rng, 16, 4096), _size(rng, 16, 4096), _size(rng, 16, 4096),
                            rng.choice(["bf16", "f16"]), rng.choice(acts), rng.randrange(2),
                            rng.randrange(2))
    if op == "norm":
        out = rng.choice(["same", "same", "e4m3_row", "e4m3_block"])
        cols = _size(rng, 64, 16384)
        return _norm(None, _size(rng, 1, 8192), cols // 32 * 32 if out.endswith("block") else cols,
                     rng.choice(["bf16", "f16", "f32"]), out, rng.random() < 0.7, rng.choice([0, 0, 3, 32]))
    return _norm_bwd(None, _size(rng, 1, 8192), _size(rng, 64, 8192), rng.choice(["bf16", "f16", "f32"]),
                     rng.random() < 0.5)


def work(case):
    if case["op"] in ("product", "product_bwd"):
        M, N, K = case["M"], case["N"], case["K"]
        e = 1 if case["dtype"] in QMAX else 2
        if case["op"] == "product":
            outs = 1 + case["residual"] + case["keep_z"]
            vectors = 2 * N * case["bias"] + (4 * (M + N) if e == 1 else 0)
            return {"bytes": e * K * (M + N) + 2 * M * N * outs + vectors, "flops": 2 * M * N * K}
        return {"bytes": 2 * (2 * K * (M + N) + 3 * M * N) + 4 * N, "flops": 4 * M * N * K}
    n, cols, rows = case["rows"] * case["cols"], case["cols"], case["rows"]
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        ins = e * n * (1 + case["residual"]) + e * cols
        h = e * n * case["residual"]
        scales = n // 32 if case["out"].endswith("block") else 4 * rows if case["out"].endswith("row") else 0
        y = e * n if case["out"] == "same" else n
        return {"bytes": ins + h + y + scales + 4 * rows, "flops": 6 * n}
    return {"bytes": e * n * (3 + case["stream"]) + (4 + e) * cols + 4 * rows, "flops": 10 * n}


# ----------------------------------------------------------------------------- inputs ----

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _padded(t, pad):
    """The same values as a slice of a tensor whose rows are `pad` longer."""
    if not pad:
        return t.contiguous()
    wide = torch.zeros((t.shape[0], t.shape[1] + pad), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _quantised(x, dtype):
    """Rows in 8 bits with one scale each, as a calibrated checkpoint or a norm leaves them."""
    s = x.abs().amax(dim=1).clamp(min=1e-20) / QMAX[dtype]
    return (x / s[:, None]).to(TYPES[dtype]), s


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] in ("product", "product_bwd"):
        M, N, K, dt = case["M"], case["N"], case["K"], TYPES[case["dtype"]]
        a = _randn(g, *((K, M) if case["ta"] else (M, K)))
        b = _randn(g, *((N, K) if case["tb"] else (K, N))) / math.sqrt(K)
        s = {"case": case}
        if case["op"] == "product":
            out = torch.bfloat16 if case["dtype"] in QMAX else dt
            if case["dtype"] in QMAX:
                a, s["row_scale"] = _quantised(a, case["dtype"])
                b, s["col_scale"] = _quantised(b, case["dtype"])
            else:
                a, b = a.to(dt), b.to(dt)
                s["row_scale"] = s["col_scale"] = None
            s["A"], s["B"] = _padded(a, case["pad"]), _padded(b, case["pad"])
            s["bias"] = (0.5 * _randn(g, N)).to(out) if case["bias"] else None
            s["residual"] = _randn(g, M, N).to(out) if case["residual"] else None
            s["out"] = out
            return s
        s["A"], s["B"] = a.to(dt), b.to(dt)
        s["Z"] = _randn(g, M, N).to(dt)
        s["dY"] = (0.1 * _randn(g, M, N)).to(dt)
        return s
    rows, cols, dt = case["rows"], case["cols"], TYPES[case["dtype"]]
    # a few channels far larger than the others, as residual streams have
    channel = 1.0 + 15.0 * (torch.rand(cols, generator=g, device="cuda") < 0.01)
    s = {"case": case, "weight": (1.0 + 0.1 * _randn(g, cols)).to(dt)}
    if case["op"] == "norm":
        s["X"] = _padded((_randn(g, rows, cols) * channel).to(dt), case["pad"])
        s["residual"] = _padded((0.5 * _randn(g, rows, cols)).to(dt), case["pad"]) if case["residual"] else None
        return s
    h = (_randn(g, rows, cols) * channel).to(dt)
    s["H"] = h
    s["rstd"] = torch.rsqrt(h.float().square().mean(dim=1) + EPS)
    s["dY"] = (0.1 * _randn(g, rows, cols)).to(dt)
    s["dH"] = (0.1 * _randn(g, rows, cols)).to(dt) if case["stream"] else None
    return s


# ------------------------------------------------------------------------- plain form ----

def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.special.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "product":
        a = s["A"].float().t() if case["ta"] else s["A"].float()
        b = s["B"].float().t() if case["tb"] else s["B"].float()
        z = a @ b
        if s["row_scale"] is not None:
            z = z * s["row_scale"][:, None] * s["col_scale"]
        if s["bias"] is not None:
            z = z + s["bias"].float()
        d = _act(z, case["act"])
        if s["residual"] is not None:
            d = d + s["residual"].float()
        out = {"D": d.to(s["out"])}
        if case["keep_z"]:
            out["Z"] = z.to(s["out"])
        return out
    if op == "product_bwd":
        dt = s["A"].dtype
        a = s["A"].float().t() if case["ta"] else s["A"].float()
        b = s["B"].float().t() if case["tb"] else s["B"].float()
        dz = s["dY"].float() * _act_grad(s["Z"].float(), case["act"])
        da = b @ dz.t() if case["ta"] else dz @ b.t()
        db = dz.t() @ a if case["tb"] else a.t() @ dz
        return {"dZ": dz.to(dt), "dA": da.to(dt), "dB": db.to(dt), "dbias": dz.sum(dim=0)}
    w = s["weight"].float()
    if op == "norm":
        dt = s["X"].dtype
        h = s["X"]
        if s["residual"] is not None:
            h = (h.float() + s["residual"].float()).to(dt)
        hf = h.float()
        rstd = torch.rsqrt(hf.square().mean(dim=1) + EPS)
        y = hf * rstd[:, None] * w
        out = {"rstd": rstd}
        if s["residual"] is not None:
            out["H"] = h
        if case["out"] == "same":
            out["Y"] = y.to(dt)
            return out
        kind, form = case["out"].split("_")
        if form == "row":
            scale = y.abs().amax(dim=1).clamp(min=AMAX_FLOOR) / QMAX[kind]
            out["Q"], out["scale"] = (y / scale[:, None]).to(TYPES[kind]), scale
            return out
        blocks = y.reshape(y.shape[0], -1, 32)
        m, e = torch.frexp(blocks.abs().amax(dim=2).clamp(min=AMAX_FLOOR) / QMAX[kind])
        e = e - (m == 0.5).to(e.dtype)       # 2^e is the smallest power of two not below
        q = torch.ldexp(blocks, -e[:, :, None])
        out["Q"] = q.reshape(y.shape).to(TYPES[kind])
        out["scale"] = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
        return out
    h, dy = s["H"].float(), s["dY"].float()
    xh = h * s["rstd"][:, None]
    g = dy * w
    dx = s["rstd"][:, None] * (g - xh * (g * xh).mean(dim=1, keepdim=True))
    if s["dH"] is not None:
        dx = dx + s["dH"].float()
    return {"dX": dx.to(s["H"].dtype), "dw": (dy * xh).sum(dim=0)}


def _own(s):
    import tile_level_gemm_amd as tg
    case, op = s["case"], s["case"]["op"]
    if op == "product":
        d = tg.gemm_ep(s["A"], s["B"], bias=s["bias"], act=case["act"], residual=s["residual"],
                       row_scale=s["row_scale"], col_scale=s["col_scale"], trans_a=case["ta"],
                       trans_b=case["tb"], out_dtype=s["out"], keep_z=case["keep_z"])
        return {"D": d[0], "Z": d[1]} if case["keep_z"] else {"D": d}
    if op == "product_bwd":
        dz, da, db, dbias = tg.gemm_ep_backward(s["dY"], s["A"], s["B"], Z=s["Z"], act=case["act"],
                                                trans_a=case["ta"], trans_b=case["tb"])
        return {"dZ": dz, "dA": da, "dB": db, "dbias": dbias}
    if op == "norm":
        kind, _, form = case["out"].partition("_")
        r = tg.rms_norm(s["X"], s["weight"], EPS, residual=s["residual"],
                        out_dtype=TYPES[kind] if form else None, scales=form or None)
        out = {"rstd": r.rstd, "Q" if form else "Y": r.y}
        if form:
            out["scale"] = r.scale
        if s["residual"] is not None:
            out["H"] = r.h
        return out
    dx, dw = tg.rms_norm_backward(s["dY"], s["H"], s["weight"], s["rstd"], dH=s["dH"])
    return {"dX": dx, "dw": dw}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------- definition ----

def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.to(torch.float32).double() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    op = case["op"]
    if op in ("product", "product_bwd"):
        A = d["A"].transpose(0, 1) if case["ta"] else d["A"]      # [M][K]
        B = d["B"].transpose(0, 1) if case["tb"] else d["B"]      # [K][N]
        normal = torch.distributions.Normal(torch.zeros((), dtype=torch.float64, device="cuda"),
                                            torch.ones((), dtype=torch.float64, device="cuda"),
                                            validate_args=False)

        def f(z):
            if case["act"] == "none":
                return z
            if case["act"] == "relu":
                return torch.where(z > 0, z, 0.0)
            if case["act"] == "gelu":
                return z * normal.cdf(z)
            if case["act"] == "gelu_tanh":
                return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
            return z * torch.sigmoid(z)

        if op == "product":
            Z = torch.matmul(A, B)
            if d["row_scale"] is not None:
                Z = torch.outer(d["row_scale"], d["col_scale"]) * Z
            if d["bias"] is not None:
                Z = Z + d["bias"][None]
            D = f(Z) if d["residual"] is None else f(Z) + d["residual"]
            return {"D": D, "Z": Z} if case["keep_z"] else {"D": D}
        with torch.enable_grad():            # the derivative of f by differentiation, in 64 bits
            z = d["Z"].clone().requires_grad_(True)
            dZ, = torch.autograd.grad(f(z), z, d["dY"])
        dA, dB = torch.matmul(dZ, B.T), torch.matmul(A.T, dZ)
        return {"dZ": dZ, "dA": dA.T.contiguous() if case["ta"] else dA,
                "dB": dB.T.contiguous() if case["tb"] else dB, "dbias": torch.sum(dZ, 0)}
    if op == "norm":
        H = d["X"]
        if d["residual"] is not None:        # the residual stream is held in the input's type
            H = (H + d["residual"]).to(TYPES[case["dtype"]]).double()
        rstd = (torch.mean(H * H, 1) + EPS) ** -0.5
        Y = torch.einsum("mn,m,n->mn", H, rstd, d["weight"])
        out = {"rstd": rstd}
        if d["residual"] is not None:
            out["H"] = H
        if case["out"] == "same":
            out["Y"] = Y
            return out
        kind, form = case["out"].split("_")
        if form == "row":
            scale = torch.clamp(torch.max(torch.abs(Y), 1).values, min=AMAX_FLOOR) / QMAX[kind]
            out["Q"], out["scale"] = Y / scale[:, None], scale
            return out
        top = torch.clamp(torch.max(torch.abs(Y).unflatten(1, (-1, 32)), 2).values, min=AMAX_FLOOR)
        scale = torch.exp2(torch.ceil(torch.log2(top / QMAX[kind])))
        # a power of two next to a border has no value that 32 bits must agree with
        out["Q"], out["scale"] = Y / scale.repeat_interleave(32, 1), None
        return out
    xh = d["H"] * d["rstd"][:, None]
    g = d["dY"] * d["weight"][None]
    dX = (g - xh * torch.mean(g * xh, 1)[:, None]) * d["rstd"][:, None]
    if d["dH"] is not None:
        dX = dX + d["dH"]
    return {"dX": dX, "dw": torch.einsum("mn,mn->n", d["dY"], xh)}
