"""Cases of the operators of a gated feed-forward layer: the gated product (two projections, the activation
and their product in one kernel) and its backward pass, the product of 8-bit integers with scales for each
token and channel, the layer norm with the residual's addition and its backward pass, and the quantisation
of rows to 8 bits.

`run` computes them in plain torch operations, in 32 bits; with `own` set it calls
tile_level_gemm_amd.  `exact` gives the same outputs in 64 bits.
"""

import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32,
         "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "i8": torch.int8}
QMAX = {"e4m3": 448.0, "e5m2": 57344.0, "i8": 127.0}
EPS = 1e-5
AMAX_FLOOR = 2.0 ** -100   # largest magnitude below which a row or block is scaled as if it had this one


# ------------------------------------------------------------------------------ cases ----

def _gated(name, M, N, K, dtype, act, tb=1, bias=False, keep_z=False, pad=0):
    """[M][K] tokens against [2N][K] weights ([K][2N] without tb), the gate's first.  pad: elements
    between the rows of A and B beyond their length (a slice of a wider tensor)."""
    c = {"op": "gated", "M": M, "N": N, "K": K, "dtype": dtype, "act": act, "tb": tb, "bias": bias,
         "keep_z": keep_z, "pad": pad}
    return dict(c, name=name) if name else c


def _gated_bwd(name, M, N, K, dtype, act, tb=1):
    c = {"op": "gated_bwd", "M": M, "N": N, "K": K, "dtype": dtype, "act": act, "tb": tb}
    return dict(c, name=name) if name else c


def _product(name, M, N, K, act, bias=True, residual=False, pad=0):
    c = {"op": "product", "M": M, "N": N, "K": K, "dtype": "i8", "act": act, "bias": bias, "residual": residual,
         "pad": pad}
    return dict(c, name=name) if name else c


def _norm(name, rows, cols, dtype, out, residual=True, bias=True, pad=0):
    c = {"op": "norm", "rows": rows, "cols": cols, "dtype": dtype, "out": out, "residual": residual,
         "bias": bias, "pad": pad}
    return dict(c, name=name) if name else c


def _norm_bwd(name, rows, cols, dtype, stream):
    c = {"op": "norm_bwd", "rows": rows, "cols": cols, "dtype": dtype, "stream": stream}
    return dict(c, name=name) if name else c


def _rows(name, rows, cols, dtype, out, pad=0):
    c = {"op": "rows", "rows": rows, "cols": cols, "dtype": dtype, "out": out, "pad": pad}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token through both projections: the weights are read once, latency counts
        _gated("gated 1 token bf16", 1, 8192, 4096, "bf16", "silu"),
        # training forward over a long batch, both projections kept for the backward pass
        _gated("gated training bf16", 8192, 8192, 4096, "bf16", "silu", keep_z=True),
        # gradients over a training batch
        _gated_bwd("gated gradients bf16", 4096, 4096, 2048, "bf16", "silu"),
        # gradients of a small ragged batch, weights stored [K][2N]
        _gated_bwd("gated gradients ragged f16", 200, 264, 520, "f16", "gelu_tanh", tb=0),
        # a small batch of tokens through an 8-bit down projection onto the residual stream
        _product("i8 product 16 tokens", 16, 8192, 4096, "none", bias=False, residual=True),
        # a long prompt in 8 bits
        _product("i8 product long", 8192, 8192, 4096, "silu"),
        # one token's norm, quantised for the product that follows
        _norm("layer norm 1 token e4m3", 1, 4096, "bf16", "e4m3_row"),
        # a long batch onto the residual stream
        _norm("layer norm long bf16", 16384, 8192, "bf16", "same"),
        # odd row length
        _norm_bwd("layer norm gradients odd f16", 1003, 2057, "f16", False),
        # training backward over a batch, with the gradient that arrives by the residual stream
        _norm_bwd("layer norm gradients bf16", 8192, 8192, "bf16", True),
        # an activation of odd width, to 8-bit integers for the product that follows
        _rows("quantise rows odd f16", 333, 2057, "f16", "i8_row"),
        # a long prompt's activation, or a weight matrix
        _rows("quantise rows long bf16", 16384, 8192, "bf16", "i8_row"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """Spread over the logarithm; half of them whole multiples of 16, the others as they fall."""
    n = _log(rng, lo, hi)
    return max(lo, n // 16 * 16) if n >= 16 and rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_bwd", "product", "norm", "norm_bwd", "rows"])
    acts = ["none", "relu", "gelu", "gelu_tanh", "silu"]
    pad = rng.choice([0, 0, 5, 16])
    if op == "gated":
        dtype = rng.choice(["bf16", "f16", "e4m3", "e5m2", "i8"])
        return _gated(None, _size(rng, 1, 8192), _size(rng, 16, 8192), _size(rng, 16, 4096), dtype,
                      rng.choice(acts), 1 if dtype in QMAX else rng.randrange(2), rng.random() < 0.5,
                      rng.random() < 0.3, pad)
    if op == "gated_bwd":
        return _gated_bwd(None, _size(rng, 16, 4096), _size(rng, 16, 4096), _size(rng, 16, 2048),
                          rng.choice(["bf16", "f16"]), rng.choice(acts), rng.randrange(2))
    if op == "product":
        return _product(None, _size(rng, 1, 8192), _size(rng, 16, 8192), _size(rng, 16, 8192), rng.choice(acts),
                        rng.random() < 0.7, rng.random() < 0.5, pad)
    rows, cols, dtype = _size(rng, 1, 8192), _size(rng, 64, 16384), rng.choice(["bf16", "f16", "f32"])
    if op == "norm":
        out = rng.choice(["same", "same", "e4m3_row", "e4m3_block"])
        return _norm(None, rows, cols // 32 * 32 if out.endswith("block") else cols, dtype, out,
                     rng.random() < 0.7, rng.random() < 0.7, rng.choice([0, 0, 3, 32]))
    if op == "norm_bwd":
        return _norm_bwd(None, rows, min(cols, 8192), dtype, rng.random() < 0.5)
    out = rng.choice(["i8_row", "i8_row", "e4m3_row", "e5m2_row", "e4m3_block"])
    return _rows(None, rows, cols // 32 * 32 if out.endswith("block") else cols, dtype, out, rng.choice([0, 0, 3, 32]))


def _scale_bytes(case):
    rows, n = case["rows"], case["rows"] * case["cols"]
    return n // 32 if case["out"].endswith("block") else 4 * rows if case["out"].endswith("row") else 0


def work(case):
    op = case["op"]
    if op in ("gated", "gated_bwd", "product"):
        M, N, K = case["M"], case["N"], case["K"]
        e = 1 if case["dtype"] in QMAX else 2
        if op == "gated":
            vectors = 4 * N * case["bias"] + (4 * (M + 2 * N) if e == 1 else 0)
            return {"bytes": e * K * (M + 2 * N) + 2 * M * N * (1 + 2 * case["keep_z"]) + vectors,
                    "flops": 4 * M * N * K}
        if op == "gated_bwd":
            return {"bytes": 2 * (2 * K * (M + 2 * N) + 5 * M * N) + 8 * N, "flops": 8 * M * N * K}
        return {"bytes": K * (M + N) + 2 * M * N * (1 + case["residual"]) + 2 * N * case["bias"] + 4 * (M + N),
                "flops": 2 * M * N * K}
    rows, cols = case["rows"], case["cols"]
    n, e = rows * cols, 4 if case["dtype"] == "f32" else 2
    if op == "norm":
        y = e * n if case["out"] == "same" else n
        return {"bytes": e * n * (1 + 2 * case["residual"]) + e * cols * (1 + case["bias"]) + y + _scale_bytes(case)
                + 8 * rows, "flops": 9 * n}
    if op == "norm_bwd":
        return {"bytes": e * n * (3 + case["stream"]) + (8 + e) * cols + 8 * rows, "flops": 13 * n}
    return {"bytes": (e + 1) * n + _scale_bytes(case), "flops": 3 * n}


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
    q = x / s[:, None]
    return (torch.clamp(torch.round(q), -127, 127) if dtype == "i8" else q).to(TYPES[dtype]), s


def prepare(case, seed):
    g, op, dt = _gen(seed), case["op"], TYPES[case["dtype"]]
    s = {"case": case}
    if op in ("gated", "gated_bwd", "product"):
        M, N, K = case["M"], case["N"], case["K"]
        width = N if op == "product" else 2 * N
        a = _randn(g, M, K)
        b = _randn(g, *((width, K) if case.get("tb", 1) else (K, width))) / math.sqrt(K)
        if op == "gated_bwd":
            s["A"], s["B"] = a.to(dt), b.to(dt)
            s["Z"] = _randn(g, M, width).to(dt)
            s["dY"] = (0.1 * _randn(g, M, N)).to(dt)
            return s
        out = torch.bfloat16 if case["dtype"] in QMAX else dt
        s["row_scale"] = s["col_scale"] = None
        if case["dtype"] in QMAX:
            a, s["row_scale"] = _quantised(a, case["dtype"])
            b, s["col_scale"] = _quantised(b, case["dtype"])
        s["A"], s["B"] = _padded(a.to(dt), case["pad"]), _padded(b.to(dt), case["pad"])
        s["bias"] = (0.5 * _randn(g, width)).to(out) if case["bias"] else None
        s["residual"] = _randn(g, M, N).to(out) if case.get("residual") else None
        s["out"] = out
        return s
    rows, cols = case["rows"], case["cols"]
    # a few channels far larger than the others, as residual streams have, about a mean of their own
    channel = 1.0 + 15.0 * (torch.rand(cols, generator=g, device="cuda") < 0.01)
    x = (_randn(g, rows, cols) * channel + 0.25).to(dt)
    if op == "rows":
        s["X"] = _padded(x, case["pad"])
        return s
    s["weight"] = (1.0 + 0.1 * _randn(g, cols)).to(dt)
    if op == "norm":
        s["X"] = _padded(x, case["pad"])
        s["bias"] = (0.1 * _randn(g, cols)).to(dt) if case["bias"] else None
        s["residual"] = _padded((0.5 * _randn(g, rows, cols)).to(dt), case["pad"]) if case["residual"] else None
        return s
    s["H"] = x
    h = x.float()
    s["mean"] = h.mean(dim=1)
    s["rstd"] = torch.rsqrt((h - s["mean"][:, None]).square().mean(dim=1) + EPS)
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


def _eight_bits(y, out):
    """Rows or blocks of 32 in 8 bits, and their scales."""
    kind, form = out.split("_")
    if form == "row":
        scale = y.abs().amax(dim=1).clamp(min=AMAX_FLOOR) / QMAX[kind]
        q = y / scale[:, None]
        return (torch.clamp(torch.round(q), -127, 127) if kind == "i8" else q).to(TYPES[kind]), scale
    blocks = y.reshape(y.shape[0], -1, 32)
    m, e = torch.frexp(blocks.abs().amax(dim=2).clamp(min=AMAX_FLOOR) / QMAX[kind])
    e = e - (m == 0.5).to(e.dtype)       # 2^e is the smallest power of two not below
    q = torch.ldexp(blocks, -e[:, :, None])
    return q.reshape(y.shape).to(TYPES[kind]), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op in ("gated", "product"):
        b = s["B"].float().t() if case.get("tb", 1) else s["B"].float()
        z = s["A"].float() @ b
        if s["row_scale"] is not None:
            z = z * s["row_scale"][:, None] * s["col_scale"]
        if s["bias"] is not None:
            z = z + s["bias"].float()
        if op == "gated":
            d = _act(z[:, :case["N"]], case["act"]) * z[:, case["N"]:]
            out = {"D": d.to(s["out"])}
            if case["keep_z"]:
                out["Z"] = z.to(s["out"])
            return out
        d = _act(z, case["act"])
        if s["residual"] is not None:
            d = d + s["residual"].float()
        return {"D": d.to(s["out"])}
    if op == "gated_bwd":
        dt, n = s["A"].dtype, case["N"]
        b = s["B"].float().t() if case["tb"] else s["B"].float()
        dy, gate, up = s["dY"].float(), s["Z"][:, :n].float(), s["Z"][:, n:].float()
        dz = torch.cat([dy * up * _act_grad(gate, case["act"]), dy * _act(gate, case["act"])], dim=1)
        a = s["A"].float()
        db = dz.t() @ a if case["tb"] else a.t() @ dz
        return {"dZ": dz.to(dt), "dA": (dz @ b.t()).to(dt), "dB": db.to(dt), "dbias": dz.sum(dim=0)}
    if op == "rows":
        q, scale = _eight_bits(s["X"].float(), case["out"])
        return {"Q": q, "scale": scale}
    w = s["weight"].float()
    if op == "norm":
        dt = s["X"].dtype
        h = s["X"]
        if s["residual"] is not None:
            h = (h.float() + s["residual"].float()).to(dt)
        hf = h.float()
        mean = hf.mean(dim=1)
        hc = hf - mean[:, None]
        rstd = torch.rsqrt(hc.square().mean(dim=1) + EPS)
        y = hc * rstd[:, None] * w
        if s["bias"] is not None:
            y = y + s["bias"].float()
        out = {"mean": mean, "rstd": rstd}
        if s["residual"] is not None:
            out["H"] = h
        if case["out"] == "same":
            out["Y"] = y.to(dt)
        else:
            out["Q"], out["scale"] = _eight_bits(y, case["out"])
        return out
    dy = s["dY"].float()
    xh = (s["H"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * w
    dx = s["rstd"][:, None] * (g - g.mean(dim=1, keepdim=True) - xh * (g * xh).mean(dim=1, keepdim=True))
    if s["dH"] is not None:
        dx = dx + s["dH"].float()
    return {"dX": dx.to(s["H"].dtype), "dw": (dy * xh).sum(dim=0), "db": dy.sum(dim=0)}


def _own(s):
    import tile_level_gemm_amd as tg
    case, op = s["case"], s["case"]["op"]
    if op == "gated":
        d = tg.gemm_gated(s["A"], s["B"], bias=s["bias"], act=case["act"], row_scale=s["row_scale"],
                          col_scale=s["col_scale"], trans_b=case["tb"], out_dtype=s["out"], keep_z=case["keep_z"])
        return {"D": d[0], "Z": d[1]} if case["keep_z"] else {"D": d}
    if op == "gated_bwd":
        dz, da, db, dbias = tg.gemm_gated_backward(s["dY"], s["A"], s["B"], s["Z"], act=case["act"],
                                                   trans_b=case["tb"])
        return {"dZ": dz, "dA": da, "dB": db, "dbias": dbias}
    if op == "product":
        return {"D": tg.gemm_ep(s["A"], s["B"], bias=s["bias"], act=case["act"], residual=s["residual"],
                                row_scale=s["row_scale"], col_scale=s["col_scale"], out_dtype=s["out"])}
    if op == "rows":
        kind, form = case["out"].split("_")
        q, scale = tg.quantize_rows(s["X"], out_dtype=TYPES[kind], scales=form)
        return {"Q": q, "scale": scale}
    if op == "norm":
        kind, _, form = case["out"].partition("_")
        r = tg.layer_norm(s["X"], s["weight"], s["bias"], EPS, residual=s["residual"],
                          out_dtype=TYPES[kind] if form else None, scales=form or None)
        out = {"mean": r.mean, "rstd": r.rstd, "Q" if form else "Y": r.y}
        if form:
            out["scale"] = r.scale
        if s["residual"] is not None:
            out["H"] = r.h
        return out
    dx, dw, db = tg.layer_norm_backward(s["dY"], s["H"], s["weight"], s["mean"], s["rstd"], dH=s["dH"])
    return {"dX": dx, "dw": dw, "db": db}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------- definition ----

def _exact_rows(Y, out):
    """The quotient that the codes round, and the scale it was taken by."""
    kind, form = out.split("_")
    if form == "row":
        scale = torch.clamp(torch.max(torch.abs(Y), 1).values, min=AMAX_FLOOR) / QMAX[kind]
        q = Y / scale[:, None]
        return torch.round(q).to(torch.int8) if kind == "i8" else q, scale
    top = torch.clamp(torch.max(torch.abs(Y).unflatten(1, (-1, 32)), 2).values, min=AMAX_FLOOR)
    scale = torch.exp2(torch.ceil(torch.log2(top / QMAX[kind])))
    # a power of two next to a border has no value that 32 bits must agree with
    return Y / scale.repeat_interleave(32, 1), None


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.to(torch.float32).double() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    op = case["op"]
    if op in ("gated", "gated_bwd", "product"):
        A = d["A"]
        B = d["B"].transpose(0, 1) if case.get("tb", 1) else d["B"]      # [K][columns]
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

        if op == "gated_bwd":
            with torch.enable_grad():        # the derivative by differentiation, in 64 bits
                z = d["Z"].clone().requires_grad_(True)
                gate, up = torch.chunk(z, 2, dim=1)
                dZ, = torch.autograd.grad(f(gate) * up, z, d["dY"])
            dA, dB = torch.matmul(dZ, B.T), torch.matmul(A.T, dZ)
            return {"dZ": dZ, "dA": dA, "dB": dB.T.contiguous() if case["tb"] else dB, "dbias": torch.sum(dZ, 0)}
        Z = torch.matmul(A, B)
        if d["row_scale"] is not None:
            Z = torch.outer(d["row_scale"], d["col_scale"]) * Z
        if d["bias"] is not None:
            Z = Z + d["bias"][None]
        if op == "gated":
            gate, up = torch.chunk(Z, 2, dim=1)
            D = f(gate) * up
            return {"D": D, "Z": Z} if case["keep_z"] else {"D": D}
        return {"D": f(Z) if d["residual"] is None else f(Z) + d["residual"]}
    if op == "rows":
        q, scale = _exact_rows(d["X"], case["out"])
        return {"Q": q, "scale": scale}
    if op == "norm":
        H = d["X"]
        if d["residual"] is not None:        # the residual stream is held in the input's type
            H = (H + d["residual"]).to(TYPES[case["dtype"]]).double()
        var, mean = torch.var_mean(H, 1, unbiased=False)
        rstd = (var + EPS) ** -0.5
        Y = torch.einsum("mn,m,n->mn", H - mean[:, None], rstd, d["weight"])
        if d["bias"] is not None:
            Y = Y + d["bias"][None]
        out = {"mean": mean, "rstd": rstd}
        if d["residual"] is not None:
            out["H"] = H
        if case["out"] == "same":
            out["Y"] = Y
        else:
            out["Q"], out["scale"] = _exact_rows(Y, case["out"])
        return out
    xh = (d["H"] - d["mean"][:, None]) * d["rstd"][:, None]
    g = d["dY"] * d["weight"][None]
    dX = (g - torch.mean(g, 1)[:, None] - xh * torch.mean(g * xh, 1)[:, None]) * d["rstd"][:, None]
    if d["dH"] is not None:
        dX = dX + d["dH"]
    return {"dX": dX, "dw": torch.einsum("mn,mn->n", d["dY"], xh), "db": torch.sum(d["dY"], 0)}
