"""Layer norm, its backward pass, quantised rows and 8-bit integer rows of the norms on the GPU, against
float64 references.  Tolerances are oracle/layer.py's bounds."""

import numpy as np
import pytest
import torch

import tile_level_gemm_amd as tg
from oracle import layer as ol

from .gpu_util import say
from .test_gpu_layer import COLS, T, check, dev, host, rand, wide

pytestmark = pytest.mark.gpu

Q8 = {**T, "i8": torch.int8}


def check_codes(q, Y, err, each, fmt):
    """Codes of Y known to within err, by the scales that were stored: rounded once."""
    got = q.cpu().numpy().astype(np.float64) if fmt == "i8" else host(q)
    h, t = (0.0, 0.5) if fmt == "i8" else (ol.HALF_STEP[fmt], ol.TINY[fmt])
    bound = (err * (1 + h) + (h + 2 * ol.U32) * np.abs(Y)) / each + t
    off = np.abs(got - Y / each) > bound
    assert not off.any(), f"{np.count_nonzero(off)} codes outside"


def check_norm(r, X, R, W, B, eps, dtype, fmt, scales):
    if R is not None:
        assert torch.equal(r.h, (X.float() + R.float()).to(X.dtype))
    Y, mean, rstd, err, merr, rel = ol.layer_norm(host(r.h), host(W), None if B is None else host(B), eps)
    check(r.mean, mean, merr + 1e-40, "mean")
    check(r.rstd, rstd, rel * rstd, "rstd")
    if scales is None:
        h = ol.HALF_STEP[dtype]
        check(r.y, Y, err * (1 + h) + h * np.abs(Y) + ol.TINY[dtype], "Y")
        return
    if scales == "row":
        s = ol.row_scale(Y, fmt)
        check(r.scale, s, err.max(axis=1) / ol.QMAX[fmt] + 4 * ol.U32 * s, "scale")
        each = host(r.scale)[:, None] * np.ones_like(Y)
    else:
        got = r.scale.view(torch.uint8).cpu().numpy().astype(np.int64) - 127
        lo, hi = (ol.block_scale(np.maximum(np.abs(Y) + k * err, 0.0), fmt) for k in (-1, 1))
        assert ((got >= lo) & (got <= hi)).all(), "block exponents"
        each = np.repeat(2.0 ** got, 32, axis=1)
    check_codes(r.y, Y, err, each, fmt)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_lengths(cols, dtype):
    say(f"layer norm cols={cols} {dtype}")
    rows = 6
    X, R = rand(cols, (rows, cols), dtype, 3.0), rand(cols + 1, (rows, cols), dtype)
    X += 1.5
    W, B = rand(cols + 2, (cols,), dtype), rand(cols + 3, (cols,), dtype)
    check_norm(tg.layer_norm(X, W), X, None, W, None, 1e-5, dtype, None, None)
    check_norm(tg.layer_norm(X, W, B, residual=R), X, R, W, B, 1e-5, dtype, None, None)
    W, B = rand(cols + 4, (cols,), "f32"), rand(cols + 5, (cols,), "f32")
    for fmt in ("e4m3", "e5m2", "i8"):
        check_norm(tg.layer_norm(X, W, B, 1e-6, residual=R, out_dtype=Q8[fmt], scales="row"), X, R, W, B, 1e-6, dtype, fmt, "row")
        if cols % 32 == 0 and fmt != "i8":
            check_norm(tg.layer_norm(X, W, None, 1e-6, out_dtype=Q8[fmt], scales="block"), X, None, W, None, 1e-6, dtype, fmt, "block")


@pytest.mark.parametrize("rows", [1, 3, 5, 513])
@pytest.mark.parametrize("cols", [96, 1024, 2336])
def test_rows_slices_and_in_place(rows, cols):
    say(f"layer norm rows={rows} cols={cols}")
    X, R, W, B = (rand(i, s, "bf16") for i, s in enumerate([(rows, cols), (rows, cols), (cols,), (cols,)]))
    base = tg.layer_norm(X, W, B, residual=R, out_dtype=torch.int8, scales="row")
    check_norm(base, X, R, W, B, 1e-5, "bf16", "i8", "row")
    for before, after in ((0, 8), (3, 2)):
        x, r = wide(X, before, after, float("nan"))[0], wide(R, before, after, float("nan"))[0]
        got = tg.layer_norm(x, W, B, residual=r, out_dtype=torch.int8, scales="row")
        for k in ("h", "mean", "rstd", "scale", "y"):
            assert torch.equal(getattr(got, k), getattr(base, k)), k
        for inplace in (0, 1):
            x, xw = wide(X, before, after, 9.0)
            r, rw = wide(R, before, after, 9.0)
            h = (x, r)[inplace]
            got = tg.layer_norm(x, W, B, residual=r, out_dtype=torch.int8, scales="row", h_out=h)
            assert torch.equal(h, base.h) and torch.equal(got.y, base.y) and torch.equal(got.mean, base.mean)
            w = (xw, rw)[inplace]
            assert bool((torch.cat([w[:, :before], w[:, before + cols:]], dim=1) == 9.0).all())


@pytest.mark.parametrize("cols", [64, 520, 2057, 20000])
@pytest.mark.parametrize("shift", [100.0, 1e4, -3e5])
def test_rows_far_from_zero_keep_their_variance(cols, shift):
    """fp32 rows whose deviations are a small part of them: the squares are taken about the mean."""
    say(f"layer norm shift={shift} cols={cols}")
    X, W = rand(cols, (4, cols), "f32") + shift, rand(1, (cols,), "f32")
    check_norm(tg.layer_norm(X, W), X, None, W, None, 1e-5, "f32", None, None)


@pytest.mark.parametrize("cols", [64, 1000, 2048, 20000])
def test_rows_of_one_value_and_of_nan(cols):
    say(f"layer norm constant and nan cols={cols}")
    X, W, B = rand(1, (5, cols), "bf16"), rand(2, (cols,), "bf16"), rand(3, (cols,), "bf16")
    X[1] = 4.0
    X[2, 3] = float("nan")
    X[3, cols - 1] = float("inf")
    X[4] *= 1e-30
    r = tg.layer_norm(X, W, B, 1e-5)
    y = host(r.y)
    assert np.array_equal(y[1], host(B)) and float(r.mean[1]) == 4.0
    assert np.isnan(y[2]).all() and np.isfinite(y[[0, 1, 4]]).all() and np.isnan(y[3]).all()
    for fmt in ("e4m3", "i8"):
        r = tg.layer_norm(X, W, B, 1e-5, out_dtype=Q8[fmt], scales="row")
        s = host(r.scale)
        assert np.isfinite(s[[0, 1, 4]]).all() and (s[[0, 1, 4]] > 0).all() and np.isnan(s[[2, 3]]).all()
        q = r.y.float().cpu().numpy()
        assert (q[[2, 3]] == 0).all() if fmt == "i8" else np.isnan(q[[2, 3]]).all()


@pytest.mark.parametrize("cols", [64, 1000, 2048, 20000])
@pytest.mark.parametrize("call", ["rms_norm", "layer_norm", "quantize_rows"])
def test_integer_rows_that_are_not_finite(cols, call):
    """A NaN or an infinity gives its row a NaN scale and codes of 0, the others are as they were."""
    say(f"{call} i8 nan cols={cols}")
    X, W = rand(1, (4, cols), "f32"), rand(2, (cols,), "f32")
    run = {"rms_norm": lambda x: (lambda r: (r.y, r.scale))(tg.rms_norm(x, W, out_dtype=torch.int8, scales="row")),
           "layer_norm": lambda x: (lambda r: (r.y, r.scale))(tg.layer_norm(x, W, out_dtype=torch.int8, scales="row")),
           "quantize_rows": tg.quantize_rows}[call]
    q0, s0 = run(X)
    X[1, cols - 1], X[2, 0] = float("nan"), float("-inf")
    q, s = run(X)
    assert not q[[1, 2]].any() and torch.isnan(s[[1, 2]]).all()
    assert torch.equal(q[[0, 3]], q0[[0, 3]]) and torch.equal(s[[0, 3]], s0[[0, 3]])


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_rms_norm_in_integer_rows(cols, dtype):
    say(f"rms norm i8 cols={cols} {dtype}")
    X, W = rand(cols, (5, cols), dtype, 3.0), rand(cols + 1, (cols,), dtype)
    r = tg.rms_norm(X, W, out_dtype=torch.int8, scales="row")
    Y, _ = ol.norm(host(X), host(W), 1e-5)
    err = (ol.norm_rel(cols) + 4 * ol.U32) * np.abs(Y)
    s = ol.row_scale(Y, "i8")
    check(r.scale, s, (ol.norm_rel(cols) + 6 * ol.U32) * s, "scale")
    check_codes(r.y, Y, err, host(r.scale)[:, None] * np.ones_like(Y), "i8")
    assert (r.y.to(torch.int32).abs().amax(dim=1) == 127).all()


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_quantised_rows(cols, dtype):
    """Scales are the fp32 quotient (integers: the product with 1/127), codes the rounded fp32 quotient by
    them: the same numbers as on the host."""
    say(f"quantise cols={cols} {dtype}")
    X = rand(cols, (7, cols), dtype, 3.0)
    X[3] = 0
    X[4] *= 1e-4
    x = X.float().cpu()
    for fmt in ("i8", "e4m3", "e5m2"):
        q, s = tg.quantize_rows(X, Q8[fmt])
        quo, want = (torch.from_numpy(v).float() for v in ol.quantised_rows(x.double().numpy(), fmt))
        assert torch.equal(s.cpu(), want), fmt
        codes = quo.round().to(torch.int8) if fmt == "i8" else quo.to(T[fmt])
        assert torch.equal(q.view(torch.int8).cpu(), codes.view(torch.int8)), fmt
        if fmt != "i8" and cols % 32 == 0:
            q, s = tg.quantize_rows(X, T[fmt], scales="block")
            e = torch.from_numpy(ol.block_scale(x.double().numpy(), fmt))
            assert torch.equal(s.view(torch.uint8).cpu(), (e + 127).to(torch.uint8))
            assert torch.equal(q.view(torch.int8).cpu(), torch.ldexp(x, -e.repeat_interleave(32, 1)).to(T[fmt]).view(torch.int8))


def test_quantised_rows_at_ties_and_extremes():
    say("quantise ties")
    # the scale is 1: halves go to the even integer
    X = torch.tensor([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5, -126.5, 3.49999, -0.0, 125.5]], device=dev())
    q, s = tg.quantize_rows(X)
    assert float(s) == 1.0 and q.cpu().tolist() == [[127, 0, 2, 2, 0, -2, -2, 126, -126, 3, 0, 126]]
    big = torch.tensor([[3e38, -3e38, 1.0, 2e36]], device=dev())
    q, s = tg.quantize_rows(big)
    assert q.cpu().tolist() == [[127, -127, 0, 1]] and np.isfinite(float(s))
    q, s = tg.quantize_rows(torch.full((2, 9), 1e-38, device=dev()))   # below the floor of the largest magnitude
    assert not q.any() and (s > 0).all()


@pytest.mark.parametrize("cols", [7, 64, 2048, 20000])
@pytest.mark.parametrize("out", [torch.float8_e4m3fn, torch.float8_e5m2])
def test_signs_of_zeros(cols, out):
    """An RMS norm's zeros have code 0 whatever their sign; quantize_rows' keep it."""
    X = torch.zeros(3, cols, device=dev())
    X[:, 0] = 1.0
    X[:, 1::2] = -0.0
    w = torch.ones(cols, device=dev())
    w[2::4] = -1.0   # zeros of either sign from a zero and its weight
    y = tg.rms_norm(X, w, scales="row", out_dtype=out).y.view(torch.uint8)
    assert not y[:, 1:].any() and y[:, 0].all()
    q, _ = tg.quantize_rows(X, out)
    assert torch.equal(q.view(torch.uint8)[:, 1:] == 0x80, torch.signbit(X[:, 1:]))


@pytest.mark.parametrize("rows,cols", [(1, 96), (9, 2057), (300, 1000), (5, 20001)])
def test_quantised_slices(rows, cols):
    say(f"quantise slices {rows}x{cols}")
    X = rand(3, (rows, cols), "bf16")
    q0, s0 = tg.quantize_rows(X)
    x = wide(X, 3, 2, float("nan"))[0]
    q, s = tg.quantize_rows(x)
    assert torch.equal(q, q0) and torch.equal(s, s0)
    Y = torch.full((rows, cols + 5), 99, dtype=torch.int8, device=dev())
    tg.tile_quantize_rows(x, Y[:, 2:2 + cols], s, rows, cols, tg.TG_BF16, tg.TG_I8, tg.TG_SCALE_ROW, ld_x=x.stride(0) if rows > 1 else 0,
                          ld_y=cols + 5)
    assert torch.equal(Y[:, 2:2 + cols], q0) and bool((Y[:, :2] == 99).all()) and bool((Y[:, 2 + cols:] == 99).all())


def grads_inputs(rows, cols, dtype):
    H, W, dY, dH = (rand(cols + i, s, dtype) for i, s in enumerate([(rows, cols), (cols,), (rows, cols), (rows, cols)]))
    H += 0.75
    h = H.float()
    mean = h.mean(dim=1)
    return H, W, dY, dH, mean, torch.rsqrt((h - mean[:, None]).square().mean(dim=1) + 1e-5)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_backward_lengths(cols, dtype):
    say(f"layer norm backward cols={cols} {dtype}")
    H, W, dY, dH, mean, rstd = grads_inputs(11, cols, dtype)
    for d in (None, dH):
        dX, dw, db = tg.layer_norm_backward(dY, H, W, mean, rstd, dH=d)
        ref, bound, wref, wbound, bref, bbound = ol.layer_norm_backward(host(dY), host(H), host(W), host(mean), host(rstd),
                                                                        None if d is None else host(d), dtype)
        check(dX, ref, bound, "dX")
        check(dw, wref, wbound, "dw")
        check(db, bref, bbound, "db")


@pytest.mark.parametrize("rows", [1, 2, 4, 5, 700, 3001])
@pytest.mark.parametrize("cols", [5, 100, 1032, 4104])
def test_backward_rows_and_workspaces(rows, cols):
    say(f"layer norm backward rows={rows} cols={cols}")
    H, W, dY, dH, mean, rstd = grads_inputs(rows, cols, "bf16")
    dX, dw, db = tg.layer_norm_backward(dY, H, W, mean, rstd, dH=dH)
    ref, bound, wref, wbound, bref, bbound = ol.layer_norm_backward(host(dY), host(H), host(W), host(mean), host(rstd), host(dH), "bf16")
    check(dX, ref, bound, "dX")
    check(dw, wref, wbound, "dw")
    check(db, bref, bbound, "db")
    for nw, nb in ((0, 1), (1, 0), (0, 0)):
        got = tg.layer_norm_backward(dY, H, W, mean, rstd, dH=dH, need_dw=nw, need_dbias=nb)
        assert torch.equal(got[0], dX)
        for g, w, n in ((got[1], dw, nw), (got[2], db, nb)):
            assert torch.equal(g, w) if n else g is None
    # fewer workgroups with smaller workspaces, dX in place of dY and of dH
    bf, least = tg.TG_BF16, 8 * rows if cols < 8 else 0
    for n in (least, least + 16 * cols, least + 80 * cols):
        ws = torch.empty(n, dtype=torch.uint8, device=dev()) if n else None
        for place in (0, 1):
            y, h = dY.clone(), dH.clone()
            w, b = torch.empty(cols, device=dev()), torch.empty(cols, device=dev())
            x = (y, h)[place]
            tg.tile_layernorm_bwd(y, H, W, mean, rstd, h, x, w, b, rows, cols, bf, bf, workspace=ws)
            assert torch.equal(x, dX)
            check(w, wref, wbound, "dw")
            check(b, bref, bbound, "db")


def test_backward_of_no_rows():
    e, W, v = torch.zeros(0, 40, device=dev()), torch.ones(40, device=dev()), torch.zeros(0, device=dev())
    dX, dw, db = tg.layer_norm_backward(e, e, W, v, v)
    assert dX.shape == (0, 40) and not dw.any() and not db.any()


@pytest.mark.parametrize("rows,cols", [(5, 7), (3, 40), (2, 1100)])
def test_gradients_against_differences(rows, cols):
    """fp32 results of the forward pass, its inputs moved by a step: sums of 64-bit differences of the
    formula, and the backward pass within 1e-3 of them."""
    say(f"layer norm differences {rows}x{cols}")
    rng = np.random.default_rng(cols)
    x, w, b, g = (rng.normal(size=s) for s in ((rows, cols), (cols,), (cols,), (rows, cols)))
    g = g.astype(np.float32).astype(np.float64)
    X = torch.from_numpy(x.astype(np.float32)).to(dev())
    W, B, G = (torch.from_numpy(v.astype(np.float32)).to(dev()) for v in (w, b, g))
    r = tg.layer_norm(X, W, B)
    dX, dw, db = (host(t) for t in tg.layer_norm_backward(G, r.h, W, r.mean, r.rstd))
    x, w, b = host(X), host(W), host(B)

    def loss(x, w, b):
        d = x - x.mean(axis=1, keepdims=True)
        return float((g * (d / np.sqrt((d * d).mean(axis=1, keepdims=True) + 1e-5) * w + b)).sum())

    for grad, at in ((dX, 0), (dw, 1), (db, 2)):
        for i in rng.choice(grad.size, size=6):
            step = np.zeros(grad.size)
            step[i] = 1e-5
            hi, lo = ([v + k * step.reshape(v.shape) if j == at else v for j, v in enumerate((x, w, b))] for k in (1, -1))
            slope = (loss(*hi) - loss(*lo)) / 2e-5
            assert abs(grad.reshape(-1)[i] - slope) <= 1e-3 * (1 + abs(slope))


@pytest.mark.parametrize("cols", [4, 8])
def test_more_rows_than_a_launch(cols):
    """2^21 rows a launch: the second launch's rows have their own means, scales and sums."""
    rows = (1 << 21) + 9
    say(f"layer norm rows={rows} cols={cols}")
    H, W, dY, _, mean, rstd = grads_inputs(rows, cols, "bf16")
    r = tg.layer_norm(H, W, out_dtype=torch.int8, scales="row")
    tail = tg.layer_norm(H[-32:], W, out_dtype=torch.int8, scales="row")
    for k in ("mean", "rstd", "scale", "y"):
        assert torch.equal(getattr(r, k)[-32:], getattr(tail, k)), k
    q, s = tg.quantize_rows(H)
    q1, s1 = tg.quantize_rows(H[-32:])
    assert torch.equal(q[-32:], q1) and torch.equal(s[-32:], s1)
    dX, dw, db = tg.layer_norm_backward(dY, H, W, mean, rstd)
    last = tg.layer_norm_backward(dY[-32:], H[-32:], W, mean[-32:], rstd[-32:])[0]
    assert torch.equal(dX[-32:], last)
    xh = (host(H) - host(mean)[:, None]) * host(rstd)[:, None]
    n = (rows + 8) * 2 * ol.U32
    check(dw, (host(dY) * xh).sum(axis=0), (n + 4 * ol.U32) * np.abs(host(dY) * xh).sum(axis=0), "dw")
    check(db, host(dY).sum(axis=0), n * np.abs(host(dY)).sum(axis=0), "db")


def test_on_another_stream_and_captured():
    say("layer norm streams and graphs")
    X, R, W, B = (rand(i, s, "bf16") for i, s in enumerate([(600, 2048), (600, 2048), (2048,), (2048,)]))

    def step():
        n = tg.layer_norm(X, W, B, residual=R)
        return (n.y, n.mean, n.rstd, *tg.quantize_rows(n.y), *tg.layer_norm_backward(R, n.h, W, n.mean, n.rstd, dH=X))

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    n = tg.layer_norm(X, W, B, residual=R, stream=s)
    q, sc = tg.quantize_rows(n.y, stream=s)
    dX, dw, db = tg.layer_norm_backward(R, n.h, W, n.mean, n.rstd, dH=X, stream=s)
    s.synchronize()
    for g, w in zip((n.y, n.mean, n.rstd, q, sc, dX, dw, db), want):
        assert torch.equal(g, w)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for k in range(3):
        X.copy_(rand(40 + k, (600, 2048), "bf16"))
        want = step()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
