"""Layer operators on the GPU against the float64 reference: product with an epilogue, RMS norm,
their backward passes.  Tolerances are oracle/layer.py's bounds."""

import ctypes

import numpy as np
import pytest
import torch

import tile_level_gemm_amd as tg
from oracle import layer as ol

from .gpu_util import say

pytestmark = pytest.mark.gpu

T = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn,
     "e5m2": torch.float8_e5m2}


def dev():
    return torch.device("cuda:0")


def host(t):
    """float64 values of a tensor."""
    return t.detach().to(torch.float32).cpu().numpy().astype(np.float64)


def rand(seed, shape, dtype, scale=1.0):
    x = torch.from_numpy(np.random.default_rng(seed).normal(size=shape).astype(np.float32) * scale)
    return x.to(T[dtype]).to(dev())


def check(got, ref, bound, what):
    got = host(got)
    assert got.shape == ref.shape, what
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    ok = np.isnan(ref) | (np.abs(got - ref) <= bound)
    if not ok.all():
        i = np.unravel_index(np.argmax(np.where(ok, 0, np.abs(got - ref) / bound)), ref.shape)
        raise AssertionError(f"{what}: {np.count_nonzero(~ok)} of {ok.size} outside, worst at {i}: got {got[i]}, "
                             f"reference {ref[i]}, bound {bound[i]}")


def wide(t, before, after, fill):
    """The same matrix as a slice of a wider one whose other columns hold `fill`."""
    w = torch.full((t.shape[0], before + t.shape[1] + after), fill, dtype=torch.float32, device=t.device).to(t.dtype)
    v = w[:, before:before + t.shape[1]]
    v.copy_(t)
    return v, w


# ------------------------------------------------------------------------------ product ----

SIZES = [(1, 1, 1), (1, 8, 64), (3, 5, 7), (2, 300, 1000), (16, 16, 32), (17, 33, 65), (33, 130, 200), (127, 129, 130),
         (128, 128, 128), (129, 257, 64), (130, 264, 1032), (256, 256, 512), (64, 72, 4096), (300, 520, 264), (5, 7, 3001),
         (1024, 520, 72)]


def operands(seed, M, N, K, ta, tb, dtype):
    a = rand(seed, (K, M) if ta else (M, K), dtype)
    b = rand(seed + 1, (N, K) if tb else (K, N), dtype, 0.25)
    return a, b, host(a).T if ta else host(a), host(b).T if tb else host(b)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("ta,tb", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_product_sizes_and_orientations(M, N, K, ta, tb, dtype):
    say(f"product {M}x{N}x{K} ta={ta} tb={tb} {dtype}")
    a, b, A, B = operands(M + N + K, M, N, K, ta, tb, dtype)
    D = tg.gemm_ep(a, b, trans_a=ta, trans_b=tb)
    ref, _, bound, _ = ol.product(A, B, out=dtype)
    check(D, ref, bound, "D")
    # without a workspace the sum is not split: the same problem on the other plan, in fp32
    D = torch.empty((M, N), device=dev())
    t = tg.TORCH_DTYPES[a.dtype]
    tg.tile_gemm_ep(a, b, D, M, N, K, ta, tb, t, t, tg.TG_F32)
    ref, _, bound, _ = ol.product(A, B, out="f32")
    check(D, ref, bound, "D without a workspace")


@pytest.mark.parametrize("M,N,K", SIZES + [(2048, 1032, 416), (20, 4096, 4096)])
@pytest.mark.parametrize("ta_,tb_", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
def test_product_fp8(M, N, K, ta_, tb_):
    say(f"product fp8 {M}x{N}x{K} {ta_} {tb_}")
    a, b = rand(M + K, (M, K), ta_, 4.0), rand(N + K, (N, K), tb_, 4.0)
    rs = torch.rand(M, device=dev()) * 0.02 + 0.01
    cs = torch.rand(N, device=dev()) * 0.02 + 0.01
    D = tg.gemm_ep(a, b, row_scale=rs, col_scale=cs)
    ref, _, bound, _ = ol.product(host(a), host(b).T, row_scale=host(rs), col_scale=host(cs), eight=True)
    check(D, ref, bound, "D")


@pytest.mark.parametrize("M,N,K,ta,tb,dtype", [
    (2304, 4112, 136, 0, 1, "bf16"), (2056, 4096, 200, 0, 0, "f16"), (2048, 2056, 1000, 1, 0, "bf16"),
    (4104, 2048, 64, 1, 1, "f16"), (256, 512, 8192, 0, 1, "bf16"), (384, 136, 5000, 1, 0, "f16")])
def test_product_large_plans(M, N, K, ta, tb, dtype):
    """256-wide blocks, partial last stages, odd stage counts, split sums."""
    say(f"product large {M}x{N}x{K} ta={ta} tb={tb} {dtype}")
    a, b, A, B = operands(M, M, N, K, ta, tb, dtype)
    bias, res = rand(5, (N,), dtype), rand(6, (M, N), dtype)
    D, Z = tg.gemm_ep(a, b, bias=bias, act="silu", residual=res, trans_a=ta, trans_b=tb, keep_z=True)
    ref, zref, bound, zbound = ol.product(A, B, "silu", host(bias), host(res), out=dtype)
    check(Z, zref, zbound, "Z")
    check(D, ref, bound, "D")
    again = tg.gemm_ep(a, b, bias=bias, act="silu", residual=res, trans_a=ta, trans_b=tb)
    assert torch.equal(again, D)   # the same bits every time


@pytest.mark.parametrize("act", ol.ACTS)
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 40, 96), (37, 75, 130), (200, 136, 2048)])
def test_epilogue_parts(act, out, M, N, K):
    say(f"epilogue {act} {out} {M}x{N}x{K}")
    a, b, A, B = operands(M, M, N, K, 0, 1, "bf16")
    bias = rand(7, (N,), "f32" if out == "f16" else out)
    res = rand(8, (M, N), out)
    rs, cs = rand(9, (M,), "f32"), rand(10, (N,), "f32")
    for use in range(8):   # each part alone and together
        kw = dict(bias=bias if use & 1 else None, residual=res if use & 2 else None,
                  row_scale=rs if use & 4 else None, col_scale=cs if use & 4 else None)
        D, Z = tg.gemm_ep(a, b, act=act, out_dtype=T[out], keep_z=True, **kw)
        ref, zref, bound, zbound = ol.product(A, B, act, out=out, **{k: None if v is None else host(v) for k, v in kw.items()})
        check(Z, zref, zbound, f"Z use={use}")
        check(D, ref, bound, f"D use={use}")


@pytest.mark.parametrize("M,N,K,ta,tb", [(40, 72, 136, 0, 1), (33, 41, 57, 0, 0), (1, 64, 256, 0, 1), (130, 264, 4096, 0, 1), (64, 40, 72, 1, 0)])
@pytest.mark.parametrize("before,after", [(0, 8), (3, 5), (8, 24)])
def test_slices_and_gaps(M, N, K, ta, tb, before, after):
    """Operands and results as slices of wider matrices: NaN in the gaps stays out, the gaps of the
    results stay as they were."""
    say(f"slices {M}x{N}x{K} ta={ta} tb={tb} {before},{after}")
    a, b, A, B = operands(3, M, N, K, ta, tb, "bf16")
    a, b = wide(a, before, after, float("nan"))[0], wide(b, before, after, float("nan"))[0]
    res = rand(4, (M, N), "bf16")
    r, _ = wide(res, before, after, float("nan"))
    d, dw = wide(torch.zeros_like(res), before, after, 77.0)
    z, zw = wide(torch.zeros_like(res), before, after, 55.0)
    lda, ldb, ldd = a.stride(0), b.stride(0), d.stride(0)
    bf = tg.TG_BF16
    nb = tg.tile_gemm_ep_workspace(M, N, K, ta, tb, bf)
    ws = torch.empty(max(nb, 16), dtype=torch.uint8, device=dev())
    tg.tile_gemm_ep(a, b, d, M, N, K, ta, tb, bf, bf, bf, lda=lda, ldb=ldb, ldd=ldd, residual=r, ld_residual=ldd, Z=z,
                    ld_z=ldd, act=tg.TG_ACT_RELU, workspace=ws)
    ref, zref, bound, zbound = ol.product(A, B, "relu", residual=host(res))
    check(d, ref, bound, "D")
    check(z, zref, zbound, "Z")
    for w, fill in ((dw, 77.0), (zw, 55.0)):
        gap = torch.cat([w[:, :before], w[:, before + N:]], dim=1)
        assert bool((gap == fill).all())
    # in place: the residual is D itself
    d2, dw2 = wide(res, before, after, 77.0)
    tg.tile_gemm_ep(a, b, d2, M, N, K, ta, tb, bf, bf, bf, lda=lda, ldb=ldb, ldd=ldd, residual=d2, ld_residual=ldd,
                    act=tg.TG_ACT_RELU, workspace=ws)
    assert torch.equal(d2, d)


def test_product_empty_extents():
    say("product empty extents")
    z = torch.zeros
    assert tg.gemm_ep(z(0, 8, dtype=T["bf16"], device=dev()), z(4, 8, dtype=T["bf16"], device=dev())).shape == (0, 4)
    bias, res = rand(1, (5,), "bf16"), rand(2, (3, 5), "bf16")
    D = tg.gemm_ep(z(3, 0, dtype=T["bf16"], device=dev()), z(5, 0, dtype=T["bf16"], device=dev()), bias=bias, act="gelu",
                   residual=res)
    ref, _, bound, _ = ol.product(np.zeros((3, 0)), np.zeros((0, 5)), "gelu", host(bias), host(res))
    check(D, ref, bound, "K = 0")


@pytest.mark.parametrize("M", [1, 5, 40, 300])
@pytest.mark.parametrize("tb", [0, 1])
def test_product_nan_and_infinity_stay_in_their_row_and_column(M, tb):
    say(f"product nan M={M} tb={tb}")
    N, K = 136, 264
    a, b, A, B = operands(5, M, N, K, 0, tb, "bf16")
    row, col = M - 1, 70
    a[row, 11] = float("nan")
    (b[col] if tb else b[:, col])[3] = float("inf")
    D = host(tg.gemm_ep(a, b, trans_b=tb))
    ref, _, bound, _ = ol.product(A, B)
    assert np.isnan(D[row]).all()
    assert not np.isfinite(D[:, col]).any()
    keep = np.ones((M, N), bool)
    keep[row], keep[:, col] = False, False
    assert (np.abs(D - ref) <= bound)[keep].all()


def test_activation_extremes():
    """Large finite arguments reach the activation's limits, not NaN."""
    say("activation extremes")
    z = torch.tensor([[0.0, -0.0, 1e4, -1e4, 6e4, -6e4, 30.0, -30.0]], dtype=T["f16"], device=dev())
    zb = torch.tensor([[0.0, -0.0, 1e19, -1e19, 3e38, -3e38, 30.0, -30.0]], dtype=T["bf16"], device=dev())
    for x in (z, zb):
        eye = torch.eye(8, dtype=x.dtype, device=dev())
        one = torch.ones_like(x)
        for kind in ol.ACTS:
            d = host(tg.gemm_ep(torch.zeros_like(x), eye, bias=x.reshape(-1), act=kind))
            dz = host(tg.gemm_ep_backward(one, x, eye, Z=x, act=kind, need_dA=False, need_dB=False)[0])
            v = host(x)
            want = v if kind == "none" else np.maximum(v, 0.0)
            slope = np.ones_like(v) if kind == "none" else np.where(v > 0, 1.0, 0.0)
            assert np.isfinite(dz).all()
            big = np.abs(v) >= 30
            assert np.allclose(d[big], want[big], rtol=2 ** -8, atol=1e-10)
            assert np.allclose(dz[big], slope[big], rtol=2 ** -8, atol=1e-9)


def test_product_offsets_past_32_bits():
    """Rows of A, B, D and Z further apart than 2^31 bytes in all: 64-bit addresses everywhere."""
    say("product offsets past 32 bits")
    M, N, K, ld = 300, 72, 96, 9_000_001
    pool = torch.empty(M * ld + 4096, dtype=torch.bfloat16, device=dev())   # 5.4 GB
    a = torch.as_strided(pool, (M, K), (ld, 1), 0)
    d = torch.as_strided(pool, (M, N), (ld, 1), 1000)
    z = torch.as_strided(pool, (M, N), (ld, 1), 2000)
    a0, b, A, B = operands(3, M, N, K, 0, 1, "bf16")
    a.copy_(a0)
    bf = tg.TG_BF16
    tg.tile_gemm_ep(a, b, d, M, N, K, 0, 1, bf, bf, bf, lda=ld, ldd=ld, Z=z, ld_z=ld)
    ref, zref, bound, zbound = ol.product(A, B)
    check(d, ref, bound, "D")
    check(z, zref, zbound, "Z")
    # A stored [K][M] with K rows that far apart
    at = torch.as_strided(pool, (K, M), (3 * ld, 1), 0)
    at.copy_(a0.t())
    check(tg.gemm_ep(at, b, trans_a=True), ref, bound, "D, A transposed")
    # one token: row pitch plays no part, weights far apart do
    bw = torch.as_strided(pool, (N, K), (ld, 1), 0)
    bw.copy_(b)
    check(tg.gemm_ep(a0[:1].contiguous(), bw), ref[:1], bound[:1], "one token")


@pytest.mark.parametrize("M,N,K,ta,tb", [(64, 72, 136, 0, 1), (33, 41, 57, 0, 0), (200, 520, 264, 1, 1), (1, 24, 40, 0, 1),
                                         (1000, 264, 128, 1, 0), (2, 1, 1, 0, 1)])
@pytest.mark.parametrize("act", ol.ACTS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_product_backward(M, N, K, ta, tb, act, dtype):
    say(f"product backward {M}x{N}x{K} ta={ta} tb={tb} {act} {dtype}")
    a, b, A, B = operands(M + K, M, N, K, ta, tb, dtype)
    dy, z = rand(8, (M, N), dtype), rand(9, (M, N), dtype, 2.0)
    dz, da, db, dbias = tg.gemm_ep_backward(dy, a, b, Z=z, act=act, trans_a=ta, trans_b=tb)
    ref, bound, sref, sbound = ol.act_backward(host(dy), host(z), act, dtype)
    check(dz, ref, bound, "dZ")
    check(dbias, sref, sbound, "dbias")
    G = host(dz)   # the products take dZ as it is held
    ref, bound = ol.matmul_bound(G, B.T, dtype)
    check(da.t() if ta else da, ref, bound, "dA")
    ref, bound = ol.matmul_bound(A.T, G, dtype)
    check(db.t() if tb else db, ref, bound, "dB")


def test_product_backward_parts_and_workspaces():
    """Any subset of the results, slices, dZ in place, small workspaces: the same numbers."""
    say("product backward parts")
    M, N, K, bf = 700, 272, 136, tg.TG_BF16
    a, b, A, B = operands(1, M, N, K, 0, 1, "bf16")
    dy, z = rand(2, (M, N), "bf16"), rand(3, (M, N), "bf16")
    dz, da, db, dbias = tg.gemm_ep_backward(dy, a, b, Z=z, act="silu")
    _, _, sref, sbound = ol.act_backward(host(dy), host(z), "silu", "bf16")
    for need in range(8):
        got = tg.gemm_ep_backward(dy, a, b, Z=z, act="silu", need_dA=need & 1, need_dB=need & 2, need_dbias=need & 4)
        for g, w, want in zip(got, (dz, da, db, dbias), (True, need & 1, need & 2, need & 4)):
            assert (g is not None and torch.equal(g, w)) if want else g is None
    for nb in (0, 4 * N * 3, 4 * N):
        s = torch.empty(N, dtype=torch.float32, device=dev())
        dzp = dy.clone()
        ws = torch.empty(nb, dtype=torch.uint8, device=dev()) if nb else None
        tg.tile_gemm_ep_bwd(dzp, z, a, b, dzp, None, None, s, M, N, K, 0, 1, bf, tg.TG_ACT_SILU, workspace=ws)
        assert torch.equal(dzp, dz)
        check(s, sref, sbound, f"dbias with {nb} bytes")
    dyw, zw = wide(dy, 3, 2, float("nan"))[0], wide(z, 3, 2, float("nan"))[0]
    got = tg.gemm_ep_backward(dyw, a, b, Z=zw, act="silu")
    assert torch.equal(got[0], dz) and torch.equal(got[1], da)
    none = tg.gemm_ep_backward(dyw, a, b)
    assert none[0] is dyw
    ref, bound = ol.matmul_bound(host(dy), B.T, "bf16")
    check(none[1], ref, bound, "dA of a slice")
    # empty batch: sums of nothing
    e = torch.zeros(0, N, dtype=T["bf16"], device=dev())
    _, _, db0, s0 = tg.gemm_ep_backward(e, a[:0], b, Z=e, act="silu")
    assert not db0.any() and not s0.any()


# --------------------------------------------------------------------------------- norm ----

COLS = [1, 7, 8, 9, 64, 96, 300, 512, 520, 1000, 1024, 1032, 2047, 2048, 2057, 4096, 5003, 8192, 8200, 16384, 16392, 20001]


def check_norm(r, X, R, W, eps, dtype, fmt, scales):
    """r against the formula on h as it is held (bit-exact sum), each result within its rounding."""
    if R is not None:
        assert torch.equal(r.h, (X.float() + R.float()).to(X.dtype))
    H, w = host(r.h), host(W)
    Y, rstd = ol.norm(H, w, eps)
    rel = ol.norm_rel(H.shape[1])
    check(r.rstd, rstd, rel * rstd, "rstd")
    err = (rel + 4 * ol.U32) * np.abs(Y)
    if scales is None:
        h = ol.HALF_STEP[dtype]
        check(r.y, Y, err * (1 + h) + h * np.abs(Y) + ol.TINY[dtype], "Y")
        return
    if scales == "row":
        s = ol.row_scale(Y, fmt)
        check(r.scale, s, (rel + 6 * ol.U32) * s, "scale")
        each = host(r.scale)[:, None] * np.ones_like(Y)
    else:
        got = r.scale.view(torch.uint8).cpu().numpy().astype(np.int64) - 127
        lo, hi = ol.block_scale(Y * (1 - rel - 4 * ol.U32), fmt), ol.block_scale(Y * (1 + rel + 4 * ol.U32), fmt)
        assert ((got >= lo) & (got <= hi)).all(), "block exponents"
        each = np.repeat(2.0 ** got, 32, axis=1)
    Q = host(r.y)
    h = ol.HALF_STEP[fmt]
    bound = (err * (1 + h) + (h + (rel + 8 * ol.U32) * 2) * np.abs(Y)) / each + ol.TINY[fmt]
    ok = np.abs(Q - Y / each) <= bound
    assert ok.all(), f"Q: {np.count_nonzero(~ok)} outside"


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_norm_lengths(cols, dtype):
    say(f"norm cols={cols} {dtype}")
    rows = 6
    X, R = rand(cols, (rows, cols), dtype, 3.0), rand(cols + 1, (rows, cols), dtype)
    W = rand(cols + 2, (cols,), dtype)
    check_norm(tg.rms_norm(X, W, 1e-5), X, None, W, 1e-5, dtype, None, None)
    check_norm(tg.rms_norm(X, W, 1e-5, residual=R), X, R, W, 1e-5, dtype, None, None)
    W32 = rand(cols + 3, (cols,), "f32")
    for fmt in ("e4m3", "e5m2"):
        check_norm(tg.rms_norm(X, W32, 1e-6, residual=R, out_dtype=T[fmt], scales="row"), X, R, W32, 1e-6, dtype, fmt, "row")
        if cols % 32 == 0:
            check_norm(tg.rms_norm(X, W, 1e-6, residual=R, out_dtype=T[fmt], scales="block"), X, R, W, 1e-6, dtype, fmt, "block")


@pytest.mark.parametrize("rows", [1, 3, 5, 513])
@pytest.mark.parametrize("cols", [96, 1024, 2336])
def test_norm_rows_slices_and_in_place(rows, cols):
    say(f"norm rows={rows} cols={cols}")
    X, R, W = rand(1, (rows, cols), "bf16"), rand(2, (rows, cols), "bf16"), rand(3, (cols,), "bf16")
    base = tg.rms_norm(X, W, residual=R, scales="row")
    check_norm(base, X, R, W, 1e-5, "bf16", "e4m3", "row")
    for before, after in ((0, 8), (3, 2)):
        x, r = wide(X, before, after, float("nan"))[0], wide(R, before, after, float("nan"))[0]
        got = tg.rms_norm(x, W, residual=r, scales="row")
        for k in ("h", "rstd", "scale"):
            assert torch.equal(getattr(got, k), getattr(base, k)), k
        assert torch.equal(got.y.view(torch.uint8), base.y.view(torch.uint8))
        for inplace in (0, 1):
            x, xw = wide(X, before, after, 9.0)
            r, rw = wide(R, before, after, 9.0)
            h = (x, r)[inplace]
            got = tg.rms_norm(x, W, residual=r, scales="row", h_out=h)
            assert torch.equal(h, base.h) and torch.equal(got.y.view(torch.uint8), base.y.view(torch.uint8))
            w = (xw, rw)[inplace]
            assert bool((torch.cat([w[:, :before], w[:, before + cols:]], dim=1) == 9.0).all())


@pytest.mark.parametrize("cols", [64, 2048, 20000])
def test_norm_rows_of_zeros_and_of_nan(cols):
    say(f"norm zeros and nan cols={cols}")
    X, W = rand(1, (5, cols), "bf16"), rand(2, (cols,), "bf16")
    X[1] = 0
    X[2, 3] = float("nan")
    X[3, cols - 1] = float("inf")
    X[4] *= 1e-30
    r = tg.rms_norm(X, W, 1e-5)
    y = host(r.y)
    assert not y[1].any() and np.isnan(y[2]).all() and np.isfinite(y[[0, 4]]).all()
    assert np.isnan(y[3, cols - 1]) and not y[3, :cols - 1].any()
    for kind in ("row", "block"):
        r = tg.rms_norm(X, W, 1e-5, scales=kind)
        s, q = host(r.scale), host(r.y)
        assert np.isfinite(s[[0, 1, 4]]).all() and (s[[0, 1, 4]] > 0).all() and not q[1].any()
        assert np.isnan(s[2]).all() and np.isnan(q[2]).all()
        assert np.isnan(s[3]).any() and np.isnan(q[3, cols - 1])
        assert np.isfinite(q[[0, 1, 4]]).all()
    zero = tg.rms_norm(torch.zeros(2, cols, dtype=T["bf16"], device=dev()), W, 0.0)   # 0·inf
    assert np.isnan(host(zero.y)).all()


def test_norm_feeds_the_products():
    """Row scales go into gemm_ep, block scales into tile_gemm_mx, as they are."""
    say("norm feeds the products")
    rows, cols, N = 64, 256, 128
    X, W = rand(1, (rows, cols), "bf16"), rand(2, (cols,), "bf16")
    w8 = rand(3, (N, cols), "e4m3", 8.0)
    cs = torch.rand(N, device=dev()) + 0.5
    r = tg.rms_norm(X, W, scales="row")
    D = tg.gemm_ep(r.y, w8, row_scale=r.scale, col_scale=cs)
    ref, _, bound, _ = ol.product(host(r.y), host(w8).T, row_scale=host(r.scale), col_scale=host(cs), eight=True)
    check(D, ref, bound, "row scales")
    r = tg.rms_norm(X, W, scales="block")
    sb = torch.full((N, cols // 32), 127, dtype=torch.uint8, device=dev())
    D = torch.empty((rows, N), device=dev())
    e4 = tg.TG_FP8_E4M3
    tg.tile_gemm_mx(r.y, w8, r.scale, sb, None, D, rows, N, cols, 0, 1, 0.0, e4, e4)
    A = host(r.y) * np.repeat(2.0 ** (r.scale.view(torch.uint8).cpu().numpy().astype(np.float64) - 127), 32, axis=1)
    ref, _, bound, _ = ol.product(A, host(w8).T, out="f32", eight=True)
    check(D, ref, bound, "block scales")


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_norm_backward_lengths(cols, dtype):
    say(f"norm backward cols={cols} {dtype}")
    rows = 11
    H, W, dY, dH = (rand(cols + i, s, dtype) for i, s in enumerate([(rows, cols), (cols,), (rows, cols), (rows, cols)]))
    rstd = torch.rsqrt(H.float().square().mean(dim=1) + 1e-5)
    for d in (None, dH):
        dX, dw = tg.rms_norm_backward(dY, H, W, rstd, dH=d)
        ref, bound, wref, wbound = ol.norm_backward(host(dY), host(H), host(W), host(rstd), None if d is None else host(d), dtype)
        check(dX, ref, bound, "dX")
        check(dw, wref, wbound, "dw")


@pytest.mark.parametrize("rows", [1, 2, 4, 5, 700, 3001])
@pytest.mark.parametrize("cols", [100, 1032, 4104])
def test_norm_backward_rows_and_workspaces(rows, cols):
    say(f"norm backward rows={rows} cols={cols}")
    H, dY, dH = (rand(i, (rows, cols), "bf16") for i in range(3))
    W = rand(4, (cols,), "f32")
    rstd = torch.rsqrt(H.float().square().mean(dim=1) + 1e-5)
    ref, bound, wref, wbound = ol.norm_backward(host(dY), host(H), host(W), host(rstd), host(dH), "bf16")
    dX, dw = tg.rms_norm_backward(dY, H, W, rstd, dH=dH)
    check(dX, ref, bound, "dX")
    check(dw, wref, wbound, "dw")
    only, none = tg.rms_norm_backward(dY, H, W, rstd, dH=dH, need_dw=False)
    assert none is None and torch.equal(only, dX)
    bf = tg.TG_BF16
    for nb in (0, 4 * cols, 4 * cols * 3):
        w = torch.empty(cols, device=dev())
        ws = torch.empty(nb, dtype=torch.uint8, device=dev()) if nb else None
        for place in (0, 1):   # in place over dY, over dH
            y, h = dY.clone(), dH.clone()
            tg.tile_rmsnorm_bwd(y, H, W, rstd, h, (y, h)[place], w, rows, cols, bf, tg.TG_F32, workspace=ws)
            assert torch.equal((y, h)[place], dX)
            check(w, wref, wbound, f"dw with {nb} bytes")
    yw, hw, dw_ = (wide(t, 3, 4, float("nan"))[0] for t in (dY, H, dH))
    got = tg.rms_norm_backward(yw, hw, W, rstd, dH=dw_)
    assert torch.equal(got[0], dX)


# ------------------------------------------------------------------- streams and graphs ----

def _chain(x, r, w, w1, b1, w2, stream=None):
    n = tg.rms_norm(x, w, residual=r, stream=stream)
    u, z = tg.gemm_ep(n.y, w1, bias=b1, act="gelu_tanh", keep_z=True, stream=stream)
    out = tg.gemm_ep(u, w2, residual=n.h, stream=stream)
    dz2, du, dw2, db2 = tg.gemm_ep_backward(out, u, w2, stream=stream)
    dz1, dn, dw1, db1 = tg.gemm_ep_backward(du, n.y, w1, Z=z, act="gelu_tanh", stream=stream)
    dx, dw = tg.rms_norm_backward(dn, n.h, w, n.rstd, dH=out, stream=stream)
    return [n.y, n.h, u, z, out, dw2, db2, dz1, dw1, db1, dx, dw]


def _chain_inputs(rows, cols, hidden):
    return (rand(1, (rows, cols), "bf16"), rand(2, (rows, cols), "bf16"), rand(3, (cols,), "bf16"),
            rand(4, (hidden, cols), "bf16", 0.1), rand(5, (hidden,), "bf16"), rand(6, (cols, hidden), "bf16", 0.1))


@pytest.mark.parametrize("rows", [3, 200])
def test_streams(rows):
    """On a stream of its own, given as an object or as a handle; results and workspaces belong to it."""
    say(f"layer streams rows={rows}")
    args = _chain_inputs(rows, 264, 1032)
    want = _chain(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for given in (s, s.cuda_stream):
        got = _chain(*args, stream=given)
        s.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)
    with torch.cuda.stream(s):
        got = _chain(*args)
    s.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("rows", [1, 200])
def test_graph_replays(rows):
    """Forward and backward captured once: every replay gives the eager results for the inputs of that
    moment, with eager work in between."""
    say(f"layer graph rows={rows}")
    args = _chain_inputs(rows, 264, 1032)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _chain(*args)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _chain(*args)
    for i in range(4):
        args[0].copy_(rand(50 + i, tuple(args[0].shape), "bf16"))
        g.replay()
        torch.cuda.synchronize()
        want = _chain(*args)
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), i


def test_calls_refuse_bad_tensors():
    say("layer refusals")
    a, b = rand(1, (4, 64), "bf16"), rand(2, (8, 64), "bf16")
    bad = [lambda: tg.gemm_ep(a, b[:, :32]), lambda: tg.gemm_ep(a, b.to(T["f16"])), lambda: tg.gemm_ep(a[0], b),
           lambda: tg.gemm_ep(a, b, bias=torch.zeros(7, device=dev())), lambda: tg.gemm_ep(a, b, act="tanh"),
           lambda: tg.gemm_ep(a, b, residual=torch.zeros(4, 8, device=dev())), lambda: tg.gemm_ep(a[:, ::2], b[:, ::2]),
           lambda: tg.gemm_ep(a, b, row_scale=torch.zeros(4, dtype=T["f16"], device=dev())),
           lambda: tg.gemm_ep(a.expand(4, 64), b.cpu()), lambda: tg.gemm_ep(a[:1].expand(4, 64), b),
           lambda: tg.gemm_ep(a, b, out=a[:, :8]), lambda: tg.gemm_ep_backward(a, a, b),
           lambda: tg.gemm_ep_backward(rand(3, (4, 8), "bf16"), a, b, act="silu"),
           lambda: tg.rms_norm(a, b[0, :32]), lambda: tg.rms_norm(a, b[0], h_out=a), lambda: tg.rms_norm(a, b[0], scales="column"),
           lambda: tg.rms_norm(a[:, :48], b[0, :48], scales="block"), lambda: tg.rms_norm_backward(a, a, b[0], torch.zeros(3, device=dev()))]
    for i, call in enumerate(bad):
        with pytest.raises(tg.TileError):
            call()
            raise AssertionError(i)
