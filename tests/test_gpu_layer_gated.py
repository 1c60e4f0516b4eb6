"""Gated product and its backward pass on the GPU against the float64 reference.  Tolerances are
oracle/layer.py's bounds."""

import numpy as np
import pytest
import torch

import tile_level_gemm_amd as tg
from oracle import layer as ol

from .gpu_util import say
from .test_gpu_layer import T, check, dev, host, rand, wide
from .test_gpu_layer_i8 import ints

pytestmark = pytest.mark.gpu

SIZES = [(1, 1, 1), (1, 8, 64), (3, 5, 7), (2, 300, 1000), (16, 16, 32), (17, 33, 65), (32, 40, 520), (33, 65, 200), (127, 63, 130),
         (128, 64, 128), (129, 130, 64), (130, 136, 1032), (256, 128, 512), (64, 40, 4096), (300, 260, 264), (5, 7, 3001),
         (1024, 264, 72), (1, 4100, 256), (20, 1024, 512)]


def operands(seed, M, N, K, tb, dtype):
    a = rand(seed, (M, K), dtype)
    b = rand(seed + 1, (2 * N, K) if tb else (K, 2 * N), dtype, 0.25)
    return a, b, host(a), host(b).T if tb else host(b)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("tb", [0, 1])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_sizes_and_orientations(M, N, K, tb, dtype):
    say(f"gated {M}x{N}x{K} tb={tb} {dtype}")
    a, b, A, B = operands(M + N + K, M, N, K, tb, dtype)
    D, Z = tg.gemm_gated(a, b, trans_b=tb, keep_z=True)
    ref, zref, bound, zbound = ol.gated(A, B, out=dtype)
    check(D, ref, bound, "D")
    check(Z, zref, zbound, "Z")
    assert torch.equal(tg.gemm_gated(a, b, trans_b=tb), D)
    # without a workspace the sum is not split: the same problem on the other plan, in fp32
    D = torch.empty((M, N), device=dev())
    t = tg.TORCH_DTYPES[a.dtype]
    tg.tile_gemm_gated(a, b, D, M, N, K, tb, t, t, tg.TG_F32, act=tg.TG_ACT_SILU)
    ref, _, bound, _ = ol.gated(A, B, out="f32")
    check(D, ref, bound, "D without a workspace")


@pytest.mark.parametrize("M,N,K", SIZES + [(2048, 520, 416), (20, 2048, 4096)])
@pytest.mark.parametrize("ta_,tb_", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2"), ("i8", "i8")])
def test_eight_bits(M, N, K, ta_, tb_):
    say(f"gated {M}x{N}x{K} {ta_} {tb_}")
    if ta_ == "i8":
        a, b = ints(M + K, (M, K)), ints(N + K, (2 * N, K))
    else:
        a, b = rand(M + K, (M, K), ta_, 4.0), rand(N + K, (2 * N, K), tb_, 4.0)
    A, B = a.float().cpu().numpy().astype(np.float64), b.float().cpu().numpy().astype(np.float64).T
    rs, cs = (torch.rand(n, device=dev()) * 0.02 + 0.001 for n in (M, 2 * N))
    D, Z = tg.gemm_gated(a, b, row_scale=rs, col_scale=cs, act="gelu", keep_z=True)
    ref, zref, bound, zbound = ol.gated(A, B, "gelu", row_scale=host(rs), col_scale=host(cs), eight=ta_ != "i8", ints=ta_ == "i8")
    check(Z, zref, zbound, "Z")
    check(D, ref, bound, "D")


@pytest.mark.parametrize("M,N,K,tb,dtype", [
    (2304, 2056, 136, 1, "bf16"), (2056, 2048, 200, 0, "f16"), (2048, 1032, 1000, 0, "bf16"), (4104, 1024, 64, 1, "f16"),
    (256, 256, 8192, 1, "bf16"), (384, 72, 5000, 0, "f16"), (4096, 1024, 8192, 1, "bf16"), (512, 2048, 2048, 1, "f16")])
def test_large_plans(M, N, K, tb, dtype):
    """256-wide blocks, partial last stages, odd stage counts, split sums."""
    say(f"gated large {M}x{N}x{K} tb={tb} {dtype}")
    a, b, A, B = operands(M, M, N, K, tb, dtype)
    bias = rand(5, (2 * N,), dtype)
    D, Z = tg.gemm_gated(a, b, bias=bias, act="gelu_tanh", trans_b=tb, keep_z=True)
    ref, zref, bound, zbound = ol.gated(A, B, "gelu_tanh", host(bias), out=dtype)
    check(Z, zref, zbound, "Z")
    check(D, ref, bound, "D")
    assert torch.equal(tg.gemm_gated(a, b, bias=bias, act="gelu_tanh", trans_b=tb), D)   # the same bits every time


@pytest.mark.parametrize("act", ol.ACTS)
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 24, 96), (37, 43, 130), (200, 136, 2048)])
def test_epilogue_parts(act, out, M, N, K):
    say(f"gated epilogue {act} {out} {M}x{N}x{K}")
    a, b, A, B = operands(M, M, N, K, 1, "bf16")
    bias = rand(7, (2 * N,), "f32" if out == "f16" else out)
    rs, cs = rand(9, (M,), "f32"), rand(10, (2 * N,), "f32")
    for use in range(8):
        kw = dict(bias=bias if use & 1 else None, row_scale=rs if use & 2 else None, col_scale=cs if use & 4 else None)
        D, Z = tg.gemm_gated(a, b, act=act, out_dtype=T[out], keep_z=True, **kw)
        ref, zref, bound, zbound = ol.gated(A, B, act, out=out, **{k: None if v is None else host(v) for k, v in kw.items()})
        check(Z, zref, zbound, f"Z use={use}")
        check(D, ref, bound, f"D use={use}")


@pytest.mark.parametrize("M,N,K,tb", [(40, 72, 136, 1), (33, 41, 57, 0), (1, 64, 256, 1), (130, 132, 4096, 1), (64, 40, 72, 0)])
@pytest.mark.parametrize("before,after", [(0, 8), (3, 5), (8, 24)])
def test_slices_and_gaps(M, N, K, tb, before, after):
    """Operands and results as slices of wider matrices: NaN in the gaps stays out, the results' gaps stay."""
    say(f"gated slices {M}x{N}x{K} tb={tb} {before},{after}")
    a, b, A, B = operands(3, M, N, K, tb, "bf16")
    a, b = wide(a, before, after, float("nan"))[0], wide(b, before, after, float("nan"))[0]
    d, dw = wide(torch.zeros(M, N, dtype=T["bf16"], device=dev()), before, after, 77.0)
    z, zw = wide(torch.zeros(M, 2 * N, dtype=T["bf16"], device=dev()), before, after, 55.0)
    bf = tg.TG_BF16
    nb = tg.tile_gemm_gated_workspace(M, N, K, tb, bf)
    ws = torch.empty(max(nb, 16), dtype=torch.uint8, device=dev())
    tg.tile_gemm_gated(a, b, d, M, N, K, tb, bf, bf, bf, lda=a.stride(0), ldb=b.stride(0), ldd=d.stride(0), Z=z, ld_z=z.stride(0),
                       act=tg.TG_ACT_RELU, workspace=ws)
    ref, zref, bound, zbound = ol.gated(A, B, "relu")
    check(d, ref, bound, "D")
    check(z, zref, zbound, "Z")
    for w, n, fill in ((dw, N, 77.0), (zw, 2 * N, 55.0)):
        assert bool((torch.cat([w[:, :before], w[:, before + n:]], dim=1) == fill).all())
    o = torch.zeros_like(d.contiguous())
    assert tg.gemm_gated(a, b, act="relu", trans_b=tb, out=o) is o and torch.equal(o, d)


@pytest.mark.parametrize("M", [1, 5, 40, 300])
@pytest.mark.parametrize("tb", [0, 1])
@pytest.mark.parametrize("N", [72, 77])
def test_nan_and_infinity_stay_in_their_row_and_column(M, tb, N):
    say(f"gated nan M={M} tb={tb}")
    K = 264
    a, b, A, B = operands(5, M, N, K, tb, "bf16")
    row, col, up = M - 1, N - 1, 3
    a[row, 11] = float("nan")
    for c in (col, N + up):
        (b[c] if tb else b[:, c])[3] = float("inf")
    D, Z = (host(t) for t in tg.gemm_gated(a, b, act="none", trans_b=tb, keep_z=True))
    ref, zref, bound, zbound = ol.gated(A, B, "none")
    assert np.isnan(D[row]).all() and np.isnan(Z[row]).all()
    assert not np.isfinite(D[:, [col, up]]).any() and not np.isfinite(Z[:, [col, N + up]]).any()
    keep, zkeep = np.ones((M, N), bool), np.ones((M, 2 * N), bool)
    keep[row], zkeep[row], keep[:, [col, up]], zkeep[:, [col, N + up]] = False, False, False, False
    assert (np.abs(D - ref) <= bound)[keep].all() and (np.abs(Z - zref) <= zbound)[zkeep].all()


def test_empty_extents():
    say("gated empty extents")
    z = lambda *s: torch.zeros(*s, dtype=T["bf16"], device=dev())   # noqa: E731
    assert tg.gemm_gated(z(0, 8), z(6, 8)).shape == (0, 3) and tg.gemm_gated(z(4, 8), z(0, 8)).shape == (4, 0)
    bias = rand(1, (10,), "bf16")
    D, Z = tg.gemm_gated(z(3, 0), z(10, 0), bias=bias, keep_z=True)
    ref, zref, bound, zbound = ol.gated(np.zeros((3, 0)), np.zeros((0, 10)), bias=host(bias))
    check(D, ref, bound, "K = 0")
    check(Z, zref, zbound, "K = 0")
    with pytest.raises(tg.TileError):
        tg.gemm_gated(z(3, 8), z(7, 8))   # no two projections
    dz, da, db, s = tg.gemm_gated_backward(z(0, 4), z(0, 8), z(8, 8), z(0, 8))
    assert dz.shape == (0, 8) and da.shape == (0, 8) and not db.any() and not s.any()


def test_offsets_past_32_bits():
    """Rows of A, B, D and Z further apart than 2^31 bytes in all, and halves of B that far apart."""
    say("gated offsets past 32 bits")
    M, N, K, ld = 300, 72, 96, 9_000_001
    pool = torch.empty(M * ld + 4096, dtype=torch.bfloat16, device=dev())   # 5.4 GB
    a, d, z = (torch.as_strided(pool, s, (ld, 1), o) for s, o in (((M, K), 0), ((M, N), 1000), ((M, 2 * N), 2000)))
    a0, b, A, B = operands(3, M, N, K, 1, "bf16")
    a.copy_(a0)
    bf = tg.TG_BF16
    tg.tile_gemm_gated(a, b, d, M, N, K, 1, bf, bf, bf, lda=ld, ldd=ld, Z=z, ld_z=ld)
    ref, zref, bound, zbound = ol.gated(A, B, "none")
    check(d, ref, bound, "D")
    check(z, zref, zbound, "Z")
    bw = torch.as_strided(pool, (2 * N, K), (ld, 1), 0)
    bw.copy_(b)
    check(tg.gemm_gated(a0, bw, act="none"), ref, bound, "weights far apart")
    check(tg.gemm_gated(a0[:1].contiguous(), bw, act="none"), ref[:1], bound[:1], "one token")
    # aligned weights, each half within 32 bits, the up projection's past them
    ld = 1 << 24
    del a, d, z, bw, pool
    pool = torch.empty(2 * N * ld, dtype=torch.bfloat16, device=dev())   # 4.8 GB
    bw = torch.as_strided(pool, (2 * N, K), (ld, 1), 0)
    bw.copy_(b)
    check(tg.gemm_gated(a0, bw, act="none"), ref, bound, "halves far apart")


@pytest.mark.parametrize("M,N,K,tb", [(64, 72, 136, 1), (33, 41, 57, 0), (200, 264, 520, 1), (200, 264, 520, 0), (1, 24, 40, 1),
                                      (1000, 136, 128, 0), (2, 1, 1, 1), (700, 40, 2048, 1)])
@pytest.mark.parametrize("act", ol.ACTS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_backward(M, N, K, tb, act, dtype):
    say(f"gated backward {M}x{N}x{K} tb={tb} {act} {dtype}")
    a, b, A, B = operands(M + K, M, N, K, tb, dtype)
    dy, z = rand(8, (M, N), dtype), rand(9, (M, 2 * N), dtype, 2.0)
    rs, cs = rand(10, (M,), "f32"), rand(11, (2 * N,), "f32")
    for r, c in ((None, None), (rs, None), (rs, cs)):
        dz, da, db, dbias = tg.gemm_gated_backward(dy, a, b, z, act=act, trans_b=tb, row_scale=r, col_scale=c)
        ref, bound, sref, sbound = ol.gated_backward(host(dy), host(z), act, dtype, None if r is None else host(r),
                                                     None if c is None else host(c))
        check(dz, ref, bound, "dZ")
        check(dbias, sref, sbound, "dbias")
        G = host(dz)   # the products take dZ as it is held
        ref, bound = ol.matmul_bound(G, B.T, dtype)
        check(da, ref, bound, "dA")
        ref, bound = ol.matmul_bound(A.T, G, dtype)
        check(db.t() if tb else db, ref, bound, "dB")


def test_backward_parts_and_workspaces():
    """Any subset of the results, slices, dZ in place of Z, small workspaces: the same numbers."""
    say("gated backward parts")
    M, N, K, bf = 700, 136, 136, tg.TG_BF16
    a, b, A, B = operands(1, M, N, K, 1, "bf16")
    dy, z = rand(2, (M, N), "bf16"), rand(3, (M, 2 * N), "bf16")
    dz, da, db, dbias = tg.gemm_gated_backward(dy, a, b, z)
    _, _, sref, sbound = ol.gated_backward(host(dy), host(z), "silu", "bf16")
    for need in range(8):
        got = tg.gemm_gated_backward(dy, a, b, z, need_dA=need & 1, need_dB=need & 2, need_dbias=need & 4)
        for g, w, want in zip(got, (dz, da, db, dbias), (True, need & 1, need & 2, need & 4)):
            assert (g is not None and torch.equal(g, w)) if want else g is None
    for nb in (0, 8 * N * 3, 8 * N):
        s = torch.empty(2 * N, dtype=torch.float32, device=dev())
        dzp = z.clone()
        ws = torch.empty(nb, dtype=torch.uint8, device=dev()) if nb else None
        tg.tile_gemm_gated_bwd(dy, dzp, a, b, dzp, None, None, s, M, N, K, 1, bf, tg.TG_ACT_SILU, workspace=ws)
        assert torch.equal(dzp, dz)
        check(s, sref, sbound, f"dbias with {nb} bytes")
    dyw, zw, aw = (wide(t, 3, 2, float("nan"))[0] for t in (dy, z, a))
    got = tg.gemm_gated_backward(dyw, aw, b, zw)
    assert torch.equal(got[0], dz) and torch.equal(got[1], da)
    ref, bound = ol.matmul_bound(A.T, host(dz), "bf16")
    check(got[2].t(), ref, bound, "dB of slices")


def test_activation_extremes():
    """Large finite gates reach the activation's limits, not NaN, with a finite up projection."""
    say("gated extremes")
    v = torch.tensor([[0.0, -0.0, 1e19, -1e19, 3e38, -3e38, 30.0, -30.0]], dtype=T["bf16"], device=dev())
    up = torch.full_like(v, 0.5)
    eye = torch.zeros(16, 8, dtype=v.dtype, device=dev())
    for kind in ol.ACTS:
        bias = torch.cat([v, up], dim=1).reshape(-1)
        d, z = tg.gemm_gated(torch.zeros_like(v), eye, bias=bias, act=kind, keep_z=True)
        assert torch.equal(z.reshape(-1), bias)
        dz = host(tg.gemm_gated_backward(torch.ones_like(v), torch.zeros_like(v), eye, z, act=kind, need_dA=False, need_dB=False)[0])
        x = host(v)
        want = x if kind == "none" else np.maximum(x, 0.0)
        slope = np.ones_like(x) if kind == "none" else np.where(x > 0, 1.0, 0.0)
        big = np.abs(x) >= 30
        assert np.allclose(host(d)[big], 0.5 * want[big], rtol=2 ** -8, atol=1e-10)
        assert np.allclose(dz[:, 8:][big], want[big], rtol=2 ** -8, atol=1e-9)
        assert np.allclose(dz[:, :8][big], 0.5 * slope[big], rtol=2 ** -8, atol=1e-9)


@pytest.mark.parametrize("act", ol.ACTS)
def test_gradients_against_differences(act):
    """dA and dB of the whole layer against 64-bit differences of the formula.  fp16 rounds G, U and dZ by
    2^-11 of them: dU moves by its slope (at most 1.13) and dG by the slope's (at most 1.6) times G's
    rounding, both by U's and their own."""
    say(f"gated differences {act}")
    M, N, K = 6, 5, 9
    a, b, A, B = operands(21, M, N, K, 1, "f16")
    dy = rand(23, (M, N), "f16")
    _, z = tg.gemm_gated(a, b, act=act, keep_z=True)
    dz, da, db, _ = tg.gemm_gated_backward(dy, a, b, z, act=act)
    w, dz, Z = host(dy), np.abs(host(dz)), host(z)
    G, U = np.abs(Z[:, :N]), np.abs(Z[:, N:])
    off = 2.0 ** -11 * (2.1 * dz + np.concatenate([1.6 * np.abs(w) * U * G, 1.13 * np.abs(w) * G], axis=1))

    def loss(A, B):
        Z = A @ B
        return float((w * ol.act(Z[:, :N], act) * Z[:, N:]).sum())

    rng = np.random.default_rng(5)
    for grad, tol, at, X in ((host(da), off @ np.abs(B).T, 0, A), (host(db).T, np.abs(A).T @ off, 1, B)):
        for i in rng.choice(X.size, size=10):
            step = np.zeros(X.size)
            step[i] = 1e-5
            step = step.reshape(X.shape)
            hi, lo = ((A + k * step, B) if at == 0 else (A, B + k * step) for k in (1, -1))
            slope = (loss(*hi) - loss(*lo)) / 2e-5
            assert abs(grad.reshape(-1)[i] - slope) <= tol.reshape(-1)[i] + 2.0 ** -11 * abs(slope) + 1e-6
    

def test_on_another_stream_and_captured():
    say("gated streams and graphs")
    a, b, _, _ = operands(1, 256, 512, 4096, 1, "bf16")
    dy = rand(5, (256, 512), "bf16")

    def step():
        d, z = tg.gemm_gated(a, b, keep_z=True)
        return (d, z, *tg.gemm_gated_backward(dy, a, b, z))

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    d, z = tg.gemm_gated(a, b, keep_z=True, stream=s)
    got = (d, z, *tg.gemm_gated_backward(dy, a, b, z, stream=s))
    s.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for k in range(3):
        a.copy_(rand(60 + k, (256, 4096), "bf16"))
        want = step()
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


def test_one_eight_bit_feed_forward_layer():
    """Layer norm to integer rows, the gated product of integers, its result quantised, the down projection
    onto the residual stream: each operator against the values it was given."""
    say("gated feed-forward i8")
    M, K, N = 48, 256, 512
    x, r, w = rand(1, (M, K), "bf16"), rand(2, (M, K), "bf16"), rand(3, (K,), "bf16")
    wg, sg = tg.quantize_rows(rand(4, (2 * N, K), "bf16", K ** -0.5))
    wd, sd = tg.quantize_rows(rand(5, (K, N), "bf16", N ** -0.5))
    n = tg.layer_norm(x, w, residual=r, out_dtype=torch.int8, scales="row")
    u = tg.gemm_gated(n.y, wg, row_scale=n.scale, col_scale=sg)
    q, sq = tg.quantize_rows(u)
    out = tg.gemm_ep(q, wd, row_scale=sq, col_scale=sd, residual=n.h)
    f = lambda t: t.float().cpu().numpy().astype(np.float64)   # noqa: E731
    ref, _, bound, _ = ol.gated(f(n.y), f(wg).T, row_scale=f(n.scale), col_scale=f(sg), ints=True)
    check(u, ref, bound, "gated")
    ref, _, bound, _ = ol.product(f(q), f(wd).T, residual=f(n.h), row_scale=f(sq), col_scale=f(sd), ints=True)
    check(out, ref, bound, "down")
