"""Every kernel of the layer operators at the sizes where it can go wrong: few rows, 64-, 128- and 256-wide
blocks, the ring of stages, register-staged edges, parts of a sum, rows of every wave count.  Bounds
are oracle/layer.py's."""

import numpy as np
import pytest
import torch

import tile_level_gemm_amd as tg
from oracle import layer as ol

from .gpu_util import say
from .test_gpu_layer import T, check, check_norm, dev, host, operands, rand, wide

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------ few rows ----

@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 32])
@pytest.mark.parametrize("N,K", [(1, 9), (3, 64), (5, 63), (31, 65), (33, 127), (130, 1025), (2049, 200), (4097, 136), (8193, 72)])
@pytest.mark.parametrize("ta,tb", [(0, 1), (0, 0), (1, 1), (1, 0)])
def test_few_rows(M, N, K, ta, tb):
    say(f"few rows {M}x{N}x{K} ta={ta} tb={tb}")
    a, b, A, B = operands(M + N, M, N, K, ta, tb, "bf16")
    bias, res = rand(3, (N,), "bf16"), rand(4, (M, N), "bf16")
    D, Z = tg.gemm_ep(a, b, bias=bias, act="silu", residual=res, trans_a=ta, trans_b=tb, keep_z=True)
    ref, zref, bound, zbound = ol.product(A, B, "silu", host(bias), host(res))
    check(Z, zref, zbound, "Z")
    check(D, ref, bound, "D")


@pytest.mark.parametrize("M", [1, 16, 23])
@pytest.mark.parametrize("N,K", [(40, 3), (100, 128), (2050, 257), (8200, 640), (64, 5000)])
@pytest.mark.parametrize("at,bt", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
def test_few_rows_fp8(M, N, K, at, bt):
    say(f"few rows fp8 {M}x{N}x{K} {at} {bt}")
    a, b = rand(M + K, (M, K), at, 4.0), rand(N + K, (N, K), bt, 4.0)
    a, b = wide(a, 3, 2, 1.0)[0], wide(b, 1, 0, 1.0)[0]   # slices at odd addresses
    rs, cs = torch.rand(M, device=dev()) * 0.02 + 0.01, torch.rand(N, device=dev()) * 0.02 + 0.01
    D = tg.gemm_ep(a, b, row_scale=rs, col_scale=cs)
    ref, _, bound, _ = ol.product(host(a), host(b).T, row_scale=host(rs), col_scale=host(cs), eight=True)
    check(D, ref, bound, "D")


@pytest.mark.parametrize("M,N,K", [(1, 40, 3056), (32, 96, 2100), (5, 4096, 2048), (16, 33, 8191)])
@pytest.mark.parametrize("ta", [0, 1])
def test_few_rows_in_parts(M, N, K, ta):
    """[K][N] weights, K cut into parts: with the workspace, with part of it and without."""
    say(f"few rows in parts {M}x{N}x{K} ta={ta}")
    a, b, A, B = operands(M + N, M, N, K, ta, 0, "f16")
    ref, _, bound, _ = ol.product(A, B, out="f16")
    h = tg.TG_F16
    need = tg.tile_gemm_ep_workspace(M, N, K, ta, 0, h)
    assert need > 0
    for nb in (0, need // 2 // 16 * 16, need):
        ws = torch.full((nb,), 255, dtype=torch.uint8, device=dev()) if nb else None   # NaN where nothing is written
        D = torch.empty((M, N), dtype=T["f16"], device=dev())
        tg.tile_gemm_ep(a, b, D, M, N, K, ta, 0, h, h, h, workspace=ws)
        check(D, ref, bound, f"D with {nb} bytes")


# --------------------------------------------------------------------------------- blocks ----

@pytest.mark.parametrize("K", [1, 7, 8, 9, 63, 64, 65, 128, 136, 200, 256, 264, 320, 520, 576])
@pytest.mark.parametrize("ta,tb", [(0, 1), (0, 0), (1, 1), (1, 0)])
@pytest.mark.parametrize("M,N", [(72, 136), (65, 67), (33, 3), (40, 9)])
def test_small_blocks_every_stage_count(M, N, K, ta, tb):
    """64-wide blocks: the ring where rows are whole 16-byte chunks, else through registers; lines
    shorter than a chunk element by element."""
    say(f"small blocks {M}x{N}x{K} ta={ta} tb={tb}")
    a, b, A, B = operands(M + K, M, N, K, ta, tb, "f16")
    res = rand(4, (M, N), "f16")
    D = tg.gemm_ep(a, b, residual=res, trans_a=ta, trans_b=tb)
    ref, _, bound, _ = ol.product(A, B, residual=host(res), out="f16")
    check(D, ref, bound, "D")


@pytest.mark.parametrize("M,N,K", [(64, 64, 4096), (70, 100, 2120), (200, 72, 5000), (65, 65, 3001), (130, 264, 2057)])
@pytest.mark.parametrize("ta,tb", [(0, 1), (1, 0)])
def test_small_blocks_in_parts(M, N, K, ta, tb):
    say(f"small blocks in parts {M}x{N}x{K} ta={ta} tb={tb}")
    a, b, A, B = operands(M + K, M, N, K, ta, tb, "bf16")
    p = tg.tile_gemm_ep_plan(a, b, torch.empty(M, N, dtype=T["bf16"], device=dev()), M, N, K, ta, tb, tg.TG_BF16, tg.TG_BF16,
                             tg.TG_BF16, workspace=torch.empty(tg.tile_gemm_ep_workspace(M, N, K, ta, tb, tg.TG_BF16),
                                                               dtype=torch.uint8, device=dev()))
    assert p.splits > 1
    D = tg.gemm_ep(a, b, act="gelu", trans_a=ta, trans_b=tb)
    ref, _, bound, _ = ol.product(A, B, "gelu")
    check(D, ref, bound, "D")


def some_rows(M):
    return np.unique(np.concatenate([np.arange(3), np.arange(M - 3, M), np.random.default_rng(M).integers(0, M, 40)]))


@pytest.mark.parametrize("M,N,K,ta,tb", [
    (2048, 1544, 200, 0, 1), (1536, 2048, 72, 0, 0), (2000, 2056, 320, 1, 0), (2048, 1600, 600, 1, 1),   # 128-wide, ring
    (2056, 3000, 136, 0, 1), (3000, 2304, 192, 1, 0),                                                    # 128-wide, two a CU
    (200, 4000, 9000, 0, 1), (264, 4104, 8200, 1, 0),                                                    # 128-wide, ring, parts
    (2001, 1999, 201, 0, 1), (2001, 1999, 201, 0, 0), (1999, 2001, 135, 1, 0),                           # 128-wide, staged
    (4096, 2048, 6208, 0, 0), (3848, 2048, 6144, 1, 1)])                                                 # 256-wide, two parts
def test_large_blocks(M, N, K, ta, tb):
    say(f"large blocks {M}x{N}x{K} ta={ta} tb={tb}")
    a, b, A, B = operands(M, M, N, K, ta, tb, "bf16")
    bias, res = rand(5, (N,), "f32"), rand(6, (M, N), "bf16")
    D, Z = tg.gemm_ep(a, b, bias=bias, act="gelu_tanh", residual=res, trans_a=ta, trans_b=tb, keep_z=True)
    r = some_rows(M)
    ref, zref, bound, zbound = ol.product(A[r], B, "gelu_tanh", host(bias), host(res)[r])
    check(Z[torch.from_numpy(r).to(dev())], zref, zbound, "Z")
    check(D[torch.from_numpy(r).to(dev())], ref, bound, "D")
    assert bool(torch.isfinite(D).all())


@pytest.mark.parametrize("M,N,K", [(2048, 2048, 384), (2048, 2050, 201), (2304, 3000, 256), (300, 520, 4224), (4096, 4352, 384), (300, 4000, 16384)])
def test_large_blocks_fp8(M, N, K):
    say(f"large blocks fp8 {M}x{N}x{K}")
    a, b = rand(M, (M, K), "e4m3", 4.0), rand(N, (N, K), "e5m2", 4.0)
    rs, cs, res = torch.rand(M, device=dev()) * 0.02, torch.rand(N, device=dev()) * 0.02, rand(6, (M, N), "bf16")
    D = tg.gemm_ep(a, b, row_scale=rs, col_scale=cs, residual=res, act="relu")
    r = some_rows(M)
    ref, _, bound, _ = ol.product(host(a)[r], host(b).T, "relu", residual=host(res)[r], row_scale=host(rs)[r], col_scale=host(cs),
                                  eight=True)
    check(D[torch.from_numpy(r).to(dev())], ref, bound, "D")


@pytest.mark.parametrize("tb", [0, 1])
@pytest.mark.parametrize("ta", [0, 1])
def test_staged_edges_read_nothing_outside_the_operand(ta, tb):
    """Operands that end with their buffer, NaN right before them and in the gaps behind every row."""
    say(f"staged edges ta={ta} tb={tb}")
    M, N, K = 77, 83, 205
    a, b, A, B = operands(9, M, N, K, ta, tb, "bf16")

    def tight(t):
        rows, cols = t.shape
        buf = torch.full((5 + rows * (cols + 3),), float("nan"), dtype=t.dtype, device=dev())
        v = buf[-((rows - 1) * (cols + 3) + cols):].as_strided((rows, cols), (cols + 3, 1))
        v.copy_(t)
        return v
    D = tg.gemm_ep(tight(a), tight(b), trans_a=ta, trans_b=tb)
    ref, _, bound, _ = ol.product(A, B)
    check(D, ref, bound, "D")


# -------------------------------------------------------------------- activation gradient ----

@pytest.mark.parametrize("M", [1, 31, 33, 255, 256, 257, 700, 3000])
@pytest.mark.parametrize("N", [1, 7, 8, 9, 63, 64, 65, 520])
def test_activation_gradient_and_bias(M, N):
    say(f"activation gradient {M}x{N}")
    K = 8
    a, b, A, B = operands(M + N, M, N, K, 0, 1, "bf16")
    dy, z = rand(8, (M, N), "bf16"), rand(9, (M, N), "bf16", 2.0)
    for act in ("gelu", "none"):
        dz, _, _, dbias = tg.gemm_ep_backward(dy, a, b, Z=z, act=act, need_dA=False, need_dB=False)
        ref, bound, sref, sbound = ol.act_backward(host(dy), host(z), act, "bf16")
        check(dz, ref, bound, "dZ")
        check(dbias, sref, sbound, "dbias")


def test_gradients_against_differences():
    """Directional differences of the forward call itself, in fp32 results: the loss is linear in the
    step up to its curvature, and the products' own rounding is counted."""
    say("gradients against differences")
    M, N, K, bf = 40, 72, 64, T["bf16"]
    g = torch.Generator(device="cuda").manual_seed(3)
    def randn(*s):
        return torch.randn(s, generator=g, device=dev())
    A, B, bias, dY = randn(M, K).to(bf), (randn(N, K) / 8).to(bf), randn(N), randn(M, N).to(bf)
    Z = tg.gemm_ep(A, B, bias=bias, out_dtype=torch.float32)
    dZ, dA, dB, dbias = tg.gemm_ep_backward(dY, A, B, Z=Z.to(bf), act="silu")

    def loss(a, b, c):
        return float((dY.double() * tg.gemm_ep(a, b, bias=c, act="silu", out_dtype=torch.float32).double()).sum())
    h = 2.0 ** -4
    # steps that are exact in bf16: whole units of h on a subset of entries
    for x, grad, at in ((A, dA, 0), (B, dB, 1), (bias, dbias, 2)):
        pick = torch.rand(x.shape, generator=g, device=dev()) < 0.05
        args = [A, B, bias]
        if x.dtype == bf:   # entries of magnitude below 4 keep multiples of 2^-6 exactly
            base = (x.float() * 64).round().clamp(-255, 255).div(64).to(bf)
            args[at] = base
            Zb = tg.gemm_ep(args[0], args[1], bias=args[2], out_dtype=torch.float32)
            grad = tg.gemm_ep_backward(dY, args[0], args[1], Z=Zb.to(bf), act="silu")[1 + at]
        up, down = list(args), list(args)
        step = pick.to(args[at].dtype) * h
        up[at], down[at] = args[at] + step, args[at] - step
        diff = (loss(*up) - loss(*down)) / (2 * h)
        want = float((grad.double() * pick.double()).sum())
        # bf16 rounding of Z (2^-8 of |Z| into the slope, at most 0.5 of curvature), dZ and the result, as
        # independent errors of the summed entries, and h^2/6 of the third derivative (at most 0.5)
        terms = float((grad.double().abs() * pick.double()).sum())
        assert abs(diff - want) <= 3 * 2.0 ** -8 * terms + 0.05 * terms * h * h * 64 + 1e-3, at


# ----------------------------------------------------------------------------------- norm ----

@pytest.mark.parametrize("cols", [1025, 1536, 2049, 3583, 4095, 4104, 7000, 8191, 8193, 12001, 16383])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_wave_counts(cols, dtype):
    say(f"norm waves cols={cols} {dtype}")
    rows = 5
    X, R, W = rand(cols, (rows, cols), dtype, 2.0), rand(cols + 1, (rows, cols), dtype), rand(cols + 2, (cols,), dtype)
    check_norm(tg.rms_norm(X, W, 1e-5, residual=R), X, R, W, 1e-5, dtype, None, None)
    check_norm(tg.rms_norm(X, W, 1e-5, residual=R, scales="row"), X, R, W, 1e-5, dtype, "e4m3", "row")


@pytest.mark.parametrize("rows", [1, 257, 1100])
@pytest.mark.parametrize("cols", [509, 1030, 2049, 4100, 8189])
def test_norm_backward_in_place_over_the_stream(rows, cols):
    """dX over dH: the columns two chunks cover are written once, after both have read them."""
    say(f"norm backward in place rows={rows} cols={cols}")
    H, dY, dH = (rand(i, (rows, cols), "bf16") for i in range(3))
    W = rand(4, (cols,), "bf16")
    rstd = torch.rsqrt(H.float().square().mean(dim=1) + 1e-5)
    ref, bound, wref, wbound = ol.norm_backward(host(dY), host(H), host(W), host(rstd), host(dH), "bf16")
    bf = tg.TG_BF16
    ws = torch.full((tg.tile_rmsnorm_bwd_workspace(rows, cols, bf),), 255, dtype=torch.uint8, device=dev())
    w = torch.empty(cols, device=dev())
    tg.tile_rmsnorm_bwd(dY, H, W, rstd, dH, dH, w, rows, cols, bf, bf, workspace=ws if ws.numel() else None)
    check(dH, ref, bound, "dX")
    check(w, wref, wbound, "dw")
