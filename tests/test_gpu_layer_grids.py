"""Layer operators past 2^32 threads a grid dimension and past 2^16 workgroups in y: many short rows, very long
rows.  Sampled rows and columns against float64."""

import numpy as np
import pytest
import torch

import tile_level_gemm_amd as tg
from oracle import layer as ol

from .gpu_util import say
from .test_gpu_layer import T, check, check_norm, dev, host

pytestmark = pytest.mark.gpu


def filled(seed, shape, dtype, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=T[dtype], device=dev()).normal_(0.0, scale, generator=g)


def some(n):
    """The first and last of n, those around powers of two, and others."""
    edges = [2 ** k + d for k in range(10, 31) for d in (-1, 0, 1)]
    r = np.concatenate([np.arange(40), np.arange(n - 40, n), edges, np.random.default_rng(n).integers(0, n, 400)])
    return torch.from_numpy(np.unique(r[(r >= 0) & (r < n)])).to(dev())


@pytest.mark.parametrize("rows,cols", [((1 << 22) + 3, 4), ((1 << 26) + 5, 8)])
def test_norm_of_many_short_rows(rows, cols):
    say(f"norm rows={rows} cols={cols}")
    X, R, W = filled(1, (rows, cols), "f16", 3.0), filled(2, (rows, cols), "f16"), filled(3, (cols,), "f16")
    pick = some(rows)
    r = tg.rms_norm(X, W, residual=R)
    part = tg.Norm(r.y[pick], None, r.rstd[pick], r.h[pick])
    check_norm(part, X[pick], R[pick], W, 1e-5, "f16", None, None)
    assert bool((r.rstd > 0).all())
    r8 = tg.rms_norm(X, W, residual=R, scales="row")
    part = tg.Norm(r8.y.view(torch.uint8)[pick].view(T["e4m3"]), r8.scale[pick], r8.rstd[pick], r8.h[pick])
    check_norm(part, X[pick], R[pick], W, 1e-5, "f16", "e4m3", "row")
    assert torch.equal(r8.rstd, r.rstd)


@pytest.mark.parametrize("rows,cols", [((1 << 22) + 3, 4), ((1 << 26) + 5, 8)])
def test_norm_backward_of_many_short_rows(rows, cols):
    say(f"norm backward rows={rows} cols={cols}")
    H, W, dY = filled(1, (rows, cols), "f16", 3.0), filled(2, (cols,), "f16"), filled(3, (rows, cols), "f16")
    rstd = torch.rsqrt(H.float().square().mean(dim=1) + 1e-5)
    dX, dw = tg.rms_norm_backward(dY, H, W, rstd)
    pick = some(rows)
    ref, bound, _, _ = ol.norm_backward(host(dY[pick]), host(H[pick]), host(W), host(rstd[pick]), None, "f16")
    check(dX[pick], ref, bound, "dX")
    terms = torch.zeros(2, cols, dtype=torch.float64, device=dev())
    for at in range(0, rows, 1 << 24):
        s = slice(at, at + (1 << 24))
        t = dY[s].double() * (H[s].double() * rstd[s, None].double())
        terms += torch.stack([t.sum(dim=0), t.abs().sum(dim=0)])
    # at most 512 workgroups share the rows, each adds its rows in turn, then up to 512 shares: 2^-24 of
    # the magnitudes for every addition on the way and three products
    adds = (rows + 511) // 512 + 512 + 3
    check(dw, host_64(terms[0]), host_64(terms[1]) * adds * 2.0 ** -24, "dw")


def host_64(t):
    return t.cpu().numpy()


@pytest.mark.parametrize("cols", [(1 << 27) + 4099])
def test_norm_of_a_very_long_row(cols):
    """More panels of 2048 columns than grid.y holds."""
    say(f"norm cols={cols}")
    X, W, dY = filled(1, (1, cols), "bf16", 3.0), filled(2, (cols,), "bf16"), filled(3, (1, cols), "bf16")
    r = tg.rms_norm(X, W)
    # 1024 threads add cols / 1024 squares each, one after the other: 2^-24 of the sum for each addition,
    # half of that in the root
    rel = (cols / 1024 + 32) * 2.0 ** -25
    want = float(torch.rsqrt(X.double().square().mean() + 1e-5))
    rstd = float(r.rstd)
    assert abs(rstd - want) <= rel * want
    pick = some(cols)
    x, w, dy = host(X[0, pick]), host(W[pick]), host(dY[0, pick])
    Y = x * rstd * w
    check(r.y[0, pick], Y, np.abs(Y) * (2.0 ** -8 + 4 * 2.0 ** -24) + ol.TINY["bf16"], "Y")
    dX, dw = tg.rms_norm_backward(dY, X, W, r.rstd)
    xh = X.double() * rstd
    t = dY.double() * W.double() * xh
    c, cerr = float(t.mean()), float(t.abs().mean()) * 2 * rel
    g = dy * w
    xh = x * rstd
    ref = rstd * (g - xh * c)
    err = rstd * (6 * 2.0 ** -24 * (np.abs(g) + np.abs(xh * c)) + np.abs(xh) * cerr)
    check(dX[0, pick], ref, err * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref) + ol.TINY["bf16"], "dX")
    check(dw[pick], dy * xh, 4 * 2.0 ** -24 * np.abs(dy * xh), "dw")


@pytest.mark.parametrize("cols", [(1 << 27) + 4099])
def test_norm_backward_sums_shares_of_very_long_rows(cols):
    """Two rows, a share of dw each."""
    say(f"norm backward shares cols={cols}")
    X, W, dY = filled(1, (2, cols), "bf16", 3.0), filled(2, (cols,), "bf16"), filled(3, (2, cols), "bf16")
    rstd = torch.tensor([0.25, 0.5], device=dev())
    _, dw = tg.rms_norm_backward(dY, X, W, rstd)
    pick = some(cols)
    t = host(dY[:, pick]) * host(X[:, pick]) * host(rstd)[:, None]
    check(dw[pick], t.sum(axis=0), 6 * 2.0 ** -24 * np.abs(t).sum(axis=0), "dw")


@pytest.mark.parametrize("M", [1, 2, 300])
@pytest.mark.parametrize("act", ["none", "relu"])
def test_bias_gradient_of_very_many_columns(M, act):
    """300 rows: narrower, but in two groups of rows."""
    N = (1 << 28) + 1033 if M < 300 else (1 << 21) - 7
    say(f"bias gradient {M}x{N} {act}")
    bf = T["bf16"]
    dY, Z = filled(1, (M, N), "bf16"), filled(2, (M, N), "bf16")
    A, B = torch.empty(M, 1, dtype=bf, device=dev()), torch.empty(N, 1, dtype=bf, device=dev())
    dZ, _, _, dbias = tg.gemm_ep_backward(dY, A, B, Z=Z, act=act, need_dA=False, need_dB=False)
    pick = some(N)
    ref, bound, sref, sbound = ol.act_backward(host(dY[:, pick]), host(Z[:, pick]), act, "bf16")
    check(dZ[:, pick], ref, bound, "dZ")
    check(dbias[pick], sref, sbound, "dbias")
    if M == 1:   # every column: one term each
        assert torch.equal(dbias, dY[0].float() if act == "none" else torch.where(Z[0] > 0, dY[0], 0).float())


def test_epilogue_of_a_zero_product_past_two_to_the_35_results():
    M, N = 1 << 18, (1 << 17) + 8
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 69 GB for the result")
    say(f"zero product {M}x{N}")
    bf = T["bf16"]
    bias = filled(1, (N,), "bf16")
    D = tg.gemm_ep(torch.empty(M, 0, dtype=bf, device=dev()), torch.empty(N, 0, dtype=bf, device=dev()), bias=bias, act="relu")
    want = torch.relu(bias)
    for at in range(0, M, 1 << 14):
        assert bool((D[at:at + (1 << 14)] == want).all()), at
    del D
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows", [1, 3, 5])
@pytest.mark.parametrize("cols", [1, 7, 16385])
def test_norm_backward_with_the_least_documented_workspace(rows, cols):
    """4 bytes a row, whatever the alignment of the shares behind them."""
    say(f"norm backward least workspace rows={rows} cols={cols}")
    H, W, dY = filled(1, (rows, cols), "bf16", 3.0), filled(2, (cols,), "bf16"), filled(3, (rows, cols), "bf16")
    rstd = torch.rsqrt(H.float().square().mean(dim=1) + 1e-5)
    dX, dw = torch.empty_like(H), torch.empty(cols, device=dev())
    ws = torch.full((64,), 255, dtype=torch.uint8, device=dev())
    bf = tg.TG_BF16
    with pytest.raises(tg.TileError):
        tg.tile_rmsnorm_bwd(dY, H, W, rstd, None, dX, dw, rows, cols, bf, bf, workspace=ws, workspace_bytes=4 * rows - 1)
    tg.tile_rmsnorm_bwd(dY, H, W, rstd, None, dX, dw, rows, cols, bf, bf, workspace=ws, workspace_bytes=4 * rows)
    ref, bound, wref, wbound = ol.norm_backward(host(dY), host(H), host(W), host(rstd), None, "bf16")
    check(dX, ref, bound, "dX")
    check(dw, wref, wbound, "dw")
    assert bool((ws[4 * rows:] == 255).all())
