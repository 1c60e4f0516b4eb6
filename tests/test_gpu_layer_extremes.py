"""Norm results where Y or the product H·w leaves the ordinary range, and 8-bit codes at their borders.
Bounds are oracle/layer.py's."""

import numpy as np
import pytest
import torch

import tile_level_gemm_amd as tg

from .gpu_util import say
from .test_gpu_layer import T, check_norm, dev, host, rand

pytestmark = pytest.mark.gpu

COLS = [5, 64, 520, 1000, 2048, 2057, 8200, 20000]   # a wave a row, workgroups, two passes


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_row_whose_result_is_infinite_gets_a_nan_scale(cols, dtype, fmt):
    """X finite, Y not: an infinite weight, or a finite one whose product overflows."""
    say(f"norm infinite result cols={cols} {dtype} {fmt}")
    X, W = rand(1, (5, cols), dtype), rand(2, (cols,), dtype)
    X[:, 3] = 4.0   # above the row's root mean square, so that 4·rstd·3e38 is past fp32
    X[1, 3] = 0.0   # 0·inf is NaN, 0·3e38 is 0
    for big in (float("inf"), 3e38):
        W[3] = big
        y = host(tg.rms_norm(X.float(), W.float(), 1e-5).y)
        r = tg.rms_norm(X, W, 1e-5, out_dtype=T[fmt], scales="row")
        s = host(r.scale)
        bad = ~np.isfinite(y).all(axis=1)
        assert bad[[0, 2, 3, 4]].any()
        assert np.array_equal(np.isnan(s), bad), (big, s)
        assert np.isnan(host(r.y)[bad]).all()


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("hx,wx", [(1e15, 1e25), (1e-18, 1e-24)])
@pytest.mark.parametrize("rows", [1, 6])
def test_row_scale_where_the_product_with_the_weight_leaves_fp32(cols, hx, wx, rows):
    """H·w overflows or loses its bits, H·rstd·w is ordinary: the scale is max|Y|/qmax all the same."""
    say(f"norm product out of range cols={cols} {hx} {wx}")
    X, W = rand(1, (rows, cols), "f32", hx), rand(2, (cols,), "f32", wx)
    for fmt in ("e4m3", "e5m2"):
        check_norm(tg.rms_norm(X, W, 0.0, out_dtype=T[fmt], scales="row"), X, None, W, 0.0, "f32", fmt, "row")


@pytest.mark.parametrize("cols", [5, 64, 1000, 2057, 4096, 20000])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_row_scaled_codes_are_the_quotient_rounded_once(cols, fmt):
    """fp32 rows: the 16-bit-free call gives the Y that the codes are made of, so every code is known."""
    say(f"norm codes cols={cols} {fmt}")
    rows = 4_000_000 // cols
    X, W = rand(cols, (rows, cols), "f32", 3.0), rand(cols + 1, (cols,), "f32")
    Y = tg.rms_norm(X, W).y
    r = tg.rms_norm(X, W, out_dtype=T[fmt], scales="row")
    want = (Y / r.scale[:, None]).to(T[fmt])
    assert torch.equal(r.y.view(torch.uint8), want.view(torch.uint8)), int((r.y.view(torch.uint8) != want.view(torch.uint8)).sum())
