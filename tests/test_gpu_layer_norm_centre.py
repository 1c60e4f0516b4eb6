"""The layer norm of rows far from zero against float64, with bounds that the mean's own size does not enter.

The mean m of n values is summed by serial chains of at most s additions a thread and a tree (10 levels), and
rounded: it is off by e, at most (s + 12) units of the rows' mean magnitude.  Deviations from it, d, are exact to half
a unit of themselves, and their mean, off by (s + 12) units of mean |d|, brings the centre back; the mean of squares
less that mean's square is the variance to (s + 14) units of mean d² + e².  So Y depends on e in no term but through
|d| <= |x - mean| + e, and e is far below the deviations in every row here."""

import numpy as np
import pytest
import torch

import tile_level_gemm_amd as tg
from oracle import layer as ol

from .gpu_util import say
from .test_gpu_layer import check, dev, host, rand
from .test_gpu_layer_norm import Q8, check_codes

pytestmark = pytest.mark.gpu


def serial(cols):
    """Additions of a thread's chain: two chunks of 8 in registers, else 8 of each 8192 columns."""
    return 16 if 8 <= cols <= 16384 else 8 * (-(-cols // 8192))


def centred(H, w, b, eps):
    """(Y, mean, rstd, bound of Y, bound of mean, bound of rstd)."""
    n, u = serial(H.shape[1]) + 14, ol.U32
    mean = H.mean(axis=1)
    d = H - mean[:, None]
    var = np.mean(d * d, axis=1)
    rstd = 1.0 / np.sqrt(var + eps)
    e = n * u * np.mean(np.abs(H), axis=1)                     # of the first mean
    near = np.mean(np.abs(d), axis=1) + e
    centre = n * u * near + 2 * u * e                          # of the mean of the deviations from it
    verr = n * u * (var + e * e) + 2 * u * near * near + 2 * e * centre + centre * centre
    rel = 0.5 * verr / (var + eps) + 4 * u
    Y = d * rstd[:, None] * w[None, :]
    err = np.abs(w)[None, :] * rstd[:, None] * (centre[:, None] + 2 * u * (np.abs(d) + e[:, None])) + (rel[:, None] + 3 * u) * np.abs(Y)
    if b is not None:
        Y = Y + b[None, :]
        err = err + u * (np.abs(Y) + err)
    return Y, mean, rstd, err, centre + u * np.abs(mean), rel * rstd


@pytest.mark.parametrize("cols", [5, 64, 520, 1000, 2057, 8192, 16384, 20000])
@pytest.mark.parametrize("shift", [100.0, 1e4, -3e5])
def test_rows_far_from_zero(cols, shift):
    """fp32 rows whose deviations are of order one about means far larger."""
    say(f"layer norm centre shift={shift} cols={cols}")
    X, W, B = rand(cols, (6, cols), "f32") + shift, rand(1, (cols,), "f32"), rand(2, (cols,), "f32")
    Y, mean, rstd, err, merr, rerr = centred(host(X), host(W), host(B), 1e-5)
    assert (err < 1e-3 * (1 + np.abs(host(W))[None, :]) * (1 + np.abs(Y))).all()   # the bound says something
    r = tg.layer_norm(X, W, B)
    check(r.rstd, rstd, rerr, "rstd")
    check(r.mean, mean, merr, "mean")
    check(r.y, Y, err + ol.HALF_STEP["f32"] * np.abs(Y) + ol.TINY["f32"], "Y")
    for fmt in ("i8", "e4m3"):
        r = tg.layer_norm(X, W, B, out_dtype=Q8[fmt], scales="row")
        s = ol.row_scale(Y, fmt)
        check(r.scale, s, err.max(axis=1) / ol.QMAX[fmt] + 4 * ol.U32 * s, "scale")
        check_codes(r.y, Y, err, host(r.scale)[:, None] * np.ones_like(Y), fmt)


@pytest.mark.parametrize("cols", [3, 72, 333, 1000, 2057, 6000, 12345, 20001])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_rows_of_one_value(cols, dtype):
    """A row of one value has no deviations: its result is the bias, however its mean is rounded."""
    say(f"layer norm of one value cols={cols} {dtype}")
    v = torch.tensor([0.1, -3.3, 100.3, 777.7, 30001.0, 60000.0], device=dev())
    X = v[:, None].expand(-1, cols).to(rand(1, (1,), dtype).dtype).contiguous()
    W, B = rand(1, (cols,), "f32"), rand(2, (cols,), "f32")
    Y, mean, rstd, err, merr, rerr = centred(host(X), host(W), host(B), 1e-5)
    r = tg.layer_norm(X, W, B)
    check(r.rstd, rstd, rerr, "rstd")
    check(r.mean, mean, merr, "mean")
    check(r.y, Y, err * 1.01 + ol.HALF_STEP[dtype] * np.abs(Y) + ol.TINY[dtype], "Y")


def test_rows_that_are_not_finite_keep_their_statistics():
    """An infinity makes the mean infinite, a NaN both; squares past fp32 make rstd 0, as documented."""
    say("layer norm centre infinite")
    for cols in (64, 1000, 3000, 20000):
        X, W = rand(1, (4, cols), "f32"), torch.ones(cols, device=dev())
        X[0, 5], X[1, 7], X[2] = float("inf"), float("nan"), X[2] * 1e30
        r = tg.layer_norm(X, W)
        m, s = host(r.mean), host(r.rstd)
        assert m[0] == np.inf and np.isnan(m[1]) and np.isfinite(m[2]) and np.isnan(s[[0, 1]]).all() and s[2] == 0
        assert np.isnan(host(r.y)[[0, 1]]).all() and not host(r.y)[2].any() and np.isfinite(host(r.y)[3]).all()
