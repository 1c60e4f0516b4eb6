"""Gradients of a product with row and column scales: against the formula in float64 and against differences of
the forward call.  Bounds are oracle/layer.py's."""

import numpy as np
import pytest
import torch

import tile_level_gemm_amd as tg
from oracle import layer as ol

from .gpu_util import say
from .test_gpu_layer import T, check, dev, host, operands, rand, wide

pytestmark = pytest.mark.gpu


def scaled(dY, Z, act, rs, cs, out):
    """(dZ with the scales, its bound, dbias, its bound)"""
    dz, err, s, serr = ol.act_backward(dY, Z, act, "f32")
    scale = (rs[:, None] if rs is not None else 1.0) * (cs[None, :] if cs is not None else 1.0) * np.ones_like(dz)
    p = dz * scale
    err = err * np.abs(scale) + 3 * ol.U32 * np.abs(p)
    h = ol.HALF_STEP[out]
    return p, err * (1 + h) + h * np.abs(p) + ol.TINY[out], s, serr


@pytest.mark.parametrize("M,N,K,ta,tb", [(64, 72, 136, 0, 1), (33, 41, 57, 0, 0), (200, 520, 264, 1, 1), (1, 24, 40, 0, 1),
                                         (1000, 264, 128, 1, 0), (300, 1, 8, 0, 1), (2, 65, 3, 0, 0)])
@pytest.mark.parametrize("act", ol.ACTS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_scaled_product_backward(M, N, K, ta, tb, act, dtype):
    say(f"scaled product backward {M}x{N}x{K} ta={ta} tb={tb} {act} {dtype}")
    a, b, A, B = operands(M + K, M, N, K, ta, tb, dtype)
    dy, z = rand(8, (M, N), dtype), rand(9, (M, N), dtype, 2.0)
    rows, cols = rand(10, (M,), "f32"), rand(11, (N,), "f32")
    for rs, cs in ((rows, cols), (rows, None), (None, cols)):
        dz, da, db, dbias = tg.gemm_ep_backward(dy, a, b, Z=z, act=act, trans_a=ta, trans_b=tb, row_scale=rs, col_scale=cs)
        ref, bound, sref, sbound = scaled(host(dy), host(z), act, None if rs is None else host(rs), None if cs is None else host(cs), dtype)
        check(dz, ref, bound, "dZ")
        check(dbias, sref, sbound, "dbias")
        G = host(dz)   # the products take dZ as it is held
        ref, bound = ol.matmul_bound(G, B.T, dtype)
        check(da.t() if ta else da, ref, bound, "dA")
        ref, bound = ol.matmul_bound(A.T, G, dtype)
        check(db.t() if tb else db, ref, bound, "dB")


def test_scaled_backward_in_place_slices_and_streams():
    say("scaled product backward parts")
    M, N, K, bf = 300, 72, 40, tg.TG_BF16
    a, b, _, _ = operands(1, M, N, K, 0, 1, "bf16")
    dy, z = rand(2, (M, N), "bf16"), rand(3, (M, N), "bf16")
    rs, cs = rand(4, (M,), "f32"), rand(5, (N,), "f32")
    for act, code in (("silu", tg.TG_ACT_SILU), ("none", tg.TG_ACT_NONE)):
        want = tg.gemm_ep_backward(dy, a, b, Z=z, act=act, row_scale=rs, col_scale=cs)
        assert want[0] is not dy
        for place in range(2 if act == "silu" else 1):   # over dY, over Z
            y, zz = dy.clone(), z.clone()
            s = torch.empty(N, device=dev())
            da = torch.empty_like(a)
            tg.tile_gemm_ep_bwd(y, zz, a, b, (y, zz)[place], da, None, s, M, N, K, 0, 1, bf, code, row_scale=rs, col_scale=cs)
            assert torch.equal((y, zz)[place], want[0]) and torch.equal(da, want[1])
        dyw, zw = wide(dy, 3, 2, float("nan"))[0], wide(z, 3, 2, float("nan"))[0]
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        got = tg.gemm_ep_backward(dyw, a, b, Z=zw, act=act, row_scale=rs, col_scale=cs, stream=st)
        st.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("act", ["none", "silu"])
def test_scaled_gradients_against_differences(act):
    """Directional differences of the forward call with fp32 results, steps exact in bf16."""
    say(f"scaled gradients against differences {act}")
    M, N, K, bf = 40, 72, 64, T["bf16"]
    g = torch.Generator(device="cuda").manual_seed(3)

    def randn(*s):
        return torch.randn(s, generator=g, device=dev())

    def grid(x):   # multiples of 2^-6 below 4: exact in bf16, also after a step
        return (x * 64).round().clamp(-255, 255).div(64).to(bf)
    A, B, bias, dY = grid(randn(M, K)), grid(randn(N, K) / 8), randn(N), randn(M, N).to(bf)
    rs, cs = torch.rand(M, generator=g, device=dev()) + 0.25, torch.rand(N, generator=g, device=dev()) + 0.25

    def forward(a, b, c):
        return tg.gemm_ep(a, b, bias=c, act=act, row_scale=rs, col_scale=cs, out_dtype=torch.float32, keep_z=True)

    def loss(a, b, c):
        return float((dY.double() * forward(a, b, c)[0].double()).sum())
    Z = forward(A, B, bias)[1]
    _, dA, dB, dbias = tg.gemm_ep_backward(dY, A, B, Z=Z.to(bf), act=act, row_scale=rs, col_scale=cs)
    h = 2.0 ** -4
    for at, grad in ((0, dA), (1, dB), (2, dbias)):
        pick = torch.rand(grad.shape, generator=g, device=dev()) < 0.05
        up, down = [A, B, bias], [A, B, bias]
        step = pick.to(up[at].dtype) * h
        up[at], down[at] = up[at] + step, down[at] - step
        diff = (loss(*up) - loss(*down)) / (2 * h)
        want = float((grad.double() * pick.double()).sum())
        # each picked entry's gradient off by three bf16 roundings (Z into a slope of curvature 0.5 at most, dZ,
        # the result), and h^2/6 of the third derivative
        terms = float((grad.double().abs() * pick.double()).sum())
        assert abs(diff - want) <= 3 * 2.0 ** -8 * terms + 0.05 * terms * h * h * 64 + 1e-3, at
