"""Wide blocks with fp32 results: scales, bias, activation, residual (also in place) and Z, on every block
kernel.  Bounds are oracle/layer.py's."""

import pytest
import torch

import tile_level_gemm_amd as tg
from oracle import layer as ol

from .gpu_util import say
from .test_gpu_layer import check, dev, host, operands, rand, wide
from .test_gpu_layer_kernels import some_rows

pytestmark = pytest.mark.gpu


def run(a, b, A, B, M, N, K, ta, tb, kernel, bs, splits, eight):
    t = tg.TORCH_DTYPES[a.dtype], tg.TORCH_DTYPES[b.dtype]
    lda, ldb = a.stride(0), b.stride(0)
    bias, res = rand(5, (N,), "bf16"), rand(6, (M, N), "f32")
    rs, cs = torch.rand(M, device=dev()) * 0.5 + 0.25, torch.rand(N, device=dev()) * 0.5 + 0.25
    nb = tg.tile_gemm_ep_workspace(M, N, K, ta, tb, t[0])
    ws = torch.full((max(nb, 16),), 255, dtype=torch.uint8, device=dev())
    d, dw = wide(torch.zeros(M, N, device=dev()), 3, 2, 77.0)
    z, zw = wide(torch.zeros(M, N, device=dev()), 1, 4, 55.0)
    kw = dict(lda=lda, ldb=ldb, ldd=d.stride(0), Z=z, ld_z=z.stride(0), row_scale=rs, col_scale=cs, bias=bias,
              act=tg.TG_ACT_SILU, workspace=ws)
    p = tg.tile_gemm_ep_plan(a, b, d, M, N, K, ta, tb, *t, tg.TG_F32, residual=res, **kw)
    assert (p.kernel, p.block_m, p.splits) == (kernel, bs, splits)
    tg.tile_gemm_ep(a, b, d, M, N, K, ta, tb, *t, tg.TG_F32, residual=res, **kw)
    r = some_rows(M)
    at = torch.from_numpy(r).to(dev())
    ref, zref, bound, zbound = ol.product(A[r], B, "silu", host(bias), host(res[at]), host(rs)[r], host(cs), "f32", eight)
    check(d[at], ref, bound, "D")
    check(z[at], zref, zbound, "Z")
    assert bool(torch.isfinite(d).all()) and bool(torch.isfinite(z).all())
    for w, before, fill in ((dw, 3, 77.0), (zw, 1, 55.0)):
        assert bool((w[:, :before] == fill).all()) and bool((w[:, before + N:] == fill).all())
    # in place: the residual is D itself
    d2, _ = wide(res, 3, 2, 77.0)
    tg.tile_gemm_ep(a, b, d2, M, N, K, ta, tb, *t, tg.TG_F32, residual=d2, ld_residual=d2.stride(0), **kw)
    assert torch.equal(d2, d)


DIRECT, STAGED = tg.TG_EP_DIRECT, tg.TG_EP_STAGED


@pytest.mark.parametrize("M,N,K,ta,tb,kernel,bs,splits", [
    (4104, 4352, 200, 0, 1, DIRECT, 256, 1), (4096, 4112, 136, 1, 0, DIRECT, 256, 1), (4088, 4104, 64, 0, 0, DIRECT, 256, 1),
    (4096, 2048, 6208, 0, 1, DIRECT, 256, 2),
    (2056, 3000, 136, 0, 1, DIRECT, 128, 1), (2000, 2056, 320, 1, 0, DIRECT, 128, 1), (264, 4104, 8200, 1, 1, DIRECT, 128, 2),
    (2001, 1999, 201, 0, 1, STAGED, 128, 1), (1999, 2001, 135, 1, 0, STAGED, 128, 1), (2001, 2003, 77, 0, 0, STAGED, 128, 1)])
def test_wide_blocks_with_fp32_results(M, N, K, ta, tb, kernel, bs, splits):
    say(f"fp32 results {M}x{N}x{K} ta={ta} tb={tb}")
    a, b, A, B = operands(M + K, M, N, K, ta, tb, "bf16")
    run(a, b, A, B, M, N, K, ta, tb, kernel, bs, splits, False)


@pytest.mark.parametrize("M,N,K,kernel,bs,splits", [
    (4096, 4352, 384, DIRECT, 256, 1), (2304, 3000, 256, DIRECT, 128, 1), (2048, 2048, 400, DIRECT, 128, 1),
    (2048, 2050, 201, STAGED, 128, 1)])
def test_wide_fp8_blocks_with_fp32_results(M, N, K, kernel, bs, splits):
    say(f"fp32 results fp8 {M}x{N}x{K}")
    a, b = rand(M, (M, K), "e4m3", 4.0), rand(N, (N, K), "e5m2", 4.0)
    run(a, b, host(a), host(b).T, M, N, K, 0, 1, kernel, bs, splits, True)
