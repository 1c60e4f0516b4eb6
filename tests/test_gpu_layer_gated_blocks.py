"""Every block kernel of the gated product by name of its plan: 8-bit operands in 256- and 128-wide blocks, 16-bit
ones in 128-wide blocks and in 256-wide ones with an edge of rows, whole and in parts, against float64 products on
the GPU (the bounds are oracle/layer.py's, evaluated there)."""

import pytest
import torch

import tile_level_gemm_amd as tg
from oracle import layer as ol

from .gpu_util import say
from .test_gpu_layer import T, dev
from .test_gpu_layer_fine import gated_check, randn, silu, within
from .test_gpu_layer_i8 import ints

pytestmark = pytest.mark.gpu

PAIRS = [("i8", "i8"), ("e4m3", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")]
DIRECT, STAGED = tg.TG_EP_DIRECT, tg.TG_EP_STAGED

# M, N, K, kernel, block, parts.  Direct 128-wide blocks: up to 256 of them run in the ring of four stages, more in
# two stages, two workgroups a CU.  Stages are 128 bytes of K.
EIGHT = [(4097, 2049, 16, DIRECT, 256, 1), (4097, 2049, 144, DIRECT, 256, 1), (4097, 2049, 272, DIRECT, 256, 1),
         (3841, 2176, 400, DIRECT, 256, 1), (4097, 2049, 1040, DIRECT, 256, 1), (4096, 1024, 12304, DIRECT, 256, 2),
         (2100, 1100, 16, DIRECT, 128, 1), (2100, 1100, 272, DIRECT, 128, 1), (2049, 1153, 528, DIRECT, 128, 1),
         (1900, 1000, 144, DIRECT, 128, 1), (1921, 961, 656, DIRECT, 128, 1), (200, 1000, 32784, DIRECT, 128, 8),
         (1900, 1000, 201, STAGED, 128, 1), (2100, 1101, 129, STAGED, 128, 1), (1921, 961, 515, STAGED, 128, 1)]
SIXTEEN = [(4100, 2056, 136, DIRECT, 256, 1), (3848, 2184, 72, DIRECT, 256, 1),
           (2100, 1104, 8, DIRECT, 128, 1), (2100, 1104, 136, DIRECT, 128, 1), (2050, 1160, 328, DIRECT, 128, 1),
           (1900, 1000, 72, DIRECT, 128, 1), (1921, 968, 392, DIRECT, 128, 1), (200, 1000, 16392, DIRECT, 128, 8),
           (1900, 1000, 101, STAGED, 128, 1), (2100, 1101, 65, STAGED, 128, 1), (1921, 961, 259, STAGED, 128, 1)]


def planned(a, b, M, N, K, tb, out, kernel, block, parts):
    ta, tw, to = (tg.TORCH_DTYPES[t] for t in (a.dtype, b.dtype, T[out]))
    ws = torch.empty(max(16, tg.tile_gemm_gated_workspace(M, N, K, tb, ta)), dtype=torch.uint8, device=dev())
    D = torch.empty(M, N, dtype=T[out], device=dev())
    p = tg.tile_gemm_gated_plan(a, b, D, M, N, K, tb, ta, tw, to, workspace=ws)
    assert (p.kernel, p.block_m, p.splits) == (kernel, block, parts)


@pytest.mark.parametrize("M,N,K,kernel,block,parts", EIGHT)
@pytest.mark.parametrize("ta,tw", PAIRS)
def test_eight_bits(ta, tw, M, N, K, kernel, block, parts):
    say(f"gated blocks {ta} {tw} {M}x{N}x{K}")
    whole = ta == "i8"
    a = ints(K, (M, K)) if whole else randn(K, M, K, dtype=ta, scale=4.0)
    b = ints(K + 1, (2 * N, K)) if whole else randn(K + 1, 2 * N, K, dtype=tw, scale=4.0)
    planned(a, b, M, N, K, 1, "bf16", kernel, block, parts)
    g = torch.Generator(device=dev()).manual_seed(M)
    small = 1.0 / (5000 if whole else 16) / K ** 0.5   # results of order one
    rs, cs = (torch.rand(n, generator=g, device=dev()) * s + 0.1 * s for n, s in ((M, small), (2 * N, 1.0)))
    bias = torch.randn(2 * N, generator=g, device=dev())
    D, Z = tg.gemm_gated(a, b, bias=bias, row_scale=rs, col_scale=cs, keep_z=True)
    A, B = a.double(), b.double().t()
    P, mag = A @ B, A.abs() @ B.abs()
    err = ol.U32 * P.abs() if whole else ((K + 8) * 2 * ol.U32 + 2.0 ** -10) * mag
    scale = rs.double()[:, None] * cs.double()
    z = P * scale
    err = err * scale + 3 * ol.U32 * z.abs()
    z = z + bias.double()
    err = err + ol.U32 * (z.abs() + err)
    within(Z, z, err, "bf16", "Z")
    u, ge, ue, s = z[:, N:], err[:, :N], err[:, N:], silu(z[:, :N])
    ae = 1.13 * ge + 16 * ol.U32 * z[:, :N].abs() + 2.0 ** -20 * s.abs()
    within(D, s * u, ae * u.abs() + s.abs() * ue + ae * ue + ol.U32 * (s * u).abs(), "bf16", "D")
    assert torch.equal(tg.gemm_gated(a, b, bias=bias, row_scale=rs, col_scale=cs), D)


@pytest.mark.parametrize("M,N,K,kernel,block,parts", SIXTEEN)
@pytest.mark.parametrize("tb", [1, 0])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_sixteen_bits(dtype, tb, M, N, K, kernel, block, parts):
    say(f"gated blocks {dtype} tb={tb} {M}x{N}x{K}")
    a, b = randn(K, M, K, dtype=dtype), randn(K + 1, *((2 * N, K) if tb else (K, 2 * N)), dtype=dtype, scale=K ** -0.5)
    planned(a, b, M, N, K, tb, dtype, kernel, block, parts)
    D, Z = tg.gemm_gated(a, b, trans_b=tb, keep_z=True)
    gated_check(a, b, tb, dtype, D, Z)
    assert torch.equal(tg.gemm_gated(a, b, trans_b=tb), D)


def test_two_calls_with_workspaces_at_once():
    """Two streams' products in parts, and their gradients, whose workspaces hold shares of the bias's gradient and
    then parts of dA: each call has its own, and none is handed on while it is read."""
    say("gated two streams in parts")
    M, N, K, bf = 4096, 1024, 8192, tg.TG_BF16
    ops = [(randn(i, M, K, dtype="bf16"), randn(i + 9, 2 * N, K, dtype="bf16", scale=K ** -0.5), randn(i + 18, M, N, dtype="bf16"))
           for i in range(2)]
    planned(ops[0][0], ops[0][1], M, N, K, 1, "bf16", DIRECT, 256, 2)
    assert tg.tile_gemm_gated_workspace(M, N, K, 1, bf) > 0 and tg.tile_gemm_gated_bwd_workspace(M, N, K, 1, bf) > 0

    def both(i, stream=None):
        a, b, dy = ops[i]
        d, z = tg.gemm_gated(a, b, keep_z=True, stream=stream)
        return (d, z, *tg.gemm_gated_backward(dy, a, b, z, stream=stream))

    want = [both(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [(i, both(i, streams[i])) for _ in range(3) for i in range(2)]
    torch.cuda.synchronize()
    for i, results in got:
        assert all(torch.equal(g, w) for g, w in zip(results, want[i]))
