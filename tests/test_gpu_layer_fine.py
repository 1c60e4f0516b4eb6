"""The 256-wide blocks on 16-row matrix instructions: every length of the K loop's tail, every orientation, edges
and parts, against float64 products on the GPU (the bounds are oracle/layer.py's, evaluated there)."""

import pytest
import torch

import tile_level_gemm_amd as tg
from oracle import layer as ol

from .gpu_util import say
from .test_gpu_layer import T, dev
from .test_gpu_layer_i8 import ints

pytestmark = pytest.mark.gpu


def randn(seed, *shape, dtype, scale=1.0):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=dev()) * scale).to(T[dtype])


def within(got, ref, err, dtype, what):
    """err: of the fp32 value, before its rounding to `dtype`."""
    h = ol.HALF_STEP[dtype]
    off = (got.double() - ref).abs() - (err * (1 + h) + h * ref.abs() + ol.TINY[dtype])
    assert bool((off <= 0).all()), f"{what}: {int((off > 0).sum())} outside"   # NaN is outside too


def sums(A, B):
    """A·B and the error of its fp32 sum."""
    return A @ B, (A.shape[1] + 8) * 2 * ol.U32 * (A.abs() @ B.abs())


def silu(z):
    return z * torch.sigmoid(z)


def gated_check(a, b, tb, dtype, D, Z):
    N = D.shape[1]
    z, err = sums(a.double(), b.double().t() if tb else b.double())
    within(Z, z, err, dtype, "Z")
    g, u, ge, ue = z[:, :N], z[:, N:], err[:, :N], err[:, N:]
    ae = 1.13 * ge + 16 * ol.U32 * g.abs() + 2.0 ** -20 * silu(g).abs()
    within(D, silu(g) * u, ae * u.abs() + silu(g).abs() * ue + ae * ue + ol.U32 * (silu(g) * u).abs(), dtype, "D")


@pytest.mark.parametrize("K", [8, 64, 72, 128, 184, 256, 320, 376, 384, 392, 448, 520, 768, 840])
@pytest.mark.parametrize("tb,dtype", [(1, "bf16"), (0, "f16")])
def test_gated_k_loop(K, tb, dtype):
    """One to fourteen stages: every tail of the loop's six, partial last stages."""
    say(f"gated fine K={K} tb={tb} {dtype}")
    M, N = 4096, 2048
    a, b = randn(K, M, K, dtype=dtype), randn(K + 1, *((2 * N, K) if tb else (K, 2 * N)), dtype=dtype, scale=0.25)
    t = tg.TORCH_DTYPES[a.dtype]
    assert tg.tile_gemm_gated_plan(a, b, a.data_ptr() + (1 << 40), M, N, K, tb, t, t, t).block_m == 256
    D, Z = tg.gemm_gated(a, b, trans_b=tb, keep_z=True)
    gated_check(a, b, tb, dtype, D, Z)


@pytest.mark.parametrize("M,N,K,tb,dtype", [(4097, 2049, 200, 1, "bf16"), (4100, 2056, 129, 0, "bf16"), (3841, 2048, 72, 1, "f16"),
                                            (4352, 1928, 264, 0, "f16")])
def test_gated_edges(M, N, K, tb, dtype):
    """Blocks that M and N end in; rows and columns far apart."""
    say(f"gated fine edges {M}x{N}x{K} tb={tb} {dtype}")
    a, b = randn(1, M, K, dtype=dtype), randn(2, *((2 * N, K) if tb else (K, 2 * N)), dtype=dtype, scale=0.25)
    D, Z = tg.gemm_gated(a, b, trans_b=tb, keep_z=True)
    gated_check(a, b, tb, dtype, D, Z)


@pytest.mark.parametrize("K", [16, 128, 144, 256, 384, 400, 640, 768, 896, 1040, 1664])
def test_integer_k_loop(K):
    say(f"i8 fine K={K}")
    M, N = 4000, 4100
    a, b = ints(K, (M, K)), ints(K + 1, (N, K))
    assert tg.tile_gemm_ep_plan(a, b, a.data_ptr() + (1 << 40), M, N, K, 0, 1, tg.TG_I8, tg.TG_I8, tg.TG_F32).block_m == 256
    D = tg.gemm_ep(a, b, out_dtype=torch.float32)
    assert torch.equal(D, (a.double() @ b.double().t()).float())


def test_integer_parts():
    """Half the chip's worth of blocks and a long sum: two parts, joined exactly."""
    say("i8 fine parts")
    M, N, K = 4096, 2048, 12304
    a, b = ints(1, (M, K)), ints(2, (N, K))
    ws = torch.empty(tg.tile_gemm_ep_workspace(M, N, K, 0, 1, tg.TG_I8), dtype=torch.uint8, device=dev())
    D = torch.empty(M, N, device=dev())
    p = tg.tile_gemm_ep_plan(a, b, D, M, N, K, 0, 1, tg.TG_I8, tg.TG_I8, tg.TG_F32, workspace=ws)
    assert p.block_m == 256 and p.splits == 2
    assert torch.equal(tg.gemm_ep(a, b, out_dtype=torch.float32), (a.double() @ b.double().t()).float())


@pytest.mark.parametrize("M,N,K,tb", [(4104, 264, 4104, 1), (4104, 264, 4104, 0), (1001, 2056, 4104, 1), (1001, 2056, 4104, 0),
                                      (4096, 3080, 2048, 1), (4096, 3080, 2048, 0)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_gradients(M, N, K, tb, dtype):
    """dA (dZ by the weights of either orientation) and dB (both operands along the tokens, an odd number of
    them) in 256-wide blocks; two parts of dA."""
    say(f"gated gradients fine {M}x{N}x{K} tb={tb} {dtype}")
    a, b = randn(1, M, K, dtype=dtype), randn(2, *((2 * N, K) if tb else (K, 2 * N)), dtype=dtype, scale=0.25)
    dy, z = randn(3, M, N, dtype=dtype, scale=0.1), randn(4, M, 2 * N, dtype=dtype)
    dz, da, db, _ = tg.gemm_gated_backward(dy, a, b, z, trans_b=tb)
    G, B = dz.double(), b.double() if tb else b.double().t()   # B [2N][K]
    within(da, *sums(G, B), dtype, "dA")
    within(db if tb else db.t(), *sums(G.t(), a.double()), dtype, "dB")


def test_two_calls_at_once():
    """Two streams' products do not meet: each has its own results and workspace."""
    say("gated fine two streams")
    M, N, K = 4096, 2048, 512
    ab = [(randn(i, M, K, dtype="bf16"), randn(i + 9, 2 * N, K, dtype="bf16", scale=0.25)) for i in range(2)]
    want = [tg.gemm_gated(a, b) for a, b in ab]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i in range(2):
            got[i].append(tg.gemm_gated(*ab[i], stream=ss[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i]) for i in range(2) for g in got[i])
