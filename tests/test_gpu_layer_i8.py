"""Products of 8-bit integers with scales for each token and channel on the GPU, against exact sums."""

import numpy as np
import pytest
import torch

import tile_level_gemm_amd as tg
from oracle import layer as ol

from .gpu_util import say
from .test_gpu_layer import T, check, dev, host, rand, wide

pytestmark = pytest.mark.gpu

I8 = tg.TG_I8


def ints(seed, shape, low=-128, high=128):
    x = np.random.default_rng(seed).integers(low, high, size=shape, dtype=np.int64).astype(np.int8)
    return torch.from_numpy(x).to(dev())


def sums(a, b):
    """Exact sums, rounded to fp32 as the epilogue takes them."""
    return (a.cpu().numpy().astype(np.float64) @ b.cpu().numpy().astype(np.float64).T).astype(np.float32)


SIZES = [(1, 1, 1), (1, 8, 64), (3, 5, 7), (2, 300, 1000), (16, 16, 32), (17, 33, 65), (33, 130, 200), (127, 129, 130),
         (128, 128, 128), (129, 257, 64), (130, 264, 1040), (256, 256, 512), (64, 72, 4096), (300, 520, 272), (5, 7, 3001),
         (1, 4096, 2048), (20, 8200, 1024), (40, 24, 15), (1024, 520, 72)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_sums_are_exact(M, N, K):
    """Without scales an fp32 result is the exact sum rounded once, also where parts of K are joined."""
    say(f"i8 {M}x{N}x{K}")
    a, b = ints(M + K, (M, K)), ints(N + K, (N, K))
    want = sums(a, b)
    assert np.array_equal(tg.gemm_ep(a, b, out_dtype=torch.float32).cpu().numpy(), want)
    D = torch.empty((M, N), device=dev())
    tg.tile_gemm_ep(a, b, D, M, N, K, 0, 1, I8, I8, tg.TG_F32)   # no workspace: one part
    assert np.array_equal(D.cpu().numpy(), want)


@pytest.mark.parametrize("M,N,K,split", [(2304, 4112, 144, False), (2048, 2056, 1040, False), (256, 512, 16384, True),
                                         (64, 64, 16384, True), (384, 136, 10000, True), (300, 200, 20001, True), (512, 4096, 4096, False)])
def test_large_plans(M, N, K, split):
    """256-, 128- and 64-wide blocks, partial last stages, parts of K."""
    say(f"i8 large {M}x{N}x{K}")
    a, b = ints(M, (M, K)), ints(N, (N, K))
    nb = tg.tile_gemm_ep_workspace(M, N, K, 0, 1, I8)
    if split:
        ws = torch.empty(nb, dtype=torch.uint8, device=dev())
        assert tg.tile_gemm_ep_plan(a, b, torch.empty((M, N), device=dev()), M, N, K, 0, 1, I8, I8, tg.TG_F32, workspace=ws).splits > 1
    assert np.array_equal(tg.gemm_ep(a, b, out_dtype=torch.float32).cpu().numpy(), sums(a, b))


@pytest.mark.parametrize("M", [1, 33])
def test_the_longest_sum_of_the_largest_values(M):
    K = 131071
    say(f"i8 K={K} M={M}")
    a, b = torch.full((M, K), -128, dtype=torch.int8, device=dev()), torch.full((40, K), -128, dtype=torch.int8, device=dev())
    b[1] = 127
    want = sums(a, b)
    assert want[0, 0] == np.float32(2147467264)
    assert np.array_equal(tg.gemm_ep(a, b, out_dtype=torch.float32).cpu().numpy(), want)


@pytest.mark.parametrize("act", ol.ACTS)
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 40, 96), (37, 75, 130), (200, 136, 4096)])
def test_epilogue_parts(act, out, M, N, K):
    say(f"i8 epilogue {act} {out} {M}x{N}x{K}")
    a, b = ints(M, (M, K)), ints(N, (N, K))
    bias, res = rand(7, (N,), "f32" if out == "f16" else out), rand(8, (M, N), out)
    rs, cs = (torch.rand(n, device=dev()) * 0.01 + 0.002 for n in (M, N))
    for use in range(4):
        kw = dict(bias=bias if use & 1 else None, residual=res if use & 2 else None, row_scale=rs, col_scale=cs)
        D, Z = tg.gemm_ep(a, b, act=act, out_dtype=T[out], keep_z=True, **kw)
        ref, zref, bound, zbound = ol.product(a.cpu().numpy().astype(np.float64), b.cpu().numpy().astype(np.float64).T, act, out=out,
                                              ints=True, **{k: None if v is None else host(v) for k, v in kw.items()})
        check(Z, zref, zbound, f"Z use={use}")
        check(D, ref, bound, f"D use={use}")


def test_default_result_is_bfloat16():
    a, b = ints(1, (4, 32)), ints(2, (8, 32))
    assert tg.gemm_ep(a, b).dtype == torch.bfloat16


@pytest.mark.parametrize("M,N,K", [(40, 72, 144), (33, 41, 57), (1, 64, 256), (130, 264, 8192)])
@pytest.mark.parametrize("before,after", [(0, 16), (3, 5), (16, 32)])
def test_slices(M, N, K, before, after):
    """Operands as slices of wider matrices, whose other columns hold values that would show."""
    say(f"i8 slices {M}x{N}x{K} {before},{after}")
    a, b = ints(3, (M, K)), ints(4, (N, K))
    va, vb = wide(a, before, after, 127.0)[0], wide(b, before, after, 127.0)[0]
    assert np.array_equal(tg.gemm_ep(va, vb, out_dtype=torch.float32).cpu().numpy(), sums(a, b))


def test_replays_of_a_captured_product():
    say("i8 graph")
    a, b, cs = ints(5, (64, 8192)), ints(6, (64, 8192)), torch.rand(64, device=dev())
    rs = torch.rand(64, device=dev())
    want = tg.gemm_ep(a, b, row_scale=rs, col_scale=cs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tg.gemm_ep(a, b, row_scale=rs, col_scale=cs)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = tg.gemm_ep(a, b, row_scale=rs, col_scale=cs)
    for k in range(3):
        a.copy_(ints(50 + k, (64, 8192)))
        want = tg.gemm_ep(a, b, row_scale=rs, col_scale=cs)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
