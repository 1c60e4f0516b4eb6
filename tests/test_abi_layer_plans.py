"""Host-only: which kernel the product with an epilogue runs, and that its plan covers the problem."""

import pytest

import tile_level_gemm_amd as tg

A, B, D, WS = (1 << 44) * 1, (1 << 44) * 2, (1 << 44) * 3, (1 << 44) * 4
BF, E4 = tg.TG_BF16, tg.TG_FP8_E4M3


def plan(M, N, K, ta=0, tb=1, t=BF, budget=None, **kw):
    nb = tg.tile_gemm_ep_workspace(M, N, K, ta, tb, t) if budget is None else budget
    return tg.tile_gemm_ep_plan(A, B, D, M, N, K, ta, tb, t, t, BF, workspace=WS if nb else None, workspace_bytes=nb, **kw)


@pytest.mark.parametrize("M", [1, 7, 16, 17, 32])
@pytest.mark.parametrize("N,cols", [(4, 4), (2047, 4), (2048, 8), (4096, 16), (8192, 32), (30000, 32)])
@pytest.mark.parametrize("t", [BF, E4])
def test_few_rows_take_the_token_kernel(M, N, cols, t):
    p = plan(M, N, 4096, t=t)
    if t == BF and M > 16 and N * 4096 > 1 << 22:   # blocks are faster where they take the operands directly
        assert p.kernel == tg.TG_EP_DIRECT
        p = plan(M, N, 4096, t=t, lda=4097)
    assert (p.kernel, p.block_n, p.splits, p.workspace_bytes) == (tg.TG_EP_TOKENS, cols, 1, 0)
    assert p.block_m >= M and p.grid * p.block_n >= N > (p.grid - 1) * p.block_n


@pytest.mark.parametrize("N,K", [(4096, 4096), (512, 8192), (40, 3056), (8192, 8192), (33, 1000)])
def test_few_rows_against_transposed_weights_part_a_long_sum(N, K):
    for M in (1, 32):
        p = plan(M, N, K, tb=0)
        if N * K > 1 << 23 and N % 8 == 0:
            assert p.kernel == tg.TG_EP_DIRECT
            p = plan(M, N, K, tb=0, lda=K + 1)
        blocks = (N + 31) // 32
        assert p.kernel == tg.TG_EP_TOKENS and p.block_n == 32 and p.grid == blocks * p.splits
        assert p.splits == 1 or (p.grid <= 256 and p.k_per_split >= 1024 and p.splits * p.k_per_split >= K)
        assert plan(M, N, K, tb=0, budget=0).splits == 1


@pytest.mark.parametrize("ta", [0, 1])
@pytest.mark.parametrize("tb", [0, 1])
@pytest.mark.parametrize("M,N,K", [(700, 272, 136), (16, 4096, 4096), (3056, 21, 27), (4096, 24, 4096), (30, 2048, 4096), (64, 4096, 64)])
def test_backward_workspace_holds_both_products_best_plans(M, N, K, ta, tb):
    need = tg.tile_gemm_ep_bwd_workspace(M, N, K, ta, tb, BF)
    da = (K, M, N, tb, 1) if ta else (M, K, N, 0, 1 - tb)
    db = (N, K, M, 1, ta) if tb else (K, N, M, 1 - ta, 0)
    for p in (da, db):
        assert need >= plan(*p).workspace_bytes


@pytest.mark.parametrize("M,N,K,bs", [
    (33, 64, 64, 64), (200, 264, 520, 64), (1024, 1024, 1024, 64), (512, 2048, 2048, 64),   # fewer than 192 128-wide blocks
    (2048, 2048, 2048, 128), (2048, 1536, 64, 128), (2048, 4096, 4096, 128), (256, 4096, 8192, 128), (256, 4096, 4096, 64),
    (4096, 4096, 64, 256), (8192, 8192, 8192, 256), (4096, 2048, 8192, 256)])
def test_block_sizes(M, N, K, bs):
    p = plan(M, N, K)
    assert (p.kernel, p.block_m, p.block_n) == (tg.TG_EP_DIRECT, bs, bs)
    assert p.grid == -(-M // bs) * -(-N // bs) * p.splits
    assert p.splits * p.k_per_split >= K > (p.splits - 1) * p.k_per_split
    q = plan(M, N, K, lda=K + 1)   # rows of A at any alignment: through registers, 128-wide at most
    assert q.kernel == tg.TG_EP_STAGED and q.block_m == (128 if -(-M // 128) * -(-N // 128) >= 192 else 64)


@pytest.mark.parametrize("M,N,K,parts", [(64, 4096, 4096, 4), (128, 4096, 4096, 2), (512, 520, 4160, 3), (64, 64, 1000, 1),
                                         (64, 64, 2048, 2), (4096, 2048, 8192, 2), (4096, 2048, 4096, 1), (2048, 2048, 8192, 1),
                                         (256, 4096, 8192, 4), (256, 4096, 4096, 1), (1024, 2048, 4096, 2)])
def test_parts_of_the_sum(M, N, K, parts):
    p = plan(M, N, K)
    assert p.splits == parts
    assert p.workspace_bytes == (parts * M * N * 4 if parts > 1 else 0)
    if parts > 1:
        assert p.k_per_split % 64 == 0 and p.k_per_split >= 16 * 64


@pytest.mark.parametrize("bad", [None, 3, "a", [1.0]])
def test_tensor_calls_name_what_is_not_a_tensor(bad):
    with pytest.raises(TypeError, match="A: expected a tensor"):
        tg.gemm_ep(bad, bad)
    with pytest.raises(TypeError, match="X: expected a tensor"):
        tg.rms_norm(bad, bad)
    with pytest.raises(TypeError, match="dY: expected a tensor"):
        tg.gemm_ep_backward(bad, bad, bad)
    with pytest.raises(TypeError, match="dY: expected a tensor"):
        tg.rms_norm_backward(bad, bad, bad, bad)


def test_unknown_names_are_refused_before_anything_else():
    for call in (lambda: tg.gemm_ep(None, None, act="tanh"), lambda: tg.gemm_ep_backward(None, None, None, act="tanh"),
                 lambda: tg.rms_norm(None, None, scales="column")):
        with pytest.raises(tg.TileError) as e:
            call()
        assert e.value.status == tg.TG_E_ARG
