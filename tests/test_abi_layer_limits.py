"""Host-only: extents at the end of the documented range are planned or refused before anything is launched."""

import pytest

import tile_level_gemm_amd as tg

A, B, D = (1 << 44) * 1, (1 << 44) * 2, (1 << 44) * 3
BF = tg.TG_BF16
TOP = 1 << 30


def plan(M, N, K, ta=0, tb=1, a=A):
    return tg.tile_gemm_ep_plan(a, B, D, M, N, K, ta, tb, BF, BF, BF)


def threads(p):
    """Threads of a workgroup at most: 64-wide blocks have 256, others 512, the token kernel one wave a K step."""
    if p.kernel == tg.TG_EP_TOKENS:
        return 64 * min(16, -(-p.k_per_split * 2 // 128))
    return 256 if p.block_m == 64 else 512


@pytest.mark.parametrize("M,N", [(33, TOP), (TOP, 33), (129, (1 << 29) + 128), ((1 << 29) + 128, 129)])
def test_products_past_the_threads_of_a_launch_are_refused(M, N):
    # at an odd address: 128-wide blocks through registers
    with pytest.raises(tg.TileError) as e:
        plan(M, N, 1, a=A + 2)
    assert e.value.status == tg.TG_E_SHAPE and "too many" in e.value.reason


@pytest.mark.parametrize("M,N,K", [(1, TOP, 8), (32, TOP, 7), (1, TOP, 64), (33, 1 << 29, 1), (33, TOP, 8), (TOP, 40, 8), (TOP, 1, 3),
                                   (128, 1 << 29, 9), (1 << 18, 1 << 18, 64)])
@pytest.mark.parametrize("a", [A, A + 2])
def test_what_is_planned_fits_a_launch(M, N, K, a):
    try:
        p = plan(M, N, K, a=a)
    except tg.TileError as e:
        assert e.status == tg.TG_E_SHAPE
        return
    assert p.grid * threads(p) < 1 << 32


def test_the_join_alone_covers_any_extent():
    p = plan(1 << 20, 1 << 21, 0)   # 2^41 results: the most
    assert p.kernel == tg.TG_EP_JOIN and p.grid == 1 << 30
    with pytest.raises(tg.TileError) as e:
        plan(1 << 21, 1 << 21, 0)
    assert e.value.status == tg.TG_E_SHAPE


@pytest.mark.parametrize("K", [(1 << 23) - 512, (1 << 23) + 1, 1 << 30])
def test_matrices_past_any_address_space_are_refused(K):
    # K rows 2^41 bytes apart: 64-bit spans wrap (K + 512 = 2^23 rows: to nothing)
    with pytest.raises(tg.TileError) as e:
        tg.tile_gemm_ep_plan(A, B, D, 64, 64, K, 1, 1, BF, BF, BF, lda=1 << 40)
    assert e.value.status == tg.TG_E_LAYOUT and "lda" in e.value.reason


def test_rows_past_any_address_space_are_refused_everywhere():
    L, far, rows = tg.lib(), 1 << 40, 1 << 29
    S, W, R = (1 << 44) * 4, (1 << 44) * 5, (1 << 44) * 6
    for ld in ((far, 0, 0, 0), (0, far, 0, 0), (0, 0, far, 0), (0, 0, 0, far)):
        assert L.tile_rmsnorm(A, B, W, R, D, None, S, rows, 8, *ld, 1e-5, BF, BF, BF, 0, None) == tg.TG_E_LAYOUT
        assert L.tile_rmsnorm_bwd(A, B, W, S, R, D, None, rows, 8, *ld, BF, BF, None, 0, None) == tg.TG_E_LAYOUT
        if ld[3] == 0:   # B has 8 rows only
            assert L.tile_gemm_ep_bwd(A, B, W, R, D, None, None, S, rows, 8, 8, *ld, 0, 0, BF, 1, None, 0, None) == tg.TG_E_LAYOUT
    for kw in (dict(ldd=far), dict(residual=R, ld_residual=far), dict(Z=R, ld_z=far)):
        with pytest.raises(tg.TileError) as e:
            tg.tile_gemm_ep_plan(A, B, D, rows, 64, 64, 0, 1, BF, BF, BF, **kw)
        assert e.value.status == tg.TG_E_LAYOUT
