"""Host-only: products of 8-bit integers are planned or refused before anything is launched."""

import pytest

import tile_level_gemm_amd as tg

A, B, D, WS = (1 << 44) * 1, (1 << 44) * 2, (1 << 44) * 3, (1 << 44) * 4
I8, E4, BF, F32 = tg.TG_I8, tg.TG_FP8_E4M3, tg.TG_BF16, tg.TG_F32


def plan(M=256, N=256, K=256, ta=0, tb=1, at=I8, bt=I8, dt=BF, a=A, **kw):
    return tg.tile_gemm_ep_plan(a, B, D, M, N, K, ta, tb, at, bt, dt, **kw)


@pytest.mark.parametrize("kw,status", [
    (dict(bt=E4), tg.TG_E_DTYPE), (dict(at=E4), tg.TG_E_DTYPE), (dict(bt=BF), tg.TG_E_DTYPE), (dict(at=tg.TG_U8, bt=tg.TG_U8), tg.TG_E_DTYPE),
    (dict(dt=I8), tg.TG_E_DTYPE), (dict(ta=1), tg.TG_E_LAYOUT), (dict(tb=0), tg.TG_E_LAYOUT), (dict(lda=255), tg.TG_E_LAYOUT),
    (dict(K=131072), tg.TG_E_SHAPE), (dict(K=1 << 30), tg.TG_E_SHAPE)])
def test_refusals(kw, status):
    with pytest.raises(tg.TileError) as e:
        plan(**kw)
    assert e.value.status == status and e.value.reason


def test_kernel_choice():
    assert plan(8192, 8192, 4096).block_m == 256 and plan(8192, 8192, 4096).block_k == 128
    assert plan(16, 8192, 4096).kernel == tg.TG_EP_TOKENS
    assert plan(K=131071).kernel == tg.TG_EP_STAGED and plan(K=131056).kernel == tg.TG_EP_DIRECT
    assert plan(a=A + 1).kernel == tg.TG_EP_STAGED    # any byte is aligned to its element
    assert plan(K=0).kernel == tg.TG_EP_JOIN


def test_parts_of_a_long_sum():
    need = tg.tile_gemm_ep_workspace(64, 64, 65536, 0, 1, I8)
    p = plan(64, 64, 65536, workspace=WS, workspace_bytes=need)
    assert p.splits > 1 and p.workspace_bytes == need


def test_gradients_take_16_bits():
    st = tg.lib().tile_gemm_ep_bwd(A, None, B, D, None, WS, None, None, 64, 64, 64, 0, 0, 0, 0, 0, 1, I8, 0, None, 0, None)
    assert st == tg.TG_E_DTYPE
    assert tg.tile_gemm_ep_bwd_workspace(64, 64, 64, 0, 1, I8) == 0
