"""Host-only checks of the gated product (no GPU): refusals, plans, workspaces."""

import pytest
import torch

import tile_level_gemm_amd as tg

from .test_binding_checks import rec  # noqa: F401  (fixture)

A, B, D, Z, R, WS = ((1 << 40) * i for i in range(1, 7))   # far apart; only alignment and overlap are looked at
BF, F16, F32, E4, E5, I8 = tg.TG_BF16, tg.TG_F16, tg.TG_F32, tg.TG_FP8_E4M3, tg.TG_FP8_E5M2, tg.TG_I8


def plan(M=256, N=256, K=256, tb=1, at=BF, bt=None, dt=BF, A_=A, B_=B, D_=D, **kw):
    return tg.tile_gemm_gated_plan(A_, B_, D_, M, N, K, tb, at, at if bt is None else bt, dt, **kw)


REFUSED = [
    (dict(M=-1), tg.TG_E_SHAPE), (dict(N=-1), tg.TG_E_SHAPE), (dict(N=(1 << 29) + 1), tg.TG_E_SHAPE), (dict(N=1 << 62), tg.TG_E_SHAPE),
    (dict(K=(1 << 30) + 1), tg.TG_E_SHAPE), (dict(at=I8, K=131072), tg.TG_E_SHAPE),
    (dict(at=F32), tg.TG_E_DTYPE), (dict(at=BF, bt=F16), tg.TG_E_DTYPE), (dict(at=E4, bt=I8), tg.TG_E_DTYPE), (dict(dt=I8), tg.TG_E_DTYPE),
    (dict(bias=R, bias_dtype=E4), tg.TG_E_DTYPE), (dict(tb=2), tg.TG_E_ARG), (dict(act=5), tg.TG_E_ARG),
    (dict(at=E4, tb=0), tg.TG_E_LAYOUT), (dict(at=I8, tb=0), tg.TG_E_LAYOUT), (dict(lda=255), tg.TG_E_LAYOUT), (dict(ldb=255), tg.TG_E_LAYOUT),
    (dict(tb=0, ldb=511), tg.TG_E_LAYOUT), (dict(ldd=255), tg.TG_E_LAYOUT), (dict(Z=Z, ld_z=511), tg.TG_E_LAYOUT),
    (dict(workspace=WS, workspace_bytes=-1), tg.TG_E_ARG), (dict(workspace_bytes=64), tg.TG_E_NULL),
    (dict(A_=None), tg.TG_E_NULL), (dict(B_=None), tg.TG_E_NULL), (dict(D_=None), tg.TG_E_NULL),
    (dict(A_=A + 1), tg.TG_E_ALIGN), (dict(D_=D + 2, dt=F32), tg.TG_E_ALIGN), (dict(col_scale=R + 2), tg.TG_E_ALIGN),
    (dict(D_=A), tg.TG_E_ALIAS), (dict(D_=B + 400 * 512), tg.TG_E_ALIAS),   # the up projection's half
    (dict(Z=D), tg.TG_E_ALIAS), (dict(Z=D - 256 * 511 * 2, ld_z=512), tg.TG_E_ALIAS), (dict(bias=D, bias_dtype=BF), tg.TG_E_ALIAS),
    (dict(col_scale=D - 300 * 4), tg.TG_E_ALIAS), (dict(workspace=D, workspace_bytes=1024), tg.TG_E_ALIAS)]


@pytest.mark.parametrize("kw,status", REFUSED, ids=[str(sorted(k.items())) for k, _ in REFUSED])
def test_refusals(kw, status):
    with pytest.raises(tg.TileError) as e:
        plan(**kw)
    assert e.value.status == status and e.value.reason


def test_a_residual_is_refused():
    ep = tg.Epilogue(None, R, None, None, None, 0, 0, 0, 0)
    out = tg.EpPlan()
    import ctypes
    st = tg.lib().tile_gemm_gated_plan(A, B, D, 64, 64, 64, 0, 0, 0, 1, BF, BF, BF, ctypes.byref(ep), None, 0, ctypes.byref(out))
    assert st == tg.TG_E_ARG


def test_kernel_choice():
    p = plan(8192, 4096, 8192)
    assert (p.kernel, p.block_m, p.splits, p.grid) == (tg.TG_EP_DIRECT, 256, 1, 1024)
    assert plan(M=16, N=8192, K=4096).kernel == tg.TG_EP_TOKENS
    assert plan(M=16, N=8192, K=4096, tb=0).kernel == tg.TG_EP_DIRECT      # [K][2N]: blocks
    assert plan(M=16, N=8193, K=4095, tb=0).kernel == tg.TG_EP_STAGED
    assert plan(M=300, N=260, tb=0).kernel == tg.TG_EP_STAGED              # the up half's chunks are not aligned
    assert plan(M=300, N=260).kernel == tg.TG_EP_DIRECT                    # rows of either half are
    assert plan(K=0).kernel == tg.TG_EP_JOIN
    assert plan(M=0).kernel == tg.TG_EP_NONE and plan(N=0, D_=None).kernel == tg.TG_EP_NONE


@pytest.mark.parametrize("M,N,K", [(256, 2048, 8192), (64, 33, 8192), (300, 100, 5000), (4096, 2048, 4096), (40, 12, 4096)])
@pytest.mark.parametrize("t", (BF, E4, I8))
def test_workspace_and_splits(M, N, K, t):
    need = tg.tile_gemm_gated_workspace(M, N, K, 1, t)
    full = plan(M, N, K, at=t, workspace=1 << 44, workspace_bytes=need) if need else plan(M, N, K, at=t)
    assert full.workspace_bytes <= need
    none = plan(M, N, K, at=t)
    assert none.splits == 1 and none.workspace_bytes == 0 and none.k_per_split >= K
    for b in range(0, need + 1, max(16, need // 7 // 16 * 16)):
        p = plan(M, N, K, at=t, workspace=1 << 44, workspace_bytes=b) if b else none
        assert 1 <= p.splits <= max(1, full.splits) and p.workspace_bytes <= b
        if p.splits > 1:
            assert p.splits * p.k_per_split >= K > (p.splits - 1) * p.k_per_split
            assert p.workspace_bytes == p.splits * M * 2 * ((N + 7) // 8 * 8) * 4
            assert p.k_per_split % p.block_k == 0


def bwd(M=64, N=64, K=64, dY=A, Z_=Z, A_=B, B_=R, rs=None, cs=None, dZ=D, dA=1 << 43, dB=1 << 44, dbias=1 << 45, tb=1, t=BF,
        act=tg.TG_ACT_SILU, ws=None, nb=0, ldy=0, ldz=0, lda=0, ldb=0):
    st = tg.lib().tile_gemm_gated_bwd(dY, Z_, A_, B_, rs, cs, dZ, dA, dB, dbias, M, N, K, ldy, ldz, lda, ldb, tb, t, act, ws, nb, None)
    return st, tg.tile_last_error()


BWD_REFUSED = [
    (dict(M=-1), tg.TG_E_SHAPE), (dict(N=(1 << 29) + 1), tg.TG_E_SHAPE), (dict(t=F32), tg.TG_E_DTYPE), (dict(t=I8), tg.TG_E_DTYPE),
    (dict(tb=3), tg.TG_E_ARG), (dict(act=9), tg.TG_E_ARG), (dict(dY=None), tg.TG_E_NULL), (dict(Z_=None), tg.TG_E_NULL),
    (dict(dZ=None), tg.TG_E_NULL), (dict(dZ=None, act=0), tg.TG_E_NULL), (dict(A_=None), tg.TG_E_NULL), (dict(B_=None), tg.TG_E_NULL),
    (dict(ldy=63), tg.TG_E_LAYOUT), (dict(ldz=127), tg.TG_E_LAYOUT), (dict(ldb=1), tg.TG_E_LAYOUT), (dict(tb=0, ldb=127), tg.TG_E_LAYOUT),
    (dict(dY=A + 1), tg.TG_E_ALIGN), (dict(dbias=(1 << 45) + 2), tg.TG_E_ALIGN), (dict(rs=WS + 2), tg.TG_E_ALIGN),
    (dict(dA=A), tg.TG_E_ALIAS), (dict(dB=1 << 43), tg.TG_E_ALIAS), (dict(dbias=D + 64 * 128), tg.TG_E_ALIAS),
    (dict(dZ=A), tg.TG_E_ALIAS), (dict(dZ=Z, ldz=256), tg.TG_E_ALIAS), (dict(dZ=Z + 2), tg.TG_E_ALIAS), (dict(dZ=R), tg.TG_E_ALIAS),
    (dict(cs=D), tg.TG_E_ALIAS), (dict(ws=D, nb=64), tg.TG_E_ALIAS), (dict(ws=None, nb=64), tg.TG_E_NULL),
    (dict(ws=WS + 4, nb=64), tg.TG_E_ALIGN), (dict(ws=WS, nb=-4), tg.TG_E_ARG)]


@pytest.mark.parametrize("kw,status", BWD_REFUSED, ids=[str(sorted(k.items(), key=str)) for k, _ in BWD_REFUSED])
def test_backward_refusals(kw, status):
    st, why = bwd(**kw)
    assert st == status and why


def test_empty_calls_and_queries():
    # no GPU here: a launch would fail
    tg.tile_gemm_gated(None, None, None, 0, 8, 8, 1, BF, BF, BF, stream=0)
    assert bwd(M=0, dY=None, dA=None, dB=None, dbias=None)[0] == tg.TG_OK
    assert tg.tile_gemm_gated_workspace(-1, 5, 5, 1, BF) == 0 and tg.tile_gemm_gated_workspace(64, 1 << 62, 64, 1, BF) == 0
    assert tg.tile_gemm_gated_workspace(64, 64, 8192, 1, F32) == 0 and tg.tile_gemm_gated_bwd_workspace(64, 64, 64, 1, E4) == 0
    assert tg.tile_gemm_gated_bwd_workspace(1000, 64, 64, 1, BF) >= 2 * 64 * 4


@pytest.mark.parametrize("M,N", [(33, 1 << 29), (1 << 30, 17), (129, (1 << 28) + 64)])
def test_products_past_the_threads_of_a_launch_are_refused(M, N):
    with pytest.raises(tg.TileError) as e:
        plan(M, N, 1, A_=A + 2, B_=1 << 50, D_=1 << 60)
    assert e.value.status == tg.TG_E_SHAPE and "too many" in e.value.reason


def test_tensor_calls_refuse_host_tensors():
    a = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: tg.gemm_gated(a, a), lambda: tg.gemm_gated_backward(a, a, a, a), lambda: tg.gemm_gated(a, a, act="swish")):
        with pytest.raises(tg.TileError):
            call()
    with pytest.raises(TypeError, match="A: expected a tensor"):
        tg.gemm_gated(None, None)
    with pytest.raises(TypeError, match="Z: expected a tensor"):
        tg.gemm_gated_backward(a, a, a, None)


def m(rows, cols, dtype=torch.bfloat16):
    return torch.zeros(rows, cols, dtype=dtype)


def product(**kw):
    a = dict(A=m(4, 64), B=m(16, 64), D=m(4, 8), M=4, N=8, K=64, transB=1, a_dtype=BF, b_dtype=BF, d_dtype=BF)
    a.update(kw)
    tg.tile_gemm_gated(**a, stream=0)


def gradients(**kw):
    a = dict(dY=m(4, 8), Z=m(4, 16), A=m(4, 64), B=m(16, 64), dZ=m(4, 16), dA=m(4, 64), dB=m(16, 64), dbias=torch.zeros(16), M=4, N=8,
             K=64, transB=1, dtype=BF, act=tg.TG_ACT_SILU)
    a.update(kw)
    tg.tile_gemm_gated_bwd(**a, stream=0)


@pytest.mark.parametrize("call", [product, gradients])
def test_whole_tensors_reach_the_library(rec, call):  # noqa: F811
    call()
    assert len(rec.calls) == 1


@pytest.mark.parametrize("call,kw,status", [
    (product, dict(B=m(8, 64)), tg.TG_E_SHAPE), (product, dict(bias=torch.zeros(8)), tg.TG_E_SHAPE), (product, dict(Z=m(4, 8)), tg.TG_E_SHAPE),
    (product, dict(col_scale=torch.zeros(8)), tg.TG_E_SHAPE), (product, dict(B=m(16, 72)[:, :64]), tg.TG_E_LAYOUT),
    (gradients, dict(Z=m(4, 8)), tg.TG_E_SHAPE), (gradients, dict(dZ=m(4, 24)[:, :16]), tg.TG_E_LAYOUT), (gradients, dict(dbias=torch.zeros(8)), tg.TG_E_SHAPE)])
def test_tensors_that_do_not_fit_are_refused(rec, call, kw, status):  # noqa: F811
    with pytest.raises(tg.TileError) as e:
        call(**kw)
    assert e.value.status == status and not rec.calls
