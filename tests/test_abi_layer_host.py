"""Host-only checks of the layer operators (no GPU): refusals, plans, workspaces."""

import ctypes

import pytest

import tile_level_gemm_amd as tg

A, B, D, Z, R, WS = (0x10000000 * i for i in range(1, 7))   # far apart; only alignment and overlap are looked at
BF, F16, F32, E4, E5 = tg.TG_BF16, tg.TG_F16, tg.TG_F32, tg.TG_FP8_E4M3, tg.TG_FP8_E5M2


def plan(M=256, N=256, K=256, ta=0, tb=1, at=BF, bt=None, dt=BF, A_=A, B_=B, D_=D, **kw):
    return tg.tile_gemm_ep_plan(A_, B_, D_, M, N, K, ta, tb, at, at if bt is None else bt, dt, **kw)


REFUSED = [
    (dict(M=-1), tg.TG_E_SHAPE), (dict(N=(1 << 30) + 1), tg.TG_E_SHAPE),
    (dict(at=F32), tg.TG_E_DTYPE), (dict(at=BF, bt=F16), tg.TG_E_DTYPE), (dict(at=E4, bt=BF), tg.TG_E_DTYPE),
    (dict(at=tg.TG_FP4_E2M1), tg.TG_E_DTYPE), (dict(dt=E4), tg.TG_E_DTYPE), (dict(dt=0), tg.TG_E_DTYPE),
    (dict(bias=R, bias_dtype=E4), tg.TG_E_DTYPE), (dict(ta=2), tg.TG_E_ARG), (dict(tb=-1), tg.TG_E_ARG),
    (dict(act=5), tg.TG_E_ARG), (dict(act=-1), tg.TG_E_ARG),
    (dict(at=E4, ta=1), tg.TG_E_LAYOUT), (dict(at=E4, tb=0), tg.TG_E_LAYOUT),
    (dict(lda=255), tg.TG_E_LAYOUT), (dict(ldb=-8), tg.TG_E_LAYOUT), (dict(ldd=8), tg.TG_E_LAYOUT),
    (dict(residual=R, ld_residual=255), tg.TG_E_LAYOUT), (dict(Z=Z, ld_z=(1 << 40) + 1), tg.TG_E_LAYOUT),
    (dict(workspace=WS, workspace_bytes=-1), tg.TG_E_ARG), (dict(workspace_bytes=64), tg.TG_E_NULL),
    (dict(workspace=WS + 8, workspace_bytes=64), tg.TG_E_ALIGN),
    (dict(A_=None), tg.TG_E_NULL), (dict(B_=None), tg.TG_E_NULL), (dict(D_=None), tg.TG_E_NULL),
    (dict(A_=A + 1), tg.TG_E_ALIGN), (dict(D_=D + 2, dt=F32), tg.TG_E_ALIGN),
    (dict(row_scale=R + 2), tg.TG_E_ALIGN), (dict(bias=R + 1, bias_dtype=BF), tg.TG_E_ALIGN),
    (dict(D_=A), tg.TG_E_ALIAS), (dict(D_=B + 64), tg.TG_E_ALIAS), (dict(Z=A), tg.TG_E_ALIAS), (dict(Z=D), tg.TG_E_ALIAS),
    (dict(residual=D + 32), tg.TG_E_ALIAS), (dict(residual=R, Z=R), tg.TG_E_ALIAS),
    (dict(bias=D, bias_dtype=BF), tg.TG_E_ALIAS), (dict(row_scale=D), tg.TG_E_ALIAS),
    (dict(workspace=A, workspace_bytes=1024), tg.TG_E_ALIAS), (dict(workspace=D, workspace_bytes=1024), tg.TG_E_ALIAS),
    (dict(residual=D, ld_residual=512), tg.TG_E_ALIAS),   # same place, other rows
]


@pytest.mark.parametrize("kw,status", REFUSED, ids=[str(sorted(k.items())) for k, _ in REFUSED])
def test_product_refusals(kw, status):
    with pytest.raises(tg.TileError) as e:
        plan(**kw)
    assert e.value.status == status and e.value.reason


def test_product_accepts_slices_of_one_matrix():
    # A, Z and D as column ranges of one wide matrix; residual exactly D
    w = 3 * 256
    assert plan(lda=w, A_=A, D_=A + 512, ldd=w, Z=A + 1024, ld_z=w, residual=A + 512, ld_residual=w).kernel
    with pytest.raises(tg.TileError):
        plan(lda=w, A_=A, D_=A + 510, ldd=w)


def test_product_kernel_choice():
    p = plan(8192, 8192, 8192)
    assert (p.kernel, p.block_m, p.splits, p.grid) == (tg.TG_EP_DIRECT, 256, 1, 1024)
    assert plan(M=300, K=257).kernel == tg.TG_EP_STAGED           # rows of B not whole 16-byte chunks
    assert plan(M=300, A_=A + 2).kernel == tg.TG_EP_STAGED
    assert plan(M=300, lda=260).kernel == tg.TG_EP_STAGED
    assert plan(M=301, ta=1).kernel == tg.TG_EP_STAGED            # [K][301]
    assert plan(M=304, N=264, K=77, ta=1, tb=0).kernel == tg.TG_EP_DIRECT   # K runs over rows of both
    assert plan(K=0).kernel == tg.TG_EP_JOIN
    assert plan(M=0).kernel == tg.TG_EP_NONE and plan(N=0, D_=None).kernel == tg.TG_EP_NONE
    # panels above the direct loads' 32-bit offsets
    assert plan(M=300, lda=1 << 22, A_=1 << 44).kernel == tg.TG_EP_STAGED
    assert plan(M=304, K=64, ta=1, lda=1 << 24, A_=1 << 44).kernel == tg.TG_EP_STAGED


@pytest.mark.parametrize("M,N,K", [(256, 4096, 8192), (64, 64, 8192), (300, 200, 5000), (512, 512, 512), (4096, 4096, 4096)])
@pytest.mark.parametrize("t", (BF, E4))
def test_product_workspace_and_splits(M, N, K, t):
    need = tg.tile_gemm_ep_workspace(M, N, K, 0, 1, t)
    full = plan(M, N, K, at=t, workspace=1 << 44, workspace_bytes=need) if need else plan(M, N, K, at=t)
    assert full.workspace_bytes <= need
    none = plan(M, N, K, at=t)
    assert none.splits == 1 and none.workspace_bytes == 0 and none.k_per_split >= K
    for b in range(0, need + 1, max(16, need // 7 // 16 * 16)):
        p = plan(M, N, K, at=t, workspace=1 << 44, workspace_bytes=b) if b else none
        assert 1 <= p.splits <= max(1, full.splits) and p.workspace_bytes <= b
        if p.splits > 1:   # the parts cover K, each of them has some of it
            assert p.splits * p.k_per_split >= K > (p.splits - 1) * p.k_per_split
            assert p.workspace_bytes == p.splits * M * ((N + 7) // 8 * 8) * 4
            assert p.k_per_split % p.block_k == 0


def bwd(M=64, N=64, K=64, dY=A, Z_=Z, A_=B, B_=R, dZ=D, dA=0x70000000, dB=0x80000000, dbias=0x90000000, ta=0, tb=1,
        t=BF, act=tg.TG_ACT_GELU, ws=None, nb=0, ldy=0, ldz=0, lda=0, ldb=0):
    L = tg.lib()
    st = L.tile_gemm_ep_bwd(dY, Z_, A_, B_, dZ, dA, dB, dbias, M, N, K, ldy, ldz, lda, ldb, ta, tb, t, act, ws, nb, None)
    return st, tg.tile_last_error()


BWD_REFUSED = [
    (dict(M=-1), tg.TG_E_SHAPE), (dict(t=F32), tg.TG_E_DTYPE), (dict(t=E4), tg.TG_E_DTYPE), (dict(ta=3), tg.TG_E_ARG),
    (dict(act=9), tg.TG_E_ARG), (dict(dY=None), tg.TG_E_NULL), (dict(Z_=None), tg.TG_E_NULL), (dict(dZ=None), tg.TG_E_NULL),
    (dict(A_=None), tg.TG_E_NULL), (dict(B_=None), tg.TG_E_NULL), (dict(ldy=63), tg.TG_E_LAYOUT), (dict(ldb=1), tg.TG_E_LAYOUT),
    (dict(dY=A + 1), tg.TG_E_ALIGN), (dict(dbias=0x90000002), tg.TG_E_ALIGN), (dict(dA=A), tg.TG_E_ALIAS),
    (dict(dB=0x70000000), tg.TG_E_ALIAS), (dict(dbias=D), tg.TG_E_ALIAS), (dict(dZ=A + 2), tg.TG_E_ALIAS),
    (dict(dZ=A, ldy=128), tg.TG_E_ALIAS), (dict(dZ=R), tg.TG_E_ALIAS), (dict(ws=D, nb=64), tg.TG_E_ALIAS),
    (dict(ws=None, nb=64), tg.TG_E_NULL), (dict(ws=WS + 4, nb=64), tg.TG_E_ALIGN), (dict(ws=WS, nb=-4), tg.TG_E_ARG),
]


@pytest.mark.parametrize("kw,status", BWD_REFUSED, ids=[str(sorted(k.items(), key=str)) for k, _ in BWD_REFUSED])
def test_product_backward_refusals(kw, status):
    st, why = bwd(**kw)
    assert st == status and why


X, W, H, Y, S, RS = (0x10000000 * i for i in range(1, 7))


def norm(rows=4, cols=64, X_=X, R_=R + 0x40000000, W_=W, H_=H, Y_=Y, S_=S, rstd=RS, t=BF, wt=BF, yt=E4, kind=tg.TG_SCALE_ROW,
         eps=1e-5, ldx=0, ldr=0, ldh=0, ldy=0):
    st = tg.lib().tile_rmsnorm(X_, R_, W_, H_, Y_, S_, rstd, rows, cols, ldx, ldr, ldh, ldy, eps, t, wt, yt, kind, None)
    return st, tg.tile_last_error()


NORM_REFUSED = [
    (dict(rows=-1), tg.TG_E_SHAPE), (dict(cols=0), tg.TG_E_SHAPE), (dict(cols=(1 << 30) + 1), tg.TG_E_SHAPE),
    (dict(t=E4), tg.TG_E_DTYPE), (dict(wt=F16), tg.TG_E_DTYPE), (dict(yt=BF), tg.TG_E_DTYPE),
    (dict(kind=tg.TG_SCALE_NONE), tg.TG_E_DTYPE), (dict(kind=tg.TG_SCALE_NONE, yt=F32), tg.TG_E_DTYPE), (dict(kind=3), tg.TG_E_ARG),
    (dict(kind=tg.TG_SCALE_BLOCK, cols=48), tg.TG_E_SHAPE), (dict(eps=-1e-6), tg.TG_E_ARG), (dict(eps=float("nan")), tg.TG_E_ARG),
    (dict(eps=float("inf")), tg.TG_E_ARG), (dict(R_=None), tg.TG_E_ARG), (dict(ldx=63), tg.TG_E_LAYOUT), (dict(ldy=-1), tg.TG_E_LAYOUT),
    (dict(X_=None), tg.TG_E_NULL), (dict(W_=None), tg.TG_E_NULL), (dict(Y_=None), tg.TG_E_NULL), (dict(S_=None), tg.TG_E_NULL),
    (dict(X_=X + 1), tg.TG_E_ALIGN), (dict(S_=S + 2), tg.TG_E_ALIGN), (dict(rstd=RS + 1), tg.TG_E_ALIGN),
    (dict(Y_=X), tg.TG_E_ALIAS), (dict(S_=W), tg.TG_E_ALIAS), (dict(rstd=S), tg.TG_E_ALIAS), (dict(H_=X + 2), tg.TG_E_ALIAS),
    (dict(H_=X, ldh=128), tg.TG_E_ALIAS), (dict(H_=W), tg.TG_E_ALIAS), (dict(Y_=H), tg.TG_E_ALIAS),
]


@pytest.mark.parametrize("kw,status", NORM_REFUSED, ids=[str(sorted(k.items(), key=str)) for k, _ in NORM_REFUSED])
def test_norm_refusals(kw, status):
    st, why = norm(**kw)
    assert st == status and why


def norm_bwd(rows=4, cols=64, dY=X, H_=H, W_=W, rstd=RS, dH=Y, dX=S, dW=0x70000000, t=BF, wt=BF, ws=None, nb=0, ldy=0,
             ldh=0, ldd=0, ldx=0):
    st = tg.lib().tile_rmsnorm_bwd(dY, H_, W_, rstd, dH, dX, dW, rows, cols, ldy, ldh, ldd, ldx, t, wt, ws, nb, None)
    return st, tg.tile_last_error()


NORM_BWD_REFUSED = [
    (dict(rows=-1), tg.TG_E_SHAPE), (dict(cols=0), tg.TG_E_SHAPE), (dict(t=E5), tg.TG_E_DTYPE), (dict(wt=F16), tg.TG_E_DTYPE),
    (dict(ldy=1), tg.TG_E_LAYOUT), (dict(ldx=(1 << 40) + 1), tg.TG_E_LAYOUT), (dict(dY=None), tg.TG_E_NULL), (dict(rstd=None), tg.TG_E_NULL),
    (dict(dX=None), tg.TG_E_NULL), (dict(dX=S + 1), tg.TG_E_ALIGN), (dict(dW=0x70000002), tg.TG_E_ALIGN), (dict(dX=H), tg.TG_E_ALIAS),
    (dict(dX=X + 2), tg.TG_E_ALIAS), (dict(dW=W), tg.TG_E_ALIAS), (dict(ws=S, nb=64), tg.TG_E_ALIAS), (dict(nb=64), tg.TG_E_NULL),
    (dict(cols=7), tg.TG_E_ARG), (dict(cols=16385), tg.TG_E_ARG), (dict(cols=7, ws=0x90000000, nb=12), tg.TG_E_ARG),
]


@pytest.mark.parametrize("kw,status", NORM_BWD_REFUSED, ids=[str(sorted(k.items(), key=str)) for k, _ in NORM_BWD_REFUSED])
def test_norm_backward_refusals(kw, status):
    st, why = norm_bwd(**kw)
    assert st == status and why


def test_empty_calls_launch_nothing():
    # no GPU here: a launch would fail
    tg.tile_gemm_ep(None, None, None, 0, 8, 8, 0, 1, BF, BF, BF, stream=0)
    assert norm(rows=0, X_=None, Y_=None)[0] == tg.TG_OK
    assert norm_bwd(rows=0, dY=None, dX=None, dW=None)[0] == tg.TG_OK
    assert bwd(M=0, dY=None, dA=None, dB=None, dbias=None)[0] == tg.TG_OK


def test_workspace_queries_take_any_arguments():
    assert tg.tile_gemm_ep_workspace(-1, 5, 5, 0, 1, BF) == 0
    assert tg.tile_gemm_ep_workspace(64, 64, 8192, 0, 1, F32) == 0
    assert tg.tile_gemm_ep_bwd_workspace(0, 0, 0, 0, 1, BF) == 0
    assert tg.tile_rmsnorm_bwd_workspace(5, 0, BF) == 0
    assert tg.tile_rmsnorm_bwd_workspace(100, 64, BF) > 0
    assert tg.tile_rmsnorm_bwd_workspace(100, 7, BF) >= 400
    assert ctypes.sizeof(tg.Epilogue) == 64 and ctypes.sizeof(tg.EpPlan) == 40


def test_tensor_calls_refuse_host_tensors():
    import torch
    a = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: tg.gemm_ep(a, a), lambda: tg.rms_norm(a, a[0]), lambda: tg.gemm_ep_backward(a, a, a),
                 lambda: tg.rms_norm_backward(a, a, a[0], torch.zeros(4))):
        with pytest.raises(tg.TileError):
            call()
