"""Host-only checks of the layer norm and the quantised rows (no GPU): refusals, workspaces."""

import pytest
import torch

import tile_level_gemm_amd as tg

from .test_binding_checks import rec  # noqa: F401  (fixture)

X, R, W, B, H, Y, S, ME, RS = (0x10000000 * i for i in range(1, 10))
BF, F16, F32, E4, E5, I8 = tg.TG_BF16, tg.TG_F16, tg.TG_F32, tg.TG_FP8_E4M3, tg.TG_FP8_E5M2, tg.TG_I8
NONE, ROW, BLOCK = tg.TG_SCALE_NONE, tg.TG_SCALE_ROW, tg.TG_SCALE_BLOCK


def norm(rows=4, cols=64, X_=X, R_=R, W_=W, B_=B, H_=H, Y_=Y, S_=S, mean=ME, rstd=RS, ldx=0, ldr=0, ldh=0, ldy=0, eps=1e-5, t=BF,
         wt=BF, yt=E4, kind=ROW):
    st = tg.lib().tile_layernorm(X_, R_, W_, B_, H_, Y_, S_, mean, rstd, rows, cols, ldx, ldr, ldh, ldy, eps, t, wt, yt, kind, None)
    return st, tg.tile_last_error()


def norm_bwd(rows=4, cols=64, dY=X, H_=H, W_=W, mean=ME, rstd=RS, dH=Y, dX=S, dW=0xa0000000, dB=0xb0000000, t=BF, wt=BF, ws=None,
             nb=0, ldy=0, ldh=0, ldd=0, ldx=0):
    st = tg.lib().tile_layernorm_bwd(dY, H_, W_, mean, rstd, dH, dX, dW, dB, rows, cols, ldy, ldh, ldd, ldx, t, wt, ws, nb, None)
    return st, tg.tile_last_error()


def quantise(rows=4, cols=64, X_=X, Y_=Y, S_=S, ldx=0, ldy=0, t=BF, yt=I8, kind=ROW):
    return tg.lib().tile_quantize_rows(X_, Y_, S_, rows, cols, ldx, ldy, t, yt, kind, None), tg.tile_last_error()


REFUSED = [(norm, kw, st) for kw, st in [
    (dict(rows=-1), tg.TG_E_SHAPE), (dict(cols=0), tg.TG_E_SHAPE), (dict(cols=(1 << 30) + 1), tg.TG_E_SHAPE), (dict(t=I8), tg.TG_E_DTYPE),
    (dict(wt=F16), tg.TG_E_DTYPE), (dict(yt=BF), tg.TG_E_DTYPE), (dict(kind=NONE), tg.TG_E_DTYPE), (dict(yt=tg.TG_U8), tg.TG_E_DTYPE),
    (dict(kind=BLOCK, yt=I8), tg.TG_E_DTYPE), (dict(kind=NONE, yt=I8), tg.TG_E_DTYPE), (dict(kind=7), tg.TG_E_ARG),
    (dict(kind=BLOCK, cols=48), tg.TG_E_SHAPE), (dict(eps=-1.0), tg.TG_E_ARG), (dict(eps=float("nan")), tg.TG_E_ARG),
    (dict(R_=None), tg.TG_E_ARG), (dict(ldx=63), tg.TG_E_LAYOUT), (dict(ldr=1), tg.TG_E_LAYOUT), (dict(ldh=-1), tg.TG_E_LAYOUT),
    (dict(ldy=(1 << 40) + 1), tg.TG_E_LAYOUT), (dict(X_=None), tg.TG_E_NULL), (dict(W_=None), tg.TG_E_NULL), (dict(Y_=None), tg.TG_E_NULL),
    (dict(S_=None), tg.TG_E_NULL), (dict(X_=X + 1), tg.TG_E_ALIGN), (dict(B_=B + 1), tg.TG_E_ALIGN), (dict(mean=ME + 2), tg.TG_E_ALIGN),
    (dict(rstd=RS + 2), tg.TG_E_ALIGN), (dict(Y_=X), tg.TG_E_ALIAS), (dict(mean=W), tg.TG_E_ALIAS), (dict(mean=RS), tg.TG_E_ALIAS),
    (dict(mean=B), tg.TG_E_ALIAS), (dict(rstd=S), tg.TG_E_ALIAS), (dict(H_=B), tg.TG_E_ALIAS), (dict(H_=X + 2), tg.TG_E_ALIAS),
    (dict(H_=X, ldh=128), tg.TG_E_ALIAS), (dict(Y_=H), tg.TG_E_ALIAS)]] + [(norm_bwd, kw, st) for kw, st in [
        (dict(rows=-1), tg.TG_E_SHAPE), (dict(cols=0), tg.TG_E_SHAPE), (dict(t=E5), tg.TG_E_DTYPE), (dict(wt=F16), tg.TG_E_DTYPE),
        (dict(ldy=1), tg.TG_E_LAYOUT), (dict(dY=None), tg.TG_E_NULL), (dict(mean=None), tg.TG_E_NULL), (dict(rstd=None), tg.TG_E_NULL),
        (dict(dX=None), tg.TG_E_NULL), (dict(dX=S + 1), tg.TG_E_ALIGN), (dict(dB=0xb0000002), tg.TG_E_ALIGN), (dict(mean=ME + 1), tg.TG_E_ALIGN),
        (dict(dX=H), tg.TG_E_ALIAS), (dict(dX=X + 2), tg.TG_E_ALIAS), (dict(dW=ME), tg.TG_E_ALIAS), (dict(dB=0xa0000000), tg.TG_E_ALIAS),
        (dict(dB=S), tg.TG_E_ALIAS), (dict(ws=S, nb=64), tg.TG_E_ALIAS), (dict(ws=ME, nb=64), tg.TG_E_ALIAS), (dict(nb=64), tg.TG_E_NULL),
        (dict(cols=7), tg.TG_E_ARG), (dict(cols=16385, ws=0xc0000000, nb=28), tg.TG_E_ARG)]] + [(quantise, kw, st) for kw, st in [
            (dict(rows=-1), tg.TG_E_SHAPE), (dict(cols=0), tg.TG_E_SHAPE), (dict(t=I8), tg.TG_E_DTYPE), (dict(yt=BF), tg.TG_E_DTYPE),
            (dict(yt=tg.TG_U8), tg.TG_E_DTYPE), (dict(kind=NONE), tg.TG_E_ARG), (dict(kind=NONE, yt=BF), tg.TG_E_ARG),
            (dict(kind=BLOCK), tg.TG_E_DTYPE), (dict(kind=BLOCK, yt=E4, cols=40), tg.TG_E_SHAPE), (dict(ldx=63), tg.TG_E_LAYOUT),
            (dict(ldy=63), tg.TG_E_LAYOUT), (dict(X_=None), tg.TG_E_NULL), (dict(Y_=None), tg.TG_E_NULL), (dict(S_=None), tg.TG_E_NULL),
            (dict(X_=X + 1), tg.TG_E_ALIGN), (dict(S_=S + 1), tg.TG_E_ALIGN), (dict(Y_=X), tg.TG_E_ALIAS), (dict(S_=X + 64), tg.TG_E_ALIAS),
            (dict(S_=Y), tg.TG_E_ALIAS)]]


@pytest.mark.parametrize("call,kw,status", REFUSED, ids=[f"{c.__name__} {sorted(k.items(), key=str)}" for c, k, _ in REFUSED])
def test_refusals(call, kw, status):
    st, why = call(**kw)
    assert st == status and why


def test_rms_norm_takes_integer_rows_only():
    L = tg.lib()
    for kind, yt in ((BLOCK, I8), (NONE, I8), (ROW, tg.TG_U8)):
        assert L.tile_rmsnorm(X, None, W, None, Y, S, RS, 4, 64, 0, 0, 0, 0, 1e-5, BF, BF, yt, kind, None) == tg.TG_E_DTYPE


def test_empty_calls_launch_nothing():
    # no GPU here: a launch would fail
    assert norm(rows=0, X_=None, Y_=None)[0] == tg.TG_OK
    assert norm_bwd(rows=0, dY=None, dX=None, mean=None, dW=None, dB=None)[0] == tg.TG_OK
    assert quantise(rows=0, X_=None, Y_=None, S_=None)[0] == tg.TG_OK


def test_workspaces():
    L = tg.tile_layernorm_bwd_workspace
    assert L(5, 0, BF) == 0 and L(-1, 8, BF) == 0 and L(8, 8, I8) == 0
    assert L(100, 64, BF) == 2 * tg.tile_rmsnorm_bwd_workspace(100, 64, BF)
    assert L(100, 7, BF) >= 800


def test_tensor_calls_refuse_host_tensors_and_what_is_none():
    a, v = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4)
    for call in (lambda: tg.layer_norm(a, a[0]), lambda: tg.layer_norm_backward(a, a, a[0], v, v), lambda: tg.quantize_rows(a),
                 lambda: tg.quantize_rows(a, scales=None), lambda: tg.quantize_rows(a, scales="tensor"),
                 lambda: tg.layer_norm(a, a[0], scales="column")):
        with pytest.raises(tg.TileError):
            call()
    with pytest.raises(TypeError, match="X: expected a tensor"):
        tg.layer_norm(None, None)
    with pytest.raises(TypeError, match="dY: expected a tensor"):
        tg.layer_norm_backward(None, None, None, None, None)
    with pytest.raises(TypeError, match="X: expected a tensor"):
        tg.quantize_rows([1.0])


def m(rows, cols, dtype=torch.bfloat16):
    return torch.zeros(rows, cols, dtype=dtype)


def v(n, dtype=torch.float32):
    return torch.zeros(n, dtype=dtype)


def a_norm(**kw):
    a = dict(X=m(4, 64), R=m(4, 64), W=v(64, torch.bfloat16), bias=v(64, torch.bfloat16), H=m(4, 64), Y=m(4, 64, torch.int8), S=v(4),
             mean=v(4), rstd=v(4), rows=4, cols=64, eps=1e-5, dtype=BF, w_dtype=BF, y_dtype=I8, scale_kind=ROW)
    a.update(kw)
    tg.tile_layernorm(**a, stream=0)


def a_gradient(**kw):
    a = dict(dY=m(4, 64), H=m(4, 64), W=v(64, torch.bfloat16), mean=v(4), rstd=v(4), dH=m(4, 64), dX=m(4, 64), dW=v(64), dbias=v(64),
             rows=4, cols=64, dtype=BF, w_dtype=BF)
    a.update(kw)
    tg.tile_layernorm_bwd(**a, stream=0)


def a_quantisation(**kw):
    a = dict(X=m(4, 64), Y=m(4, 64, torch.int8), S=v(4), rows=4, cols=64, dtype=BF, y_dtype=I8, scale_kind=ROW)
    a.update(kw)
    tg.tile_quantize_rows(**a, stream=0)


@pytest.mark.parametrize("call", [a_norm, a_gradient, a_quantisation])
def test_whole_tensors_reach_the_library(rec, call):  # noqa: F811
    call()
    assert len(rec.calls) == 1


@pytest.mark.parametrize("call,kw,status", [
    (a_norm, dict(X=m(4, 72)[:, :64]), tg.TG_E_LAYOUT), (a_norm, dict(bias=v(32, torch.bfloat16)), tg.TG_E_SHAPE),
    (a_norm, dict(mean=v(3)), tg.TG_E_SHAPE), (a_norm, dict(bias=v(64)), tg.TG_E_DTYPE), (a_norm, dict(S=v(3)), tg.TG_E_SHAPE),
    (a_gradient, dict(dbias=v(128)[::2]), tg.TG_E_LAYOUT), (a_gradient, dict(mean=v(2)), tg.TG_E_SHAPE),
    (a_gradient, dict(dX=m(4, 64, torch.float32)), tg.TG_E_DTYPE), (a_quantisation, dict(Y=m(4, 72, torch.int8)[:, :64]), tg.TG_E_LAYOUT),
    (a_quantisation, dict(Y=m(4, 64)), tg.TG_E_DTYPE), (a_quantisation, dict(S=v(2)), tg.TG_E_SHAPE)])
def test_tensors_that_do_not_fit_are_refused(rec, call, kw, status):  # noqa: F811
    with pytest.raises(tg.TileError) as e:
        call(**kw)
    assert e.value.status == status and not rec.calls
