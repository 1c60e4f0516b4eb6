"""Host-only: refusals of the scaled product's gradients."""

import pytest

import tile_level_gemm_amd as tg

from .test_abi_layer_host import A, B, BWD_REFUSED, D, R, Z, BF

RS, CS = 0xa0000000, 0xb0000000


def bwd(M=64, N=64, K=64, dY=A, Z_=Z, A_=B, B_=R, rs=RS, cs=CS, dZ=D, dA=0x70000000, dB=0x80000000, dbias=0x90000000, ta=0, tb=1,
        t=BF, act=tg.TG_ACT_GELU, ws=None, nb=0, ldy=0, ldz=0, lda=0, ldb=0):
    st = tg.lib().tile_gemm_ep_bwd_scaled(dY, Z_, A_, B_, rs, cs, dZ, dA, dB, dbias, M, N, K, ldy, ldz, lda, ldb, ta, tb, t, act,
                                          ws, nb, None)
    return st, tg.tile_last_error()


@pytest.mark.parametrize("kw,status", BWD_REFUSED + [
    (dict(rs=RS + 2), tg.TG_E_ALIGN), (dict(cs=CS + 1), tg.TG_E_ALIGN), (dict(dZ=None, act=tg.TG_ACT_NONE), tg.TG_E_NULL),
    (dict(dZ=None, act=tg.TG_ACT_NONE, cs=None), tg.TG_E_NULL), (dict(dZ=RS), tg.TG_E_ALIAS), (dict(dZ=CS + 16), tg.TG_E_ALIAS),
    (dict(dA=RS), tg.TG_E_ALIAS), (dict(dbias=CS), tg.TG_E_ALIAS), (dict(ws=RS, nb=64), tg.TG_E_ALIAS)],
    ids=lambda x: str(sorted(x.items(), key=str)) if isinstance(x, dict) else str(x))
def test_scaled_backward_refusals(kw, status):
    st, why = bwd(**kw)
    assert st == status and why


def test_scaled_backward_of_nothing():
    assert bwd(M=0, dY=None, dA=None, dB=None, dbias=None)[0] == tg.TG_OK
