"""The layer operators' address-level calls refuse tensors whose strides are not what the call reads and
writes (CPU only: the library is replaced by a recorder)."""

import pytest
import torch

import tile_level_gemm_amd as tg

from .test_binding_checks import rec  # noqa: F401  (fixture)

BF = tg.TG_BF16


def m(rows, cols, dtype=torch.bfloat16):
    return torch.zeros(rows, cols, dtype=dtype)


def slice_of(rows, cols, dtype=torch.bfloat16):
    return m(rows, cols + 8, dtype)[:, :cols]


def every_second(n, dtype=torch.float32):
    return torch.zeros(2 * n, dtype=dtype)[::2]


def product(**kw):
    a = dict(A=m(4, 64), B=m(8, 64), D=m(4, 8), M=4, N=8, K=64, transA=0, transB=1, a_dtype=BF, b_dtype=BF, d_dtype=BF)
    a.update(kw)
    tg.tile_gemm_ep(**a, stream=0)


def gradients(**kw):
    a = dict(dY=m(4, 8), Z=m(4, 8), A=m(4, 64), B=m(8, 64), dZ=m(4, 8), dA=m(4, 64), dB=m(8, 64), dbias=torch.zeros(8),
             M=4, N=8, K=64, transA=0, transB=1, dtype=BF, act=tg.TG_ACT_SILU)
    a.update(kw)
    tg.tile_gemm_ep_bwd(**a, stream=0)


def norm(**kw):
    a = dict(X=m(4, 64), R=m(4, 64), W=torch.zeros(64, dtype=torch.bfloat16), H=m(4, 64), Y=m(4, 64, torch.uint8),
             S=torch.zeros(4), rstd=torch.zeros(4), rows=4, cols=64, eps=1e-5, dtype=BF, w_dtype=BF, y_dtype=tg.TG_FP8_E4M3,
             scale_kind=tg.TG_SCALE_ROW)
    a.update(kw)
    tg.tile_rmsnorm(**a, stream=0)


def norm_gradients(**kw):
    a = dict(dY=m(4, 64), H=m(4, 64), W=torch.zeros(64, dtype=torch.bfloat16), rstd=torch.zeros(4), dH=m(4, 64), dX=m(4, 64),
             dW=torch.zeros(64), rows=4, cols=64, dtype=BF, w_dtype=BF)
    a.update(kw)
    tg.tile_rmsnorm_bwd(**a, stream=0)


@pytest.mark.parametrize("call", [product, gradients, norm, norm_gradients])
def test_whole_tensors_reach_the_library(rec, call):  # noqa: F811
    call()
    assert len(rec.calls) == 1


MATRICES = [(product, "A", "lda", (4, 64)), (product, "B", "ldb", (8, 64)), (product, "D", "ldd", (4, 8)),
            (product, "residual", "ld_residual", (4, 8)), (product, "Z", "ld_z", (4, 8)),
            (gradients, "dY", "ld_dy", (4, 8)), (gradients, "Z", "ld_z", (4, 8)), (gradients, "A", "lda", (4, 64)),
            (gradients, "B", "ldb", (8, 64)), (norm, "X", "ld_x", (4, 64)), (norm, "R", "ld_r", (4, 64)), (norm, "H", "ld_h", (4, 64)),
            (norm_gradients, "dY", "ld_dy", (4, 64)), (norm_gradients, "H", "ld_h", (4, 64)),
            (norm_gradients, "dH", "ld_dh", (4, 64)), (norm_gradients, "dX", "ld_dx", (4, 64))]


@pytest.mark.parametrize("call,name,ld,shape", MATRICES, ids=[f"{c.__name__}-{n}" for c, n, _, _ in MATRICES])
def test_a_slice_goes_with_its_leading_dimension_only(rec, call, name, ld, shape):  # noqa: F811
    x = slice_of(*shape)
    call(**{name: x, ld: shape[1] + 8})
    assert len(rec.calls) == 1
    bad = [(x, 0), (x, shape[1]), (x, shape[1] + 16), (m(shape[1], shape[0]).t(), 0), (m(shape[0], 2 * shape[1])[:, ::2], 2 * shape[1]),
           (m(1, shape[1]).expand(*shape), 0), (torch.zeros(2, *shape, 2, dtype=torch.bfloat16)[..., 0], 0)]
    for t, l in bad:
        with pytest.raises(tg.TileError) as e:
            call(**{name: t, ld: l})
        assert e.value.status in (tg.TG_E_LAYOUT, tg.TG_E_SHAPE) and name in e.value.reason
    assert len(rec.calls) == 1


VECTORS = [(product, "bias", lambda: every_second(8)), (product, "row_scale", lambda: every_second(4)),
           (product, "col_scale", lambda: every_second(8)), (product, "workspace", lambda: every_second(64)),
           (gradients, "dZ", lambda: slice_of(4, 8)), (gradients, "dA", lambda: slice_of(4, 64)), (gradients, "dB", lambda: slice_of(8, 64)),
           (gradients, "dbias", lambda: every_second(8)), (gradients, "row_scale", lambda: every_second(4)),
           (gradients, "col_scale", lambda: every_second(8)), (gradients, "workspace", lambda: every_second(64)),
           (norm, "W", lambda: every_second(64, torch.bfloat16)), (norm, "S", lambda: every_second(4)), (norm, "rstd", lambda: every_second(4)),
           (norm_gradients, "W", lambda: every_second(64, torch.bfloat16)), (norm_gradients, "rstd", lambda: every_second(4)),
           (norm_gradients, "dW", lambda: every_second(64)), (norm_gradients, "workspace", lambda: every_second(64))]


@pytest.mark.parametrize("call,name,make", VECTORS, ids=[f"{c.__name__}-{n}" for c, n, _ in VECTORS])
def test_packed_arguments_have_no_gaps(rec, call, name, make):  # noqa: F811
    with pytest.raises(tg.TileError) as e:
        call(**{name: make()})
    assert e.value.status == tg.TG_E_LAYOUT and name in e.value.reason and not rec.calls


def test_flat_buffers_and_single_rows_need_no_shape(rec):  # noqa: F811
    product(A=torch.zeros(3 * 80 + 64, dtype=torch.bfloat16), lda=80)          # a flat buffer with any leading dimension
    product(A=m(4, 80)[:1, :64], D=m(4, 16)[1:2, :8], M=1)                      # one row: its stride plays no part
    product(D=m(4, 16)[:, 3:11], ldd=16, residual=m(4, 32)[:, 5:13], ld_residual=32)
    assert len(rec.calls) == 3


@pytest.mark.parametrize("call", [product, gradients, norm_gradients])
def test_a_workspace_by_address_needs_its_size(rec, call):  # noqa: F811
    with pytest.raises(tg.TileError) as e:
        call(workspace=1 << 20)
    assert e.value.status == tg.TG_E_ARG and not rec.calls
    call(workspace=1 << 20, workspace_bytes=64)
    assert len(rec.calls) == 1


def test_a_bias_has_the_elements_its_type_says(rec):  # noqa: F811
    with pytest.raises(tg.TileError) as e:
        product(bias=torch.zeros(8), bias_dtype=BF)
    assert e.value.status == tg.TG_E_DTYPE and "bias" in e.value.reason and not rec.calls
    product(bias=torch.zeros(8), bias_dtype=tg.TG_F32)
    product(bias=torch.zeros(8, dtype=torch.bfloat16))
    assert len(rec.calls) == 2
