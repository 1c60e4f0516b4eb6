"""The layer operators next to autograd: written tensors count as changed, a lost gradient is said."""

import warnings

import pytest
import torch

import tile_level_gemm_amd as tg

from .gpu_util import say
from .test_gpu_layer import T, dev, rand

pytestmark = pytest.mark.gpu


def test_written_tensors_have_a_new_version():
    say("autograd: out and h_out")
    a, b, w = rand(1, (4, 64), "bf16"), rand(2, (64, 64), "bf16"), rand(3, (64,), "bf16")
    for write in (lambda t: tg.gemm_ep(a, b, out=t), lambda t: tg.gemm_ep(a, b, out=t, keep_z=True),
                  lambda t: tg.rms_norm(a, w, residual=t, h_out=t)):
        out = rand(4, (4, 64), "bf16")
        p = torch.ones_like(out, requires_grad=True)
        loss = (p * out).sum()   # saves out
        before = out._version
        write(out)
        assert out._version > before
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    with torch.inference_mode():
        out = torch.empty(4, 64, dtype=T["bf16"], device=dev())
    tg.gemm_ep(a, b, out=out)   # inference tensors keep no version


def test_a_refused_call_leaves_the_version():
    say("autograd: refused call")
    a, b = rand(1, (4, 64), "bf16"), rand(2, (8, 64), "bf16")
    out = torch.empty(4, 7, dtype=T["bf16"], device=dev())
    with pytest.raises(tg.TileError):
        tg.gemm_ep(a, b, out=out)
    assert out._version == 0


def test_inputs_that_require_gradients_are_pointed_to_the_backward_calls():
    say("autograd: warning")
    a, w = rand(1, (4, 64), "bf16"), rand(3, (64,), "bf16")
    b = rand(2, (8, 64), "bf16").requires_grad_()
    p = w.clone().requires_grad_()
    calls = [lambda: tg.gemm_ep(a, b), lambda: tg.rms_norm(a, p).y]
    always = torch.is_warn_always_enabled()
    torch.set_warn_always(True)
    try:
        for call in calls:
            with pytest.warns(UserWarning, match="no autograd history"):
                assert not call().requires_grad
            with warnings.catch_warnings():
                warnings.simplefilter("error")
                with torch.no_grad():
                    call()
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            tg.gemm_ep(a, b.detach())
            tg.rms_norm(a, w)
    finally:
        torch.set_warn_always(always)
