"""Rows quantised to 8-bit integers have the scales and codes of the same computation in torch on the GPU, bit for
bit: max / 127 and round(x / scale) in fp32, so that weights may be quantised by either."""

import pytest
import torch

import tile_level_gemm_amd as tg

from .gpu_util import say
from .test_gpu_layer import T, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(1, 5), (37, 72), (300, 1000), (1024, 4096), (512, 8200), (40, 20000)])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_integer_rows(rows, cols, dtype):
    say(f"rows as torch's {rows}x{cols} {dtype}")
    g = torch.Generator(device=dev()).manual_seed(rows + cols)
    X = (torch.randn(rows, cols, generator=g, device=dev()) * (1 + 15 * (torch.rand(cols, generator=g, device=dev()) < 0.01))).to(T[dtype])
    X[:, 0] = X.abs().amax(dim=1)
    X[:, 1] = X[:, 0] / 2   # 63.5 steps: the scale's last bit decides the code
    q, s = tg.quantize_rows(X)
    x = X.float()
    scale = x.abs().amax(dim=1) / 127.0
    assert torch.equal(s, scale)
    assert torch.equal(q, torch.round(x / scale[:, None]).clamp(-127, 127).to(torch.int8))
