"""The feed-forward example: training and serving, against its 64-bit reference."""

import importlib.util
import os

import pytest

from .gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width,hidden,tokens", [(1024, 4096, 512), (264, 1032, 37)])
def test_feed_forward_example(width, hidden, tokens):
    say(f"feed-forward example {width} {hidden} {tokens}")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")
    spec = importlib.util.spec_from_file_location("feed_forward", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    example.main(width, hidden, tokens)
