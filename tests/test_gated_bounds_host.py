"""Host-only bounds of a gated block's weight loads: every chunk, stage, part and edge, both orientations."""

import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def walker(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("gated") / "gated_bounds")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-o", exe, os.path.join(HERE, "host", "gated_bounds.cpp")], check=True)
    return exe


def walk(exe, cases):
    assert cases
    r = subprocess.run([exe] + [str(x) for c in cases for x in c], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
    assert r.stdout.strip() == f"{len(cases)} operands"


@pytest.mark.parametrize("bs,group", [(64, 16), (128, 16), (256, 32), (256, 64)])
@pytest.mark.parametrize("kind,eb", [(0, 2), (1, 2), (0, 1)])
def test_every_chunk(walker, kind, eb, bs, group):
    ve, bk = 16 // eb, 128 // eb
    ns = [n for n in [4, 5, 8, 9, 15, 16, 17, 31, 32, 33, 40, 63, 64, 65, 72, 127, 128, 129, 136, 200] if kind == 0 or 2 * n >= ve]
    ks = sorted({k for k in [ve, ve + 1, 2 * ve - 1, bk - 1, bk, bk + ve, 2 * bk + 1, 3 * bk + 5, 4 * bk] if k >= ve})
    walk(walker, [(kind, eb, bs, group, n, k, gap, k) for n in ns for k in ks for gap in (0, 3, 16)])


@pytest.mark.parametrize("bs,group", [(64, 16), (128, 16), (256, 32), (256, 64)])
@pytest.mark.parametrize("kind,eb", [(0, 2), (1, 2), (0, 1)])
def test_every_chunk_of_a_part(walker, kind, eb, bs, group):
    ve, bk = 16 // eb, 128 // eb
    walk(walker, [(kind, eb, bs, group, n, p * bk * m + tail, gap, p * bk) for n in (8, 33, 64, 130) for p in (1, 2) for m in (1, 2)
                  for tail in (1, ve, bk - 1) for gap in (0, 5, 16)])
