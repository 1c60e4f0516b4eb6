"""Host-only bounds of the register-staged loads: every chunk of every lane, stage, part and edge."""

import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def walker(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("staged") / "staged_bounds")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-o", exe,
                    os.path.join(HERE, "host", "staged_bounds.cpp")], check=True)
    return exe


def walk(exe, cases):
    assert cases
    r = subprocess.run([exe] + [str(x) for c in cases for x in c], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    assert r.stdout.strip() == f"{len(cases)} operands"


@pytest.mark.parametrize("bs", [64, 128])
@pytest.mark.parametrize("kind,eb", [(0, 2), (1, 2), (0, 1)])
def test_every_chunk_lies_inside_the_operand(walker, kind, eb, bs):
    ve, bk = 16 // eb, 128 // eb
    extents = [ve - 7, ve - 1, ve, ve + 1, 63, 64, 65, 71, 72, 73, 127, 128, 129, 135, 136, 200, 257] if kind == 0 else \
        [ve, ve + 1, 15, 17, 63, 64, 65, 71, 72, 73, 127, 128, 129, 135, 136, 200, 257]
    ks = sorted({k for k in [ve - 1, ve, ve + 1, 2 * ve - 1, bk - 1, bk, bk + 1, bk + ve - 1, 2 * bk - 1, 2 * bk + 1, 3 * bk + 5,
                             4 * bk, 5 * bk + ve + 3] if k >= ve})
    walk(walker, [(kind, eb, bs, m, k, gap, k) for m in extents if m > 0 for k in ks for gap in (0, 3)])


@pytest.mark.parametrize("bs", [64, 128])
@pytest.mark.parametrize("kind,eb", [(0, 2), (1, 2), (0, 1)])
def test_every_chunk_of_a_part_lies_inside_the_operand(walker, kind, eb, bs):
    """Parts of whole stages; the last part may be shorter than a chunk."""
    ve, bk = 16 // eb, 128 // eb
    walk(walker, [(kind, eb, bs, m, p * bk * n + tail, gap, p * bk) for m in (ve, 65, 130) for p in (1, 2, 3) for n in (1, 2)
                  for tail in (1, ve - 1, ve, ve + 1, bk - 1) for gap in (0, 5)])


def test_the_walk_sees_a_chunk_outside(walker):
    # lines shorter than a chunk are not for these loads (the kernel takes them element by element)
    r = subprocess.run([walker, "0", "2", "64", "5", "7", "0", "7"], capture_output=True, text=True, timeout=60)
    assert r.returncode == 1 and "outside the operand" in r.stdout
