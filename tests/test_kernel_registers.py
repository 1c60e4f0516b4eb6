"""Registers of the built kernels, from the metadata that the compiler puts into libtilegemm.so: the block kernels
of the products with an epilogue hold all they need in registers.  A spilled one would be loaded again in the K
loop, on the counter that the operands' loads wait on, so that each such load waits for them too."""

import struct

import msgpack
import pytest

from tile_level_gemm_amd import build


def code_objects(blob):
    """The gfx950 images of a library's offload bundles."""
    magic, at = b"__CLANG_OFFLOAD_BUNDLE__", 0
    while (at := blob.find(magic, at)) >= 0:
        (count,), p = struct.unpack_from("<Q", blob, at + len(magic)), at + len(magic) + 8
        for _ in range(count):
            offset, size, n = struct.unpack_from("<QQQ", blob, p)
            if b"gfx950" in blob[p + 24:p + 24 + n] and size:
                yield blob[at + offset:at + offset + size]
            p += 24 + n
        at += len(magic)


def kernels(image):
    """The kernels' entries of an ELF image's metadata note."""
    headers, = struct.unpack_from("<Q", image, 40)
    each, count = struct.unpack_from("<HH", image, 58)
    for i in range(count):
        kind, = struct.unpack_from("<I", image, headers + i * each + 4)
        p, size = struct.unpack_from("<QQ", image, headers + i * each + 24)
        end = p + size
        while kind == 7 and p < end:   # SHT_NOTE
            name, desc, note = struct.unpack_from("<III", image, p)
            p += 12 + (name + 3) // 4 * 4
            if note == 32:             # NT_AMDGPU_METADATA
                yield from msgpack.unpackb(image[p:p + desc])["amdhsa.kernels"]
            p += (desc + 3) // 4 * 4


@pytest.fixture(scope="module")
def built():
    with open(build.LIB, "rb") as f:
        blob = f.read()
    return {k[".name"]: k for image in code_objects(blob) for k in kernels(image)}


@pytest.mark.parametrize("family", ["gemm_ep_staged", "gemm_ep_ring", "gemm_ep_direct", "gemm_ep_fine", "gemm_ep_tokens"])
def test_block_kernels_spill_nothing(built, family):
    those = {n: k for n, k in built.items() if family in n}
    assert len(those) >= 10   # types and orientations
    bad = {n: (k[".vgpr_spill_count"], k[".private_segment_fixed_size"]) for n, k in those.items()
           if k[".vgpr_spill_count"] or k[".private_segment_fixed_size"]}
    assert not bad
