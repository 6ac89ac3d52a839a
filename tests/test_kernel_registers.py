"""What the compiled kernels keep in memory instead of registers, from the metadata of the built library (no GPU)."""
import struct

import msgpack
import pytest

from tile_binned_gaussian_amd import binding, build

BUNDLE, NOTE, METADATA = b"__CLANG_OFFLOAD_BUNDLE__", 7, 32
# bytes of memory a lane. The most are the spills of the large tiles of products and weight gradients and of the router
# above 1024 experts (at most 226 registers of 4 bytes); accumulators alone would be 1024 beside those.
MOST = 1024


def code_objects(data):
    """The gfx950 code objects of the library's bundles."""
    at = data.find(BUNDLE)
    while at >= 0:
        (count,), p = struct.unpack_from("<Q", data, at + 24), at + 32
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", data, p)
            if b"gfx950" in data[p + 24:p + 24 + length]:
                yield data[at + offset:at + offset + size]
            p += 24 + length
        at = data.find(BUNDLE, at + 1)


def kernels(elf):
    """The kernels' metadata from the notes of a 64-bit ELF file."""
    (sections,), (size, count) = struct.unpack_from("<Q", elf, 40), struct.unpack_from("<HH", elf, 58)
    for i in range(count):
        kind, = struct.unpack_from("<I", elf, sections + i * size + 4)
        at, length = struct.unpack_from("<QQ", elf, sections + i * size + 24)
        end = at + length
        while kind == NOTE and at < end:
            name, body, note = struct.unpack_from("<III", elf, at)
            at += 12 + (name + 3) // 4 * 4
            if note == METADATA:
                yield from msgpack.unpackb(elf[at:at + body])["amdhsa.kernels"]
            at += (body + 3) // 4 * 4


@pytest.fixture(scope="module")
def built():
    if build.stale():
        build.build()
    with open(binding.LIB_PATH, "rb") as f:
        return {k[".name"]: k for elf in code_objects(f.read()) for k in kernels(elf)}


def test_no_kernel_keeps_its_accumulators_in_memory(built):
    assert len(built) > 100 and any("weight_grad_kernel" in name for name in built)
    assert {n: k[".private_segment_fixed_size"] for n, k in built.items() if k[".private_segment_fixed_size"] > MOST} == {}


def test_a_loop_that_is_not_unrolled_ends_the_build():
    assert "-Werror=pass-failed" in build.HIPCC_FLAGS
