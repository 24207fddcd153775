"""What the compiler gave the feed-forward kernels, read from the built library's own
metadata (no GPU needed): none of them keeps values in scratch memory, which stands for
registers that did not suffice or an array that was addressed at run time, and costs more
than the kernels' design counts with."""
import os
import struct

import msgpack
import pytest

from fp4_block_quantization_amd.build import LIB

EM_AMDGPU, NT_AMDGPU_METADATA, SHT_NOTE = 224, 32, 7


def code_objects(blob):
    """The GPU's ELF files inside the library."""
    at = blob.find(b"\x7fELF", 4)
    while at >= 0:
        if struct.unpack_from("<H", blob, at + 18)[0] == EM_AMDGPU:
            yield at
        at = blob.find(b"\x7fELF", at + 4)


def notes(blob, elf):
    shoff, = struct.unpack_from("<Q", blob, elf + 40)
    entsize, count = struct.unpack_from("<HH", blob, elf + 58)
    for i in range(count):
        _, kind, _, _, offset, size = struct.unpack_from("<IIQQQQ", blob, elf + shoff + i * entsize)
        at, end = elf + offset, elf + offset + size
        while kind == SHT_NOTE and at < end:
            name_size, desc_size, note = struct.unpack_from("<III", blob, at)
            desc = at + 12 + (name_size + 3) // 4 * 4
            if note == NT_AMDGPU_METADATA:
                yield msgpack.unpackb(blob[desc:desc + desc_size])
            at = desc + (desc_size + 3) // 4 * 4


@pytest.fixture(scope="module")
def scratch():
    """Bytes of scratch memory a lane, by the kernel's mangled name."""
    with open(LIB, "rb") as f:
        blob = f.read()
    return {k[".name"]: k[".private_segment_fixed_size"] for elf in code_objects(blob)
            for meta in notes(blob, elf) for k in meta["amdhsa.kernels"]}


def test_the_library_was_read(scratch):
    assert os.path.getsize(LIB) > 0 and len(scratch) > 200
    assert any("rmsnorm_kernel" in k for k in scratch)


# products with an epilogue: of NVFP4 (with kFused or kGated; the plain product shares the
# kernel) and MXFP4 records
@pytest.mark.parametrize("kernel", ["qlinear_lds_kernel", "mx_flow_kernel"])
def test_products_with_an_epilogue_keep_nothing_in_scratch(scratch, kernel):
    mine = {k: v for k, v in scratch.items() if kernel in k}
    assert len(mine) >= 8 and not {k: v for k, v in mine.items() if v}


def test_norms_keep_nothing_in_scratch(scratch):
    mine = {k: v for k, v in scratch.items() if "rmsnorm" in k}
    assert any("rmsnorm_bwd_kernelILi512ELi4" in k for k in mine)      # the longest rows
    assert not {k: v for k, v in mine.items() if v}
