"""Registers of the operators' kernels: none of them keeps registers in memory.

Reads the kernel descriptions that the compiler leaves in the library (the
metadata note of every gfx950 code object).  Runs without a GPU."""
import struct

import msgpack
import pytest

from bit_gemm_block_amd import build as b

NAMES = ("shrink_rows_kernel", "shrink_stage_kernel", "expand_rows_kernel", "expand_many_kernel",
         "norm_residual_kernel", "gated_kernel")
ELF, AMDGPU, NOTE, METADATA = b"\x7fELF", 224, 7, 32


def notes(elf):
    """The descriptors of an ELF file's metadata notes."""
    shoff, = struct.unpack_from("<Q", elf, 0x28)
    size, count = struct.unpack_from("<HH", elf, 0x3A)
    for i in range(count):
        kind, = struct.unpack_from("<I", elf, shoff + i * size + 4)
        at, length = struct.unpack_from("<QQ", elf, shoff + i * size + 0x18)
        end = at + length
        while kind == NOTE and at + 12 <= end:
            n, d, t = struct.unpack_from("<III", elf, at)
            desc = at + 12 + (n + 3) // 4 * 4
            if t == METADATA:
                yield elf[desc:desc + d]
            at = desc + (d + 3) // 4 * 4


@pytest.fixture(scope="module")
def kernels():
    with open(b.LIB, "rb") as f:
        lib = f.read()
    found, at = {}, lib.find(ELF, 1)
    while at >= 0:
        if struct.unpack_from("<H", lib, at + 18)[0] == AMDGPU:
            for note in notes(lib[at:]):
                for k in msgpack.unpackb(note)["amdhsa.kernels"]:
                    found[k[".name"]] = k
        at = lib.find(ELF, at + 4)
    return found


@pytest.mark.parametrize("name", NAMES)
def test_no_scratch(kernels, name):
    mine = {k: v for k, v in kernels.items() if name in k}
    assert mine
    for k, v in mine.items():
        assert v[".private_segment_fixed_size"] == 0 and v[".vgpr_spill_count"] == 0, (
            k, v[".private_segment_fixed_size"], v[".vgpr_spill_count"])
