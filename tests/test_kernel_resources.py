"""What the built kernels take of a CU, from the notes that the compiler leaves in the library."""

import re
import struct

import pytest

from segmented_gather_gemm_amd import build

LDS, REGISTERS = 160 * 1024, 512   # of a CU, and of a SIMD for each lane


def unpack(data, at=0):
    """One value of a MessagePack text, and where it ends: what the notes are written in."""
    b, at = data[at], at + 1

    def number(form):
        size = struct.calcsize(form)
        return struct.unpack_from(form, data, at)[0], at + size

    if b < 0x80 or b >= 0xe0:
        return (b if b < 0x80 else b - 0x100), at
    if b in (0xc2, 0xc3):
        return b == 0xc3, at
    if 0xcc <= b <= 0xd3:
        return number(">" + "BHIQbhiq"[b - 0xcc])
    if 0xa0 <= b < 0xc0 or b in (0xd9, 0xda, 0xdb):
        n, at = (b & 31, at) if b < 0xc0 else number(">" + "BHI"[b - 0xd9])
        return data[at:at + n].decode(), at + n
    assert 0x80 <= b < 0xa0 or 0xdc <= b <= 0xdf, hex(b)
    n, at = (b & 15, at) if b < 0xa0 else number(">" + "HI"[b & 1])
    is_map, values = b < 0x90 or b in (0xde, 0xdf), []
    for _ in range(2 * n if is_map else n):
        x, at = unpack(data, at)
        values.append(x)
    return (dict(zip(values[::2], values[1::2])) if is_map else values), at


def kernels():
    """Name -> notes of every kernel in the library."""
    data, at, found = open(build.LIB, "rb").read(), 0, {}
    while (at := data.find(b"AMDGPU\0\0", at)) >= 0:
        name, size, kind = struct.unpack_from("<III", data, at - 12)
        at += 8
        if (name, kind) == (7, 32):
            notes = unpack(data[at:at + size])[0]
            found.update((k[".name"], k) for k in notes["amdhsa.kernels"])
    return found


def latent_kernels():
    """(fp16, e4m3, columns, row fragments, groups, stages) -> notes."""
    found = {}
    for name, k in kernels().items():
        m = re.match(r"_ZN3sgg13latent_kernelILb(\d)ELb(\d)ELi(\d+)ELi(\d)ELi(\d)ELi(\d)E", name)
        if m:
            found[tuple(map(int, m.groups()))] = k
    return found


def test_every_instance_is_there():
    assert len(latent_kernels()) == 32


@pytest.mark.parametrize("e4m3", [0, 1])
@pytest.mark.parametrize("columns", [256, 512])
def test_two_workgroups_of_up_to_64_rows_on_a_cu(e4m3, columns):
    """The division of the work counts on 512 of them on the GPU at once."""
    seen = 0
    for key, k in latent_kernels().items():
        if key[1:3] == (e4m3, columns) and key[4] == 1:
            seen += 1
            # four waves, one a SIMD; LDS is given out in pieces of 1280 bytes
            assert -(-k[".group_segment_fixed_size"] // 1280) * 1280 <= LDS // 2, key
            assert -(-k[".vgpr_count"] // 8) * 8 <= REGISTERS // 2, key
    assert seen == 6


def test_spilled_registers_of_the_latent_kernels():
    """Only blocks of 64 and 128 rows of up to 512 columns spill, and no more than the constants of
    a unit and of tiles that not every row sees: what is reloaded on the way of every tile waits for
    the loads of the next."""
    for (fp16, e4m3, columns, rows, groups, stages), k in latent_kernels().items():
        allowed = 46 if (columns, rows) == (512, 4) else 0
        assert k[".vgpr_spill_count"] <= allowed, (fp16, e4m3, columns, rows, groups, k)
