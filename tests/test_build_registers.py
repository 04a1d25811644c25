"""Registers of built kernels whose launch counts on two workgroups of a compute unit, read from the library's own code
objects (no GPU)."""
import pathlib
import struct

import pytest

msgpack = pytest.importorskip("msgpack")


def kernels(path):
    """The metadata of every kernel in the code objects that the library holds, by name."""
    data, found, at = pathlib.Path(path).read_bytes(), {}, 0
    while (at := data.find(b"\x7fELF", at + 1)) > 0:
        if struct.unpack_from("<H", data, at + 18)[0] != 224:  # EM_AMDGPU
            continue
        off, = struct.unpack_from("<Q", data, at + 32)
        size, count = struct.unpack_from("<HH", data, at + 54)
        for i in range(count):
            head = at + off + i * size
            kind, = struct.unpack_from("<I", data, head)
            start, = struct.unpack_from("<Q", data, head + 8)
            length, = struct.unpack_from("<Q", data, head + 32)
            if kind != 4:  # PT_NOTE
                continue
            name, desc, note = struct.unpack_from("<III", data, at + start)
            body = at + start + 12 + (name + 3) // 4 * 4
            if note == 32 and desc <= length:  # NT_AMDGPU_METADATA
                for k in msgpack.unpackb(data[body:body + desc]).get("amdhsa.kernels", []):
                    found[k[".name"]] = k
    return found


@pytest.fixture(scope="module")
def built():
    import grouped_mixed_input_amd as g

    if not g.LIB_PATH.exists():
        from grouped_mixed_input_amd import build

        build.build()
    return kernels(g.LIB_PATH)


@pytest.mark.parametrize("name", ["k_route_place", "k_group_place"])
def test_second_launches_of_1024_threads_share_a_compute_unit(built, name):
    # 512 registers a lane and SIMD serve eight waves of 64; two workgroups of 1024 threads are eight waves a SIMD
    found = [k for n, k in built.items() if name in n]
    assert len(found) == 1
    k = found[0]
    assert k[".max_flat_workgroup_size"] == 1024
    assert k[".vgpr_count"] <= 64 and k[".private_segment_fixed_size"] == 0
    assert 2 * k[".group_segment_fixed_size"] <= 160 * 1024
