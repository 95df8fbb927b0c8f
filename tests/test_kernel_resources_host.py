"""Registers and scratch of kernels in the built library, from the notes of its
code objects: what a kernel's launch counts on."""
import os
import re
import struct
import subprocess

import pytest

mod = pytest.importorskip("expert_grouping_dispatch_amd")
READELF = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-readelf")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Kernel name -> (vector registers, bytes of scratch a lane)."""
    data, found, at = open(mod.LIB_PATH, "rb").read(), {}, 0
    path = str(tmp_path_factory.mktemp("code") / "object")
    while (at := data.find(MAGIC, at)) >= 0:
        n, = struct.unpack_from("<Q", data, at + len(MAGIC))
        entry = at + len(MAGIC) + 8
        for _ in range(n):
            offset, size, length = struct.unpack_from("<QQQ", data, entry)
            target = data[entry + 24:entry + 24 + length]
            entry += 24 + length
            if b"gfx950" not in target or size == 0:
                continue
            with open(path, "wb") as f:
                f.write(data[at + offset:at + offset + size])
            notes = subprocess.run([READELF, "--notes", path], capture_output=True, text=True, check=True).stdout
            for k in re.split(r"\n +- \.agpr_count:", notes)[1:]:
                name = re.search(r"\.name: +(\S+)", k[k.index(".max_flat_workgroup_size"):]).group(1)
                found[name] = (int(re.search(r"\.vgpr_count: +(\d+)", k).group(1)),
                               int(re.search(r"\.private_segment_fixed_size: +(\d+)", k).group(1)))
        at += len(MAGIC)
    return found


def _of(kernels, *parts):
    got = {k: v for k, v in kernels.items() if all(p in k for p in parts)}
    assert got, parts
    return got


def test_few_rows_in_int8_have_four_waves_a_simd(kernels):
    """512 registers a lane of a SIMD: 128 for each of four waves, so that 1024 workgroups are on the GPU at once."""
    for name, (registers, scratch) in _of(kernels, "k_matmul_few", "MatI8").items():
        assert registers <= 128 and scratch == 0, (name, registers, scratch)


@pytest.mark.parametrize("parts", [("k_matmul_",), ("k_few_",), ("k_quantize_",), ("k_dispatch_f8",), ("k_dispatch_i8",)])
def test_kernels_of_the_products_keep_to_registers(kernels, parts):
    for name, (_, scratch) in _of(kernels, *parts).items():
        assert scratch == 0, (name, scratch)
