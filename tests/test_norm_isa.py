"""Registers and scratch of the block norm's and the fp8b format's kernels, from the
metadata of the built library's gfx950 code (host only)."""

import os
import re
import struct
import subprocess

import pytest

import sparse_dense_gemm_amd as sdg

LLVM = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects(data):
    """The gfx950 objects of a library: bundles of (offset, size, name) entries."""
    at = data.find(MAGIC)
    while at >= 0:
        n, pos = struct.unpack_from("<Q", data, at + 24)[0], at + 32
        for _ in range(n):
            offset, size, length = struct.unpack_from("<QQQ", data, pos)
            name, pos = data[pos + 24:pos + 24 + length], pos + 24 + length
            if name.endswith(b"gfx950") and size:
                yield data[at + offset:at + offset + size]
        at = data.find(MAGIC, at + 32)


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Name -> (bytes a lane in scratch, vector registers)."""
    readelf = os.path.join(LLVM, "llvm-readelf")
    if not os.path.exists(readelf):
        pytest.skip("llvm-readelf not available")
    found, folder = {}, tmp_path_factory.mktemp("objects")
    with open(sdg.LIB_PATH, "rb") as f:
        objects = list(code_objects(f.read()))
    assert objects
    for i, o in enumerate(objects):
        path = folder / f"{i}.o"
        path.write_bytes(o)
        t = subprocess.run([readelf, "--notes", str(path)], capture_output=True, text=True).stdout
        for block in re.split(r"- \.agpr_count:", t)[1:]:
            field = lambda f: re.search(rf"\.{f}:\s+(\S+)", block).group(1)
            found[field("name")] = int(field("private_segment_fixed_size")), int(field("vgpr_count"))
    return found


def test_norm(kernels):
    """Rows in one piece a thread and long rows keep nothing in scratch; rows in four pieces 116 bytes a lane at most, and
    nothing where O and the residual are bf16."""
    norms = {n: k for n, k in kernels.items() if re.search(r"norm(_long)?_kernelI", n)}
    four = [n for n in norms if "Li4EEE" in n]
    assert len(norms) == 80 and len(four) == 32
    for name, (scratch, registers) in norms.items():
        assert registers <= 128, name  # 16 waves of a workgroup fit a CU
        assert scratch <= (116 if name in four and "norm_kernelItt" not in name else 0), (name, scratch)


def test_format(kernels):
    of = [n for n in kernels if re.search(r"quantize_(rows|blocks)_kernel|dequantize_kernel", n)]
    assert len(of) >= 10
    for name in of:
        assert kernels[name][0] == 0, name
