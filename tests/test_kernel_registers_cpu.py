"""Kernels whose working arrays are to lie in registers: the built library says how much memory each kernel has per lane."""
import os
import re
import struct
import subprocess

import pytest

import ssm_decode_amd as rs

READELF = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-readelf")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def _code_objects(data):
    """The gfx950 code objects of the library's offload bundles."""
    at = data.find(MAGIC)
    while at >= 0:
        n = struct.unpack_from("<Q", data, at + len(MAGIC))[0]
        entry = at + len(MAGIC) + 8
        for _ in range(n):
            offset, size, length = struct.unpack_from("<QQQ", data, entry)
            target = data[entry + 24:entry + 24 + length].decode()
            entry += 24 + length
            if "gfx950" in target and size:
                yield data[at + offset:at + offset + size]
        at = data.find(MAGIC, at + len(MAGIC))


@pytest.fixture(scope="module")
def scratch(tmp_path_factory):
    """Bytes of scratch per lane of every kernel."""
    if not os.path.exists(READELF):
        pytest.skip("llvm-readelf not available")
    rs.lib()
    with open(rs._lib.LIB_PATH, "rb") as f:
        data = f.read()
    kernels = {}
    for i, code in enumerate(_code_objects(data)):
        path = tmp_path_factory.mktemp("code") / f"{i}.o"
        path.write_bytes(code)
        notes = subprocess.run([READELF, "--notes", str(path)], capture_output=True, text=True, check=True).stdout
        for part in notes.split("- .agpr_count")[1:]:
            kernels[re.search(r"\.name:\s+(\S+)", part).group(1)] = int(re.search(r"\.private_segment_fixed_size:\s+(\d+)", part).group(1))
    assert len(kernels) > 100
    return kernels


@pytest.mark.parametrize("kernel", ["delta_scan_split_kernel", "delta_reverse_split_kernel", "delta_prepare_kernel", "delta_step_kernel",
                                    "qk_norm_kernel", "qk_norm_backward_kernel", "ragged_kernel"])
def test_no_scratch(scratch, kernel):
    named = {k: b for k, b in scratch.items() if kernel in k}
    assert named and not {k: b for k, b in named.items() if b}
