"""The host code of a Mamba-2 layer's calls under AddressSanitizer and UndefinedBehaviorSanitizer (built host-only)."""
import os

import pytest

from test_prompt_sanitizers import ROCM, ROOT, _run


def test_layer_abi_host_code_under_asan_ubsan(tmp_path):
    hipcc, clang = os.path.join(ROCM, "bin", "hipcc"), os.path.join(ROCM, "llvm", "bin", "clang++")
    if not (os.path.exists(hipcc) and os.path.exists(clang)):
        pytest.skip("ROCm compilers not available")
    flags = ["-x", "hip", "--cuda-host-only", "--offload-arch=gfx950", "-std=c++17", "-O1", "-g",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=all",
             "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "ssm_decode_amd", "csrc")]
    objs = []
    for src in (os.path.join(ROOT, "ssm_decode_amd", "csrc", "api_layer.cpp"), os.path.join(ROOT, "tests", "sanitize", "layer_driver.cpp")):
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        rc, out = _run([hipcc] + flags + ["-c", src, "-o", objs[-1]])
        assert rc == 0, out
    exe = str(tmp_path / "layer_san")
    rc, out = _run([clang, "-fsanitize=address,undefined", "-o", exe] + objs +
                   ["-L", os.path.join(ROCM, "lib"), "-lamdhip64", "-Wl,-rpath," + os.path.join(ROCM, "lib")])
    assert rc == 0, out
    rc, out = _run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1"))
    assert rc == 0 and "failures=0" in out, out
