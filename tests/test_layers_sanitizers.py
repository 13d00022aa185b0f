"""The token-sum layers' C-ABI layer under AddressSanitizer and
UndefinedBehaviorSanitizer on the CPU: built with g++ against the stand-ins of
tests/sanitize/layers_driver.cpp, which write every part of a workspace of
exactly the size the library asks for."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = ["-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer"]
DRIVER = os.path.join(ROOT, "tests", "sanitize", "layers_driver.cpp")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_layers_abi_layer_under_sanitizers(tmp_path):
    if not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h") or not os.path.exists(DRIVER):
        pytest.skip("HIP headers or the driver are not here")
    exe = tmp_path / "layers_driver"
    r = subprocess.run(["g++", "-std=c++17", "-Wall", *SAN, "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I",
                        os.path.join(ROOT, "include"), DRIVER,
                        os.path.join(ROOT, "gradient_all_reduce_amd", "csrc", "gb_layers_api.cpp"), "-o", str(exe)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300,
                         env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1"))
    assert out.returncode == 0 and " 0 failed" in out.stdout, out.stdout + out.stderr
    assert "runtime error" not in out.stderr
