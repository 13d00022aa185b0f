"""The token-sum layers' launches at the documented limits, on the CPU:
gb_norm.hip and gb_embed.hip compiled for the host alone, with stand-ins for
the HIP runtime's launch calls that record every grid."""
import os
import shutil
import subprocess

import pytest

from gradient_all_reduce_amd import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DRIVER = os.path.join(ROOT, "tests", "sanitize", "launch_driver.cpp")


def test_every_launch_of_the_documented_sizes_fits(tmp_path):
    """A launch of 2^32 lanes or more is refused by the runtime, after the
    launches before it are enqueued; the table's sums come to more workgroups
    than that for 2^30 rows of few columns, and for 2^30 tokens."""
    if not os.path.exists(B.HIPCC) or shutil.which("g++") is None or not os.path.exists(DRIVER):
        pytest.skip("needs hipcc, g++ and the driver")
    objects = []
    for name in ("gb_norm.hip", "gb_embed.hip", "gb_layers_api.cpp", DRIVER):
        path = os.path.join(B.CSRC, name)  # DRIVER's is absolute
        objects.append(str(tmp_path / (os.path.basename(name) + ".o")))
        if name.endswith(".hip"):
            command = [B.HIPCC, "-x", "hip", "--offload-arch=gfx950", "--offload-host-only"]
        else:
            command = ["g++", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include"]
        r = subprocess.run([*command, "-O1", "-std=c++17", "-Wall", "-I", B.INCLUDE, "-c", path, "-o", objects[-1]],
                           capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr
    exe = str(tmp_path / "launches")
    # the device code, which is not here, is the only symbol left open
    r = subprocess.run(["g++", *objects, "-Wl,--unresolved-symbols=ignore-in-object-files", "-no-pie", "-o", exe],
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and " 0 failed" in out.stdout, out.stdout[-4000:] + out.stderr
