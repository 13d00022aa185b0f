"""What the compiled kernels of the token-sum layers hold to, read from the
assembly that the library's own flags give for gfx950 (CPU only, needs
hipcc)."""
import concurrent.futures
import os
import re
import subprocess

import pytest

from gradient_all_reduce_amd import build as B

SOURCES = ("gb_norm.hip", "gb_embed.hip")


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    """(assembly, what the compiler printed) of each source."""
    if not os.path.exists(B.HIPCC):
        pytest.skip("needs hipcc")
    out = tmp_path_factory.mktemp("asm")

    def compile_one(name):
        to = out / (name + ".s")
        r = subprocess.run([B.HIPCC, *B.FLAGS, "-x", "hip", "--offload-device-only", "-S", os.path.join(B.CSRC, name),
                            "-o", str(to)], capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr
        return to.read_text(), r.stderr

    with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as pool:
        return dict(zip(SOURCES, pool.map(compile_one, SOURCES)))


def kernels(text):
    """The body of every kernel by its mangled name."""
    return {m.group(1): m.group(2) for m in re.finditer(r"^(_ZN\w+):(.*?)^\.Lfunc_end", text, re.M | re.S)}


@pytest.mark.parametrize("source", SOURCES)
def test_no_access_is_a_flat_one(compiled, source):
    """A flat access may be to LDS or to memory, so it waits for both kinds and
    keeps no order with the LDS instructions, on which the sort's counters
    rely."""
    found = kernels(compiled[source][0])
    assert len(found) > 20
    flat = {name: re.findall(r"^\s+(flat_(?:load|store|atomic)\w*)", body, re.M) for name, body in found.items()}
    assert not {name: ops for name, ops in flat.items() if ops}


@pytest.mark.parametrize("source", SOURCES)
def test_the_compiler_follows_every_request(compiled, source):
    """A pragma that cannot be followed is a warning: a loop whose ballots
    stand under a condition of run time is not unrolled."""
    warnings = [line for line in compiled[source][1].splitlines() if source in line and "warning:" in line]
    assert not warnings
