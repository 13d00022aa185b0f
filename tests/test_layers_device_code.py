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


def spills(text):
    """(vector registers, bytes of scratch) that each kernel spills."""
    found = {}
    for part in re.findall(r"^  - \.agpr_count.*?\.wavefront_size", text, re.M | re.S):
        value = {key: re.search(rf"\.{key}:\s+(\S+)", part).group(1)
                 for key in ("name", "vgpr_spill_count", "private_segment_fixed_size")}
        found[value["name"]] = int(value["vgpr_spill_count"]), int(value["private_segment_fixed_size"])
    return found


def test_only_the_widest_rows_spill(compiled):
    """The layer norm's lanes hold K vectors of 16 bytes.  32 columns a lane
    spill forward and backward; backward 16 columns spill 3 registers at most;
    nothing else does."""
    for name, (registers, scratch) in spills(compiled["gb_embed.hip"][0]).items():
        assert (registers, scratch) == (0, 0), name
    seen = 0
    for name, (registers, scratch) in spills(compiled["gb_norm.hip"][0]).items():
        m = re.search(r"(norm_kernel|norm_grad_kernel)ILi(\d)ELi\d+ELi\d+ELi(\d)E", name)
        columns = int(m.group(3)) * (4 if m.group(2) == "0" else 8) if m else 0
        seen += columns > 0
        if columns == 16 and m.group(1) == "norm_grad_kernel":
            assert registers <= 3 and scratch <= 16, name
        elif columns < 32:
            assert (registers, scratch) == (0, 0), name
    assert seen == 2 * (12 + 11 + 11)
