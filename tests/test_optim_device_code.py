"""What the optimizer's kernels promise the compiler, read from the device IR
that the library's own flags give for gfx950 (CPU only, needs hipcc):
accesses to parameters, gradients and copies assume the alignment of one
element and no more, since these may be views into a bucket; and the lanes
that open a step read the control block before any of them writes it."""
import os
import re
import subprocess

import pytest

from gradient_all_reduce_amd import build as B

# byte offsets of OptimTensor's pointers (gb_optim.h)
FIELDS = {8: "p", 16: "g", 24: "copy", 32: "m", 40: "v", 48: "ms", 56: "vs"}
F32_KERNELS = [f"adamw_f32_kernelILi{t}E" for t in range(3)]
E4M3_KERNELS = [f"adamw_e4m3_kernelILi{t}E" for t in range(3)]
NORM_KERNELS = ["optim_norm_kernelILb0E", "optim_norm_kernelILb1E", "optim_norm_small_kernelE"]


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """The IR of every kernel of gb_optim.hip as a list of lines, by mangled name."""
    if not os.path.exists(B.HIPCC):
        pytest.skip("needs hipcc")
    out = tmp_path_factory.mktemp("ir") / "gb_optim.ll"
    subprocess.run([B.HIPCC, *B.FLAGS, "-x", "hip", "--offload-device-only", "-S", "-emit-llvm",
                    os.path.join(B.CSRC, "gb_optim.hip"), "-o", str(out)], check=True, capture_output=True, timeout=300)
    found = {}
    for part in re.findall(r"^define [^\n]*amdgpu_kernel.*?^}", out.read_text(), re.M | re.S):
        found[re.search(r"@(\w+)\(", part).group(1)] = part.splitlines()
    return found


def kernel(kernels, name):
    match = [body for mangled, body in kernels.items() if name in mangled]
    assert len(match) == 1, name
    return match[0]


def definitions(body):
    return dict(m.groups() for m in (re.match(r"\s+(%[\w.]+) = (.*)", line) for line in body) if m)


def field_of(pointer, defs):
    """The OptimTensor field that a pointer was loaded from, through address
    arithmetic and casts."""
    for _ in range(20):
        d = defs.get(pointer, "")
        if m := re.match(r"load ptr, ptr addrspace\(\d\) (%[\w.]+)", d):
            at = re.search(r"^getelementptr .* i64 (\d+)$", defs.get(m.group(1), ""))
            return FIELDS.get(int(at.group(1))) if at else None
        m = re.match(r"(?:getelementptr [^%]*|addrspacecast )ptr(?: addrspace\(1\))? (%[\w.]+)", d)
        if not m:
            return None
        pointer = m.group(1)
    return None


def vector_accesses(body):
    """(field, bytes, align) of every vector load and store of a kernel through
    a pointer of the plan's table."""
    defs, got = definitions(body), []
    width = {"float": 4, "i32": 4, "half": 2, "bfloat": 2, "i16": 2}
    for line in body:
        m = (re.search(r"= load <(\d+) x (\w+)>, ptr(?: addrspace\(1\))? (%[\w.]+), align (\d+)", line)
             or re.search(r"store <(\d+) x (\w+)> [^,]+, ptr(?: addrspace\(1\))? (%[\w.]+), align (\d+)", line))
        if m:
            field = field_of(m.group(3), defs)
            assert field is not None, f"no field found for: {line.strip()}"
            got.append((field, int(m.group(1)) * width[m.group(2)], int(m.group(4))))
    return got


@pytest.mark.parametrize("name", F32_KERNELS + E4M3_KERNELS + NORM_KERNELS)
def test_views_off_16_bytes_are_accessed_at_their_elements_alignment(kernels, name):
    got = vector_accesses(kernel(kernels, name))
    fields = {f for f, _, _ in got}
    assert {"g"} <= fields if name in NORM_KERNELS else {"p", "g", "copy"} <= fields
    for field, size, align in got:
        if field in ("p", "g", "copy"):
            # 16 bytes are four binary32 values, 8 bytes four of 2 bytes
            assert align == {16: 4, 8: 2}[size], (field, size, align)
        else:
            assert name in F32_KERNELS and field in ("m", "v") and (size, align) == (16, 16)


def test_every_lane_reads_the_step_count_before_one_writes_it(kernels):
    """optim_begin_kernel's lanes all read control->step and one of them adds
    to it: a barrier stands between."""
    body = kernel(kernels, "optim_begin_kernelE")
    loads = [i for i, line in enumerate(body) if re.search(r"= load \w+, ptr addrspace\(1\)", line)]
    stores = [i for i, line in enumerate(body) if re.search(r"^\s+store \w+ [^,]+, ptr addrspace\(1\)", line)]
    barriers = [i for i, line in enumerate(body) if "@llvm.amdgcn.s.barrier()" in line]
    assert loads and stores and barriers
    assert max(loads) < min(barriers) and max(barriers) < min(stores)


def test_lds_reservations_leave_the_workgroups_they_are_named_for():
    """LDS is handed out in granules of 1,280 bytes, 128 to a CU (counted on
    the hardware: 11,520 bytes leave 14 workgroups, 11,521 leave 12)."""
    text = open(os.path.join(B.CSRC, "gb_optim.hip")).read()
    names = {"Eight": 8, "Nine": 9, "Ten": 10, "Eleven": 11, "Twelve": 12, "Fourteen": 14, "Sixteen": 16}
    found = re.findall(r"\bk([A-Z][a-z]+)PerCuLds = ([^,;]+)[,;]", text)
    assert found
    for name, value in found:
        size = eval(re.sub(r"(\d)u\b", r"\1", value), {"kLdsGranule": 1280})
        assert 128 // -(-size // 1280) == names[name], (name, value)
