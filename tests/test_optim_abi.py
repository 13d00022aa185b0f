"""The optimizer calls' host side, without a GPU: sizes, and every refusal,
each before anything is enqueued."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def gb():
    import gradient_all_reduce_amd as lib
    return lib


def test_constants_and_structures_match_the_header(gb):
    text = open(os.path.join(ROOT, "include", "gbreduce.h")).read()
    for name in ("GB_OPTIM_CONTROL_BYTES", "GB_OPTIM_MAX_TENSORS"):
        assert getattr(gb, name) == int(re.search(rf"#define {name} (\d+)", text).group(1))
    for name in ("GB_STATE_F32", "GB_STATE_E4M3"):
        assert getattr(gb, name) == int(re.search(rf"\b{name} = (\d+)", text).group(1))
    assert ctypes.sizeof(gb._OptimTensor) == 88 and ctypes.sizeof(gb._OptimHandle) == 192
    assert [f[0] for f in gb._OptimTensor._fields_] == ["n", "param", "grad", "copy", "m", "v", "m_scale", "v_scale",
                                                       "dtype", "copy_dtype", "state", "reserved", "lr_scale", "weight_decay"]


def test_plan_bytes(gb):
    one = gb.gb_optim_plan_bytes([1])
    assert one > 0 and gb.gb_optim_plan_bytes([]) > 0
    assert gb.gb_optim_plan_bytes([1] * 1000) > one
    assert gb.gb_optim_plan_bytes([1 << 30]) > gb.gb_optim_plan_bytes([1 << 20])
    assert gb.gb_optim_plan_bytes([gb.GB_MAX_N + 1]) == 0
    assert gb.gb_optim_plan_bytes([gb.GB_MAX_N, 1]) == 0
    assert gb._lib.gb_optim_plan_bytes(None, 1) == 0
    assert gb._lib.gb_optim_plan_bytes(None, -1) == 0
    assert gb._lib.gb_optim_plan_bytes(None, gb.GB_OPTIM_MAX_TENSORS + 1) == 0


# made-up device addresses: a refused call looks at none of them
GOOD = dict(n=1000, param=0x100000, grad=0x200000, copy=None, m=0x300000, v=0x400000, m_scale=None, v_scale=None,
            dtype=0, copy_dtype=0, state=0, reserved=0, lr_scale=1.0, weight_decay=0.0)
CODED = dict(GOOD, m_scale=0x500000, v_scale=0x600000, state=1)


def plan(gb, tensors, workspace=0x900000, workspace_bytes=None, beta1=0.9, beta2=0.999, eps=1e-8, handle=True,
         count=None, table=True):
    arr = (gb._OptimTensor * max(1, len(tensors)))(
        *[gb._OptimTensor(*[t[f[0]] for f in gb._OptimTensor._fields_]) for t in tensors])
    need = gb.gb_optim_plan_bytes([t["n"] for t in tensors])
    h = gb._OptimHandle()
    return gb._lib.gb_optim_plan(ctypes.byref(h) if handle else None, arr if table else None,
                                 len(tensors) if count is None else count, beta1, beta2, eps, 0, workspace,
                                 need if workspace_bytes is None else workspace_bytes, None)


INV, MIS, UNS, WS = 1, 2, 3, 4
CASES = [
    ("a NULL handle", lambda gb: plan(gb, [GOOD], handle=False), INV, "plan is NULL"),
    ("a negative count", lambda gb: plan(gb, [GOOD], count=-1), INV, "count = -1"),
    ("too many tensors", lambda gb: plan(gb, [GOOD], count=gb.GB_OPTIM_MAX_TENSORS + 1), INV, "outside 0.."),
    ("a NULL table", lambda gb: plan(gb, [GOOD], table=False), INV, "tensors is NULL"),
    ("beta1 = 1", lambda gb: plan(gb, [GOOD], beta1=1.0), INV, "beta1"),
    ("beta2 below 0", lambda gb: plan(gb, [GOOD], beta2=-0.1), INV, "beta2"),
    ("beta2 NaN", lambda gb: plan(gb, [GOOD], beta2=float("nan")), INV, "beta2"),
    ("eps 0", lambda gb: plan(gb, [GOOD], eps=0.0), INV, "eps"),
    ("eps 0 in binary32", lambda gb: plan(gb, [GOOD], eps=1e-60), INV, "eps"),
    ("eps infinite", lambda gb: plan(gb, [GOOD], eps=float("inf")), INV, "eps"),
    ("too many values", lambda gb: plan(gb, [dict(GOOD, n=gb.GB_MAX_N), GOOD]), INV, "exceed GB_MAX_N"),
    ("a NULL workspace", lambda gb: plan(gb, [GOOD], workspace=None), WS, "workspace"),
    ("a small workspace", lambda gb: plan(gb, [GOOD], workspace_bytes=100), WS, "100 bytes"),
    ("a misaligned workspace", lambda gb: plan(gb, [GOOD], workspace=0x900010), MIS, "workspace"),
    ("a float64 gradient", lambda gb: plan(gb, [dict(GOOD, dtype=3)]), UNS, "tensors[0].dtype"),
    ("an integer gradient", lambda gb: plan(gb, [GOOD, dict(GOOD, dtype=6)]), UNS, "tensors[1].dtype"),
    ("an unknown state", lambda gb: plan(gb, [dict(GOOD, state=2)]), UNS, "state"),
    ("an infinite lr_scale", lambda gb: plan(gb, [dict(GOOD, lr_scale=float("inf"))]), INV, "lr_scale"),
    ("a NaN weight decay", lambda gb: plan(gb, [dict(GOOD, weight_decay=float("nan"))]), INV, "weight_decay"),
    ("scales of float32 moments", lambda gb: plan(gb, [dict(GOOD, m_scale=0x500000)]), INV, "scales"),
    ("codes without a scale", lambda gb: plan(gb, [dict(CODED, v_scale=None)]), INV, "v_scale is NULL"),
    ("a misaligned scale", lambda gb: plan(gb, [dict(CODED, v_scale=0x600002)]), MIS, "v_scale"),
    ("a float32 copy", lambda gb: plan(gb, [dict(GOOD, copy=0x700000)]), UNS, "copy"),
    ("a misaligned copy", lambda gb: plan(gb, [dict(GOOD, copy_dtype=2, copy=0x700001)]), MIS, "copy"),
    ("a copy of an unknown type", lambda gb: plan(gb, [dict(GOOD, copy_dtype=9, copy=0x700000)]), UNS, "copy_dtype"),
    ("moments off 16 bytes", lambda gb: plan(gb, [dict(GOOD, m=0x300004)]), MIS, "m = "),
    ("codes off 16 bytes", lambda gb: plan(gb, [dict(CODED, v=0x400001)]), MIS, "v = "),
    ("a parameter off its element", lambda gb: plan(gb, [dict(GOOD, param=0x100002)]), MIS, "param"),
    ("a gradient off its element", lambda gb: plan(gb, [dict(GOOD, grad=0x200001, dtype=1)]), MIS, "grad"),
    ("a gradient over its parameter", lambda gb: plan(gb, [dict(GOOD, grad=0x100004)]), INV, "overlaps"),
    ("two tensors in one buffer", lambda gb: plan(gb, [GOOD, GOOD]), INV, "overlaps"),
    ("a moment in the workspace", lambda gb: plan(gb, [dict(GOOD, m=0x900100)]), INV, "overlaps"),
    ("scales over codes", lambda gb: plan(gb, [dict(CODED, m_scale=0x300100)]), INV, "overlaps"),
    ("a copy over the gradient", lambda gb: plan(gb, [dict(GOOD, copy_dtype=2, copy=0x200002)]), INV, "overlaps"),
] + [(f"a NULL {f}", lambda gb, f=f: plan(gb, [dict(GOOD, **{f: None})]), INV, f"{f} is NULL")
     for f in ("param", "grad", "m", "v")]


@pytest.mark.parametrize("name,call,status,text", CASES, ids=[c[0].replace(" ", "_") for c in CASES])
def test_plan_refusals(gb, name, call, status, text):
    assert call(gb) == status
    assert gb.gb_last_error().startswith("gb_optim_plan: ") and text in gb.gb_last_error()


def test_step_calls_refuse_what_is_no_plan_and_bad_arguments(gb):
    L = gb._lib
    bad = gb._OptimHandle()
    for call in (lambda h, c: L.gb_optim_begin(h, c, 1.0, None), lambda h, c: L.gb_adamw_step(h, c, None),
                 lambda h, c: L.gb_optim_begin_clip(h, c, 1.0, 1.0, None)):
        assert call(None, 0x1000) == INV and "not made by gb_optim_plan" in gb.gb_last_error()
        assert call(ctypes.byref(bad), 0x1000) == INV and "not made by gb_optim_plan" in gb.gb_last_error()
    # a handle as gb_optim_plan leaves it, of no tensors: the other arguments come next
    made = gb._OptimHandle()
    made.opaque[0] = 0x67626F7074696D31
    h = ctypes.byref(made)
    assert L.gb_optim_begin(h, None, 1.0, None) == INV and "control is NULL" in gb.gb_last_error()
    assert L.gb_adamw_step(h, 0x1004, None) == MIS and "control" in gb.gb_last_error()
    for scale in (0.0, -1.0, float("nan"), float("inf"), 1e-60, 1e60):
        assert L.gb_optim_begin(h, 0x1000, scale, None) == INV and "inv_scale" in gb.gb_last_error()
        assert L.gb_optim_begin_clip(h, 0x1000, 1.0, scale, None) == INV
    for norm in (0.0, -1.0, float("nan")):
        assert L.gb_optim_begin_clip(h, 0x1000, norm, 1.0, None) == INV and "max_norm" in gb.gb_last_error()


def test_the_binding_refuses_host_tensors_and_wrong_types(gb):
    import torch
    x = torch.zeros(8)
    with pytest.raises(ValueError, match=r"tensors\[0\].param must be in device memory"):
        gb.gb_optim_plan([gb.GbOptimTensor(x, x, x, x)], torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="control"):
        gb.gb_optim_control(torch.zeros(64, dtype=torch.uint8))



class OnAnotherDevice:
    """What a control block in another GPU's memory looks like to the binding."""
    dtype, is_cuda = None, True

    def __init__(self, torch):
        self.dtype, self.device = torch.uint8, torch.device("cuda", 1)

    numel = staticmethod(lambda: 64)
    is_contiguous = staticmethod(lambda: True)
    get_device = staticmethod(lambda: 1)
    data_ptr = staticmethod(lambda: 0x1000)


def made_plan(gb):
    """A plan of no tensors on GPU 0, as gb_optim_plan leaves one."""
    import torch
    handle = gb._OptimHandle()
    handle.opaque[0] = 0x67626F7074696D31

    class Workspace:
        device = torch.device("cuda", 0)
    return gb.GbOptimPlan(handle, [], Workspace)


def test_the_step_calls_refuse_a_control_block_of_another_device(gb):
    import torch
    control, plan = OnAnotherDevice(torch), made_plan(gb)
    for call in (gb.gb_optim_begin, lambda p, c: gb.gb_optim_begin_clip(p, c, 1.0), gb.gb_adamw_step):
        with pytest.raises(ValueError, match="control is on cuda:1, the plan on cuda:0"):
            call(plan, control)


def test_the_step_calls_refuse_a_control_block_inside_the_workspace(gb):
    """The tables there hold the addresses that the kernels follow."""
    L = gb._lib
    made = gb._OptimHandle()
    table, chunks, partials = 0x900000, 0x900100, 0x900200
    end = partials + 1024 * 8
    for word, value in enumerate((0x67626F7074696D31, table, chunks, partials)):
        made.opaque[word] = value
    h = ctypes.byref(made)
    for control in (table, chunks + 16, table - 16, partials, end - 16):
        for call in (lambda c: L.gb_optim_begin(h, c, 1.0, None), lambda c: L.gb_adamw_step(h, c, None),
                     lambda c: L.gb_optim_begin_clip(h, c, 1.0, 1.0, None)):
            assert call(control) == INV, hex(control)
            assert "control overlaps workspace" in gb.gb_last_error()
    for control in (table - 64, end):  # beside it: refused only for want of a scale
        assert L.gb_optim_begin(h, control, 0.0, None) == INV and "inv_scale" in gb.gb_last_error()


def test_the_current_stream_is_found_without_torchs_private_lookup():
    """A torch without torch._C._cuda_getCurrentRawStream: the public one serves."""
    code = """if True:
        import types, torch
        del torch._C._cuda_getCurrentRawStream
        import gradient_all_reduce_amd as gb
        asked = []
        def current_stream(device):
            asked.append(device)
            return types.SimpleNamespace(cuda_stream=0x1234)
        torch.cuda.current_stream = current_stream
        plan = types.SimpleNamespace(device_index=3)
        assert gb._plan_stream(plan, None) == 0x1234 and asked == [3]
        assert gb._plan_stream(plan, types.SimpleNamespace(cuda_stream=5)) == 5 and asked == [3]
        """
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
