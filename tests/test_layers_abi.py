"""The token-sum layers' host side, without a GPU: sizes, and every refusal,
each before anything is enqueued."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, MIS, UNS, WS = 1, 2, 3, 4
F32, F16, BF16, F64, I32, I64 = 0, 1, 2, 3, 6, 7
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def gb():
    import gradient_all_reduce_amd as lib
    return lib


def test_constants_match_the_header(gb):
    text = open(os.path.join(ROOT, "include", "gbreduce.h")).read()
    for name in ("GB_NORM_MAX_COLS", "GB_EMBEDDING_MAX_TOKENS", "GB_EMBEDDING_MAX_VOCAB", "GB_EMBEDDING_MAX_DIM"):
        value = re.search(rf"#define {name} \(?([\d< ]+)\)?", text).group(1)
        assert getattr(gb, name) == eval(value)


def test_workspace_bytes(gb):
    norm, table = gb.gb_layer_norm_workspace_bytes, gb.gb_embedding_workspace_bytes
    assert norm(0, 100) == 0 and norm(1, 1) > 0
    assert norm(10, 0) == norm(10, gb.GB_NORM_MAX_COLS + 1) == norm(gb.GB_MAX_N, 2) == 0
    # grows with the rows until every workgroup has some, and with the columns
    assert norm(1, 100) < norm(100, 100) < norm(1 << 20, 100) == norm(1 << 22, 100) < norm(1 << 20, 1000)
    assert norm(1 << 20, 4096) < 64 << 20
    assert table(0, 10, 10) == table(10, 0, 10) == table(10, 10, 0) == 0
    assert table(gb.GB_EMBEDDING_MAX_TOKENS + 1, 1, 1) == table(1, gb.GB_EMBEDDING_MAX_VOCAB + 1, 1) == 0
    assert table(1, 1, gb.GB_EMBEDDING_MAX_DIM + 1) == table(1 << 30, 1, 1 << 20) == table(1, 1 << 30, 1 << 20) == 0
    assert 0 < table(1, 1, 1) < table(100, 1, 1) <= table(8192, 1, 1) < table(8193, 1, 1)
    assert table(100, 1 << 20, 4) - table(100, 1, 4) >= (1 << 20) - 256


# made-up device addresses: a refused call looks at none of them
def forward(gb, dtype=BF16, y=0x10000000, y_stride=100, x=0x20000000, x_stride=100, rows=50, cols=100, param=F32,
            w=0x30000000, b=0x31000000, eps=1e-5, mean=0x32000000, rstd=0x33000000):
    return gb._lib.gb_layer_norm_forward(dtype, y, y_stride, x, x_stride, rows, cols, param, w, b, eps, mean, rstd,
                                         None)


def backward(gb, dtype=BF16, dx=0x10000000, dx_stride=100, dy=0x20000000, dy_stride=100, x=0x28000000, x_stride=100,
             rows=50, cols=100, mean=0x32000000, rstd=0x33000000, param=F32, w=0x30000000, grad=F32, dw=0x34000000,
             db=0x35000000, accumulate=0, ws=0x40000000, ws_bytes=1 << 30):
    return gb._lib.gb_layer_norm_backward(dtype, dx, dx_stride, dy, dy_stride, x, x_stride, rows, cols, mean, rstd,
                                          param, w, grad, dw, db, accumulate, ws, ws_bytes, None)


def look(gb, out_type=BF16, out=0x10000000, out_stride=64, table_type=F32, table=0x20000000, table_stride=64,
         vocab=1000, dim=64, id_type=I64, ids=0x30000000, tokens=300, first=0, scale=1.0):
    return gb._lib.gb_embedding_forward(out_type, out, out_stride, table_type, table, table_stride, vocab, dim,
                                        id_type, ids, tokens, first, scale, None)


def grad(gb, grad_type=F32, dtable=0x10000000, dtable_stride=64, vocab=1000, dim=64, dtype=BF16, dout=0x20000000,
         dout_stride=64, id_type=I64, ids=0x30000000, tokens=300, first=0, padding=-1, scale=1.0, accumulate=0,
         ws=0x40000000, ws_bytes=1 << 30):
    return gb._lib.gb_embedding_backward(grad_type, dtable, dtable_stride, vocab, dim, dtype, dout, dout_stride,
                                         id_type, ids, tokens, first, padding, scale, accumulate, ws, ws_bytes, None)


N = 1 << 39
CASES = [(forward, k, s, t) for k, s, t in [
    (dict(dtype=F64), UNS, "dtype = 3"), (dict(param=I32), UNS, "param_dtype"), (dict(cols=0), INV, "cols = 0"),
    (dict(cols=32769), INV, "outside 1.."), (dict(cols=(1 << 32) + 1), INV, "cols"),
    (dict(rows=N, cols=2), INV, "GB_MAX_N"),
    (dict(eps=0.0), INV, "eps"), (dict(eps=-1.0), INV, "eps"), (dict(eps=NAN), INV, "eps"), (dict(eps=INF), INV, "eps"),
    (dict(eps=1e-60), INV, "eps"), (dict(eps=1e60), INV, "eps"), (dict(y=None), INV, "y is NULL"),
    (dict(x=None), INV, "x is NULL"), (dict(y=0x10000001), MIS, "y = "), (dict(x=0x20000001), MIS, "x = "),
    (dict(dtype=F32, x=0x20000002), MIS, "x = "), (dict(w=0x30000002), MIS, "weight"),
    (dict(b=0x31000001), MIS, "bias"),
    (dict(mean=0x32000002), MIS, "mean"), (dict(rstd=0x33000001), MIS, "rstd"),
    (dict(y_stride=99), INV, "y_stride = 99"),
    (dict(x_stride=N), INV, "x_stride"), (dict(y=0x20000002), INV, "overlaps"),
    (dict(y=0x20000000, y_stride=101), INV, "overlaps"),
    (dict(mean=0x33000000), INV, "overlaps"), (dict(w=0x32000004), INV, "overlaps"),
    (dict(b=0x10000010), INV, "overlaps"),
]] + [(backward, k, s, t) for k, s, t in [
    (dict(dtype=I32), UNS, "dtype"), (dict(param=F64), UNS, "param_dtype"), (dict(grad=F64), UNS, "grad_dtype"),
    (dict(cols=0), INV, "cols"), (dict(rows=N), INV, "GB_MAX_N"), (dict(accumulate=2), INV, "accumulate = 2"),
    (dict(dx=None, dw=None, db=None), INV, "all NULL"), (dict(dy=None), INV, "dy is NULL"),
    (dict(x=None), INV, "x is NULL"),
    (dict(mean=None), INV, "mean is NULL"), (dict(rstd=None), INV, "rstd is NULL"), (dict(dx=0x10000001), MIS, "dx"),
    (dict(dw=0x34000002), MIS, "dweight"), (dict(db=0x35000001), MIS, "dbias"), (dict(dx_stride=10), INV, "dx_stride"),
    (dict(dy_stride=N), INV, "dy_stride"), (dict(ws=None), WS, "workspace"), (dict(ws_bytes=100), WS, "100 bytes"),
    (dict(ws=0x40000008), MIS, "workspace"), (dict(dx=0x20000002), INV, "overlaps"),
    (dict(dx=0x28000000, dx_stride=101), INV, "overlaps"), (dict(dw=0x35000004), INV, "overlaps"),
    (dict(dw=0x30000000), INV, "overlaps"), (dict(ws=0x20000000), INV, "overlaps"),
    (dict(db=0x40000010), INV, "overlaps"),
    (dict(mean=0x34000000), INV, "overlaps"),
]] + [(look, k, s, t) for k, s, t in [
    (dict(out_type=F64), UNS, "out_dtype"), (dict(table_type=I64), UNS, "table_dtype"),
    (dict(id_type=F32), UNS, "id_dtype"),
    (dict(tokens=(1 << 30) + 1), INV, "beyond"), (dict(vocab=1 << 31), INV, "beyond"),
    (dict(dim=(1 << 20) + 1), INV, "beyond"),
    (dict(tokens=1 << 30, dim=1 << 10), INV, "GB_MAX_N"), (dict(vocab=1 << 30, dim=1 << 10), INV, "GB_MAX_N"),
    (dict(ids=None), INV, "ids is NULL"), (dict(ids=0x30000004), MIS, "ids"), (dict(out=None), INV, "out is NULL"),
    (dict(table=None), INV, "table is NULL"), (dict(out=0x10000001), MIS, "out"),
    (dict(table=0x20000002), MIS, "table"),
    (dict(out_stride=63), INV, "out_stride"), (dict(table_stride=N), INV, "table_stride"),
    (dict(scale=NAN), INV, "scale"),
    (dict(scale=INF), INV, "scale"), (dict(scale=1e60), INV, "scale"), (dict(first=(1 << 63) - 1000), INV, "first"),
    (dict(out=0x20000004), INV, "overlaps"), (dict(ids=0x10000010), INV, "overlaps"),
]] + [(grad, k, s, t) for k, s, t in [
    (dict(grad_type=F64), UNS, "grad_dtype"), (dict(dtype=I64), UNS, "dtype"), (dict(id_type=BF16), UNS, "id_dtype"),
    (dict(tokens=(1 << 30) + 1), INV, "beyond"), (dict(scale=-INF), INV, "scale"),
    (dict(accumulate=-1), INV, "accumulate"),
    (dict(first=(1 << 63) - 500), INV, "first"), (dict(ids=None), INV, "ids is NULL"),
    (dict(dtable=None), INV, "dtable is NULL"),
    (dict(dout=None), INV, "dout is NULL"), (dict(dtable=0x10000002), MIS, "dtable"),
    (dict(dout=0x20000001), MIS, "dout"),
    (dict(dtable_stride=63), INV, "dtable_stride"), (dict(dout_stride=N), INV, "dout_stride"),
    (dict(ws=None), WS, "workspace"),
    (dict(ws_bytes=10), WS, "10 bytes"), (dict(ws=0x40000004), MIS, "workspace"),
    (dict(dtable=0x20000000), INV, "overlaps"),
    (dict(ids=0x40000000), INV, "overlaps"), (dict(ws=0x10000000), INV, "overlaps"),
]]


@pytest.mark.parametrize("call,arguments,status,text", CASES,
                         ids=[f"{c[0].__name__}-{'-'.join(f'{k}={v}' for k, v in c[1].items())}" for c in CASES])
def test_refusals(gb, call, arguments, status, text):
    assert call(gb, **arguments) == status
    name = {forward: "layer_norm_forward", backward: "layer_norm_backward", look: "embedding_forward",
            grad: "embedding_backward"}[call]
    assert gb.gb_last_error().startswith(f"gb_{name}: ") and text in gb.gb_last_error(), gb.gb_last_error()


def test_calls_with_nothing_to_do_are_ok(gb):
    assert forward(gb, rows=0, x=None, y=None, mean=None, rstd=None) == 0
    assert backward(gb, rows=0, dw=None, db=None, dx=None, dy=None, x=None) == 0
    assert backward(gb, rows=0, accumulate=1, dy=None, x=None, ws=None, ws_bytes=0) == 0
    assert look(gb, tokens=0, out=None, ids=None) == 0 and look(gb, dim=0, out=None, ids=None, table=None) == 0
    assert grad(gb, tokens=0, accumulate=1, dout=None, ids=None, ws=None, ws_bytes=0) == 0
    assert grad(gb, vocab=0, dtable=None) == 0 and grad(gb, dim=0, dtable=None, ids=None) == 0


def test_the_binding_refuses_what_the_library_cannot_see(gb):
    import torch
    x, ids = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="x must be in device memory"):
        gb.gb_layer_norm_forward(x, x)
    with pytest.raises(TypeError, match="x must be a tensor of one of"):
        gb.gb_layer_norm_backward(x, x, x, x, x.double(), x, x)
    with pytest.raises(TypeError, match="table must be a torch.Tensor"):
        gb.gb_embedding_forward(x, None, ids)
    with pytest.raises(ValueError, match="dtable must be in device memory"):
        gb.gb_embedding_backward(x, x, ids)


class On:
    """What the binding sees of a tensor on a GPU of its own choosing."""

    def __new__(cls, torch, shape, dtype, device=0, stride=None):
        t = torch.empty(shape, dtype=dtype, device="meta")
        if stride is not None:
            t = t.as_strided(shape, stride)

        class Fake(torch.Tensor):
            def get_device(self):
                return device
        return t.as_subclass(Fake)


def test_the_binding_refuses_shapes_types_and_devices_that_do_not_match(gb):
    import torch
    f, h, i = torch.float32, torch.float16, torch.int64
    x = On(torch, (4, 8), f)
    cases = [
        (lambda: gb.gb_layer_norm_forward(On(torch, (4, 9), f), x), ValueError, "y has 4 rows of 9 values"),
        (lambda: gb.gb_layer_norm_forward(On(torch, (4, 8), h), x), TypeError, "y must be torch.float32"),
        (lambda: gb.gb_layer_norm_forward(On(torch, (4, 8), f, 1), x), ValueError, "y is on"),
        (lambda: gb.gb_layer_norm_forward(x, On(torch, (4, 8), f, 0, (1, 4))), ValueError, "x must be 2-D"),
        (lambda: gb.gb_layer_norm_forward(x, x, On(torch, (7,), f)), ValueError, "weight has 7 elements"),
        (lambda: gb.gb_layer_norm_forward(x, x, On(torch, (8,), f), On(torch, (8,), h)), TypeError, "bias must be"),
        (lambda: gb.gb_layer_norm_forward(x, x, mean=On(torch, (4,), h)), TypeError, "mean must be"),
        (lambda: gb.gb_layer_norm_forward(x, x, rstd=On(torch, (5,), f)), ValueError, "rstd has 5"),
        (lambda: gb.gb_layer_norm_backward(x, On(torch, (8,), f, 0, (2,)), None, x, x, None, None), ValueError,
         "dweight must be contiguous"),
        (lambda: gb.gb_layer_norm_backward(None, None, None, x, x, None, None, workspace=On(torch, (8,), f)), TypeError,
         "workspace"),
        (lambda: gb.gb_embedding_forward(x, x, On(torch, (4,), f)), TypeError, "ids must be"),
        (lambda: gb.gb_embedding_forward(x, x, On(torch, (5,), i)), ValueError, "out has 4 rows"),
        (lambda: gb.gb_embedding_forward(x, x, On(torch, (4,), i, 1)), ValueError, "ids is on"),
        (lambda: gb.gb_embedding_backward(x, On(torch, (4, 7), f), On(torch, (4,), i)), ValueError, "dout has"),
        (lambda: gb.gb_embedding_backward(x, x, On(torch, (4,), i, 0, (2,))), ValueError, "ids must be contiguous"),
        (lambda: gb.gb_embedding_forward(x, x, On(torch, (4,), i), first=1 << 63), ValueError, "first = .* 64-bit"),
        (lambda: gb.gb_embedding_backward(x, x, On(torch, (4,), i), padding=-(1 << 63) - 1), ValueError, "padding ="),
    ]
    for call, error, text in cases:
        with pytest.raises(error, match=text):
            call()


def test_no_workload_runs_the_layers_that_the_kernel_hash_leaves_out():
    """bench.py's hash of the kernel sources leaves gb_norm.hip and
    gb_embed.hip out, since no workload runs them."""
    text = open(os.path.join(ROOT, "bench.py")).read() + open(os.path.join(ROOT, "workloads.py")).read()
    assert "gb_norm.hip" in text and "gb_embed.hip" in text
    assert not re.findall(r"gb_(?:layer_norm|embedding)_\w+", text)
