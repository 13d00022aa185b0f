"""Layer norm on the GPU, forward and backward: against binary64 within bounds
derived from the roundings, and, over integers that make every sum exact, the
weight's and the bias' gradients value for value."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from oracle import layers as Y  # noqa: E402
from tests.test_gpu_embedding import Guarded, QUIET, TYPES, bits, f32  # noqa: E402

DEV = "cuda:0"
EPS = 1e-5
# around every change of the number of lanes, wavefronts and vectors that hold a row
WIDTHS = [1, 2, 3, 7, 8, 9, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 771, 1023, 1024, 1025,
          2047, 2048, 2049, 4095, 4096, 4097, 8191, 8192, 8193, 12289, 16383, 16384, 16385, 32767, 32768]


@pytest.fixture(scope="module")
def gb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_all_reduce_amd as lib
    return lib


def close(got, want, bound, kind, what):
    got = f32(got).astype(np.float64)
    limit = bound + Y.rounding(np.abs(want) + bound, kind)
    bad = np.argwhere(~(np.abs(got - want) <= limit))
    assert len(bad) == 0, f"{what}: {len(bad)} of {got.size} beyond the bound, first at {bad[0]}: " \
                          f"{got[tuple(bad[0])]} and {want[tuple(bad[0])]}, bound {limit[tuple(bad[0])]}"


def inputs(rng, rows, cols, kind, shift=0, gap=0):
    x = Guarded(rows, cols, TYPES[kind], shift, gap)
    values = rng.standard_normal((rows, cols), dtype=np.float32) * np.exp(rng.standard_normal((rows, 1))) + 0.5
    x.view.copy_(torch.from_numpy(values.astype(np.float32)))
    return x


def vector(rng, n, kind, shift=0, centre=0.0):
    v = Guarded(1, n, TYPES[kind], shift)
    v.view.copy_(torch.from_numpy((centre + 0.3 * rng.standard_normal((1, n))).astype(np.float32)))
    return v


def forward(gb, rows, cols, kind="f32", param="f32", shift=0, gap=0, weight=True, bias=True, stats=True, seed=0):
    rng = np.random.default_rng(seed + cols)
    x, y = inputs(rng, rows, cols, kind, shift, gap), Guarded(rows, cols, TYPES[kind], shift, gap + 1)
    w = vector(rng, cols, param, shift, 1.0).view[0] if weight else None
    b = vector(rng, cols, param, shift).view[0] if bias else None
    mean, rstd = (Guarded(1, rows, torch.float32) if stats else None for _ in range(2))
    gb.gb_layer_norm_forward(y.view, x.view, w, b, EPS, mean and mean.view[0], rstd and rstd.view[0])
    want, m, r, e_y, e_m, e_r = Y.norm(f32(x.view), None if w is None else f32(w), None if b is None else f32(b), EPS)
    what = f"{rows} x {cols} {kind}"
    close(y.view, want, e_y, kind, what)
    y.check()
    if stats:
        close(mean.view[0], m, e_m, "f32", what + " mean")
        close(rstd.view[0], r, e_r, "f32", what + " rstd")
        mean.check()
        rstd.check()


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("kind,param", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16")])
def test_forward_widths(gb, cols, kind, param):
    forward(gb, 5 if cols > 600 else 133, cols, kind, param)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 31, 32, 33, 1000, 8191, 70_001])
@pytest.mark.parametrize("kind,param", [("f32", "bf16"), ("bf16", "bf16"), ("f16", "f32")])
def test_forward_lengths(gb, rows, kind, param):
    forward(gb, rows, 40, kind, param)
    if rows < 10_000:
        forward(gb, rows, 700, kind, param, bias=False)


@pytest.mark.parametrize("shift,gap", [(1, 0), (3, 5), (0, 1), (2, 64)])
@pytest.mark.parametrize("kind", list(TYPES))
def test_forward_of_views(gb, shift, gap, kind):
    for cols in (13, 128, 777, 4100):
        forward(gb, 37, cols, kind, kind, shift, gap, weight=cols != 13, stats=cols != 128)


@pytest.mark.parametrize("kind", list(TYPES))
def test_forward_in_place_and_into_more_dimensions(gb, kind):
    rng = np.random.default_rng(0)
    x = inputs(rng, 24, 300, kind).view.contiguous()
    y = torch.empty_like(x)
    gb.gb_layer_norm_forward(y, x)
    cube = x.clone().view(2, 3, 4, 300)
    gb.gb_layer_norm_forward(cube, cube)
    assert torch.equal(cube.view(24, 300), y)
    row = x[3].clone()
    gb.gb_layer_norm_forward(row, row)
    assert torch.equal(row, y[3])
    same_row = torch.empty_like(x)
    gb.gb_layer_norm_forward(same_row, x[3:4].expand(24, 300))
    assert torch.equal(same_row, y[3:4].expand(24, 300))


def test_forward_loses_nothing_to_a_large_mean(gb):
    """Rows of mean 4096 and deviation 1/16: a sum of squares less the square
    of the sum would keep no digit of the variance."""
    rng = np.random.default_rng(0)
    x = torch.from_numpy((4096 + rng.integers(-4, 5, (64, 1000)) / 16).astype(np.float32)).to(DEV)
    y = torch.empty_like(x)
    gb.gb_layer_norm_forward(y, x)
    want, _, _, e_y, _, _ = Y.norm(f32(x), None, None, EPS)
    close(y, want, e_y, "f32", "a large mean")


def test_forward_of_rows_that_are_constant_or_not_finite(gb):
    for kind in TYPES:
        for cols in (5, 300, 5000):
            x = torch.randn(7, cols, device=DEV).to(TYPES[kind])
            clean, y = torch.empty_like(x), torch.empty_like(x)
            mean, rstd = torch.empty(7, device=DEV), torch.empty(7, device=DEV)
            gb.gb_layer_norm_forward(clean, x)
            x[0] = 3.0  # no variance: y is 0, rstd 1 / sqrt(eps)
            x[2, cols // 2] = float("nan")
            x[4, 0] = float("inf")
            x[6, cols - 1] = -float("inf")
            gb.gb_layer_norm_forward(y, x, eps=EPS, mean=mean, rstd=rstd)
            assert bool((y[0] == 0).all()) and abs(float(rstd[0]) * EPS ** 0.5 - 1) < 1e-6
            for r in (1, 3, 5):
                assert torch.equal(y[r], clean[r])
            assert (bits(y[2]) == QUIET[kind]).all() and (bits(mean[2:3]) == 0x7FC00000).all()
            for r in (4, 6):  # an infinity leaves an infinite mean and no number
                assert bool(torch.isnan(y[r]).all()) and bool(torch.isinf(mean[r]))


def backward(gb, rows, cols, kind="f32", param="f32", into="f32", accumulate=False, shift=0, gap=0, weight=True,
             alias=None, seed=0):
    rng = np.random.default_rng(seed + cols)
    x, dy = inputs(rng, rows, cols, kind, shift, gap), inputs(rng, rows, cols, kind, shift, gap)
    w = vector(rng, cols, param, shift, 1.0).view[0] if weight else None
    dx = {None: Guarded(rows, cols, TYPES[kind], shift, gap + 1), "dy": dy, "x": x}[alias]
    dw, db = vector(rng, cols, into, shift), vector(rng, cols, into, shift)
    xs, dys = f32(x.view), f32(dy.view)
    old = [f32(v.view[0]).astype(np.float64) * accumulate for v in (dw, db)]
    _, m, r, _, _, _ = Y.norm(xs, None, None, EPS)
    mean, rstd = (torch.from_numpy(v.astype(np.float32)).to(DEV) for v in (m, r))
    need = gb.gb_layer_norm_workspace_bytes(rows, cols)
    ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    gb.gb_layer_norm_backward(dx.view, dw.view[0], db.view[0], dy.view, x.view, mean, rstd, w, accumulate, ws[:need])
    wdx, wdw, wdb, e_dx, e_dw, e_db = Y.norm_gradients(dys, xs, f32(mean), f32(rstd), None if w is None else f32(w))
    what = f"{rows} x {cols} {kind}"
    close(dx.view, wdx, e_dx, kind, what + " dx")
    for got, want, e, o, name in ((dw, wdw, e_dw, old[0], "dw"), (db, wdb, e_db, old[1], "db")):
        close(got.view[0], want + o, e + 2 * Y.U * np.abs(want + o), into, f"{what} {name}")
        got.check()
    dx.check()
    assert bool((ws[need:] == 0xA5).all()), "the workspace's end was passed"


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("kind,param", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16")])
def test_backward_widths(gb, cols, kind, param):
    backward(gb, 5 if cols > 600 else 133, cols, kind, param, accumulate=cols % 2 == 1)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 31, 32, 33, 1000, 8191, 70_001])
@pytest.mark.parametrize("kind,into", [("f32", "bf16"), ("bf16", "bf16"), ("f16", "f32"), ("f16", "f16")])
def test_backward_lengths(gb, rows, kind, into):
    backward(gb, rows, 40, kind, kind, into)
    if rows < 10_000:
        backward(gb, rows, 700, kind, "f32", into, accumulate=True, weight=False)


@pytest.mark.parametrize("shift,gap", [(1, 0), (3, 5), (0, 1), (2, 64)])
@pytest.mark.parametrize("kind", list(TYPES))
def test_backward_of_views_and_in_place(gb, shift, gap, kind):
    for cols, alias in ((13, None), (128, "dy"), (777, "x"), (4100, "dy")):
        backward(gb, 37, cols, kind, kind, shift=shift, gap=gap, alias=alias)


EXACT = [(1, 1), (3, 5), (64, 8), (100, 13), (1000, 64), (4096, 128), (5000, 257), (7001, 130), (33, 1000),
         (2049, 771), (515, 2050), (3000, 513), (700, 4097), (1500, 8200), (600, 16384), (513, 32768), (20_000, 24)]


@pytest.mark.parametrize("rows,cols", EXACT)
@pytest.mark.parametrize("kind", list(TYPES))
def test_parameter_gradients_of_integers_are_exact(gb, rows, cols, kind):
    """mean 1, rstd 2, small integers: every product and sum is a whole number
    below 2^24, so any order gives the same bits, and a value left out or
    taken twice shows."""
    rng = np.random.default_rng(rows + cols)
    x, dy = (rng.integers(-3, 4, (rows, cols)) for _ in range(2))
    dw, db = torch.full((cols,), 5.0, device=DEV), torch.full((cols,), -4.0, device=DEV)
    ws = torch.empty(gb.gb_layer_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    d = [torch.from_numpy(v.astype(np.float32)).to(DEV).to(TYPES[kind]) for v in (dy, x)]
    mean, rstd = torch.full((rows,), 1.0, device=DEV), torch.full((rows,), 2.0, device=DEV)
    for accumulate in (False, True):
        gb.gb_layer_norm_backward(None, dw, db, *d, mean, rstd, accumulate=accumulate, workspace=ws)
        times = 2 if accumulate else 1
        assert (f32(dw) == times * (dy * (x - 1) * 2).sum(0)).all()
        assert (f32(db) == times * dy.sum(0)).all()
    # one of them alone leaves the other be
    dw.fill_(5.0)
    gb.gb_layer_norm_backward(None, None, db, *d, mean, rstd, workspace=ws)
    assert (f32(db) == dy.sum(0)).all() and bool((dw == 5.0).all())
    db.fill_(5.0)
    dx = torch.empty_like(d[0])
    gb.gb_layer_norm_backward(dx, dw, None, *d, mean, rstd, workspace=ws)
    assert (f32(dw) == (dy * (x - 1) * 2).sum(0)).all() and bool((db == 5.0).all())
    alone = torch.empty_like(dx)
    gb.gb_layer_norm_backward(alone, None, None, *d, mean, rstd)
    assert torch.equal(alone, dx)


def test_backward_repeats_bit_for_bit(gb):
    for rows, cols, kind in ((5003, 1000, "bf16"), (900, 8192, "f32"), (20_000, 64, "f16")):
        x, dy = (torch.randn(rows, cols, device=DEV).to(TYPES[kind]) for _ in range(2))
        mean, rstd = torch.randn(rows, device=DEV), torch.rand(rows, device=DEV)
        got = []
        for fill in (0, 255):
            dw, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
            ws = torch.full((gb.gb_layer_norm_workspace_bytes(rows, cols),), fill, dtype=torch.uint8, device=DEV)
            dx = torch.empty_like(x)
            gb.gb_layer_norm_backward(dx, dw, db, dy, x, mean, rstd, workspace=ws)
            got.append((dx, dw, db))
        assert all(torch.equal(a, b) for a, b in zip(*got))


def test_backward_without_rows(gb):
    none, stat = torch.zeros(0, 9, device=DEV), torch.zeros(0, device=DEV)
    dw, db = torch.full((9,), 5.0, device=DEV), torch.full((9,), 5.0, device=DEV)
    gb.gb_layer_norm_backward(none, dw, db, none, none, stat, stat, accumulate=True)
    assert bool((dw == 5).all()) and bool((db == 5).all())
    gb.gb_layer_norm_backward(none, dw, db, none, none, stat, stat)
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_backward_of_rows_that_are_not_finite(gb):
    """A row without a number spoils its own dx and the sums it is part of, and
    no other row; large means do not reach the columns beyond a row's end."""
    for kind in TYPES:
        for cols in (5, 300, 5001):
            rows = 9
            x, dy = (torch.randn(rows, cols, device=DEV).to(TYPES[kind]) for _ in range(2))
            mean, rstd = torch.zeros(rows, device=DEV), torch.ones(rows, device=DEV)
            ws = torch.empty(gb.gb_layer_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
            clean, dx = torch.empty_like(x), torch.empty_like(x)
            dw, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
            gb.gb_layer_norm_backward(clean, dw, db, dy, x, mean, rstd, workspace=ws)
            dy[4, cols // 2] = float("nan")
            gb.gb_layer_norm_backward(dx, dw, db, dy, x, mean, rstd, workspace=ws)
            assert (bits(dx[4]) == QUIET[kind]).all()
            keep = [r for r in range(rows) if r != 4]
            assert torch.equal(dx[keep], clean[keep])
            assert torch.isnan(dw).nonzero().flatten().tolist() == [cols // 2]
            assert torch.isnan(db).nonzero().flatten().tolist() == [cols // 2]
            # x is constant, h is 0: the product of mean and rstd alone is beyond binary32
            big = torch.full((rows, cols), 2.0 ** 15, device=DEV).to(TYPES[kind])
            mean.fill_(2.0 ** 15)
            rstd.fill_(2.0 ** 120)
            dy.fill_(0.0)
            gb.gb_layer_norm_backward(dx, dw, db, dy, big, mean, rstd, workspace=ws)
            assert bool((dx == 0).all()) and bool((dw == 0).all())


def test_offsets_beyond_32_bits(gb):
    """More than 2^32 values, and more than 2^32 between two rows."""
    rows, cols = (1 << 21) + 3, 2049
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    some = [0, 1, rows // 2, (1 << 32) // cols, (1 << 32) // cols + 1, rows - 2, rows - 1]
    x[some] = torch.randn(len(some), cols, device=DEV).bfloat16()
    y = torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    gb.gb_layer_norm_forward(y, x, mean=mean, rstd=rstd)
    few = x[some].contiguous()
    want, m, r = torch.empty_like(few), torch.empty(len(some), device=DEV), torch.empty(len(some), device=DEV)
    gb.gb_layer_norm_forward(want, few, mean=m, rstd=r)
    assert torch.equal(y[some], want) and torch.equal(mean[some], m) and torch.equal(rstd[some], r)
    y[some] = 0
    assert int(torch.count_nonzero(y)) == 0
    # dy is 1 in those rows alone
    y[some] = 1
    dx, dw, db = x, torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    ws = torch.empty(gb.gb_layer_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    gb.gb_layer_norm_backward(dx, dw, db, y, x, mean, rstd, workspace=ws)
    assert bool((db == len(some)).all())
    want_dx, want_dw = torch.empty_like(few), torch.empty(cols, device=DEV)
    gb.gb_layer_norm_backward(want_dx, want_dw, None, torch.ones_like(few), few, m, r, workspace=ws)
    assert torch.equal(dx[some], want_dx)
    assert bool(((dw - want_dw).abs() <= 2.0 ** -18 * len(some)).all())
    del x, y, dx
    # two rows more than 2^32 apart
    far = torch.zeros((1 << 32) + 64, dtype=torch.float16, device=DEV).as_strided((2, 50), ((1 << 32) + 7, 1))
    far.copy_(few[:2, :50])
    out = torch.empty(2, 50, dtype=torch.float16, device=DEV)
    gb.gb_layer_norm_forward(out, far)
    near = torch.empty_like(out)
    gb.gb_layer_norm_forward(near, far.contiguous())
    assert torch.equal(out, near) and bool((out[1] != 0).any())
