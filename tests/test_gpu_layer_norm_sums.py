"""The layer norm's weight and bias gradients against binary64, within bounds
that count the additions on a term's way as the kernels make them."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from tests.test_gpu_embedding import TYPES  # noqa: E402

DEV = "cuda:0"


@pytest.fixture(scope="module")
def gb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_all_reduce_amd as lib
    return lib


def additions(rows):
    """At most: a lane's rows in turn (256 workgroups or more where there are
    as many rows, or one row each), 3 between the teams of a wavefront, 15
    between wavefronts, and of up to 1024 workgroups' sums 16 in turn in each
    of 64 slices, whose sums are joined by 7 additions and 7 more."""
    return -(-rows // 256) + 3 + 15 + 16 + 14


@pytest.mark.parametrize("rows,cols", [(70_001, 40), (70_001, 3), (70_001, 8), (20_000, 130), (8191, 700), (4097, 1500),
                                       (3001, 4097), (2000, 8200), (1500, 12_289), (700, 20_000), (257, 513)])
@pytest.mark.parametrize("kind", list(TYPES))
def test_sums_over_the_rows(gb, rows, cols, kind):
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    # values of one sign as well: their sums grow, and a sum that loses to its size shows
    x = (torch.randn(rows, cols, generator=g, device=DEV) + 0.5).to(TYPES[kind])
    dy = (torch.randn(rows, cols, generator=g, device=DEV).abs() + 0.01).to(TYPES[kind])
    mean, rstd = x.float().mean(1), 0.5 + torch.rand(rows, generator=g, device=DEV)
    dw, db = (torch.empty(cols, device=DEV) for _ in range(2))
    ws = torch.empty(gb.gb_layer_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    gb.gb_layer_norm_backward(None, dw, db, dy, x, mean, rstd, workspace=ws)
    d, h = dy.double(), (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    # h has two roundings of its own; a fused product and sum has one, which is the addition's
    for got, terms, steps, name in ((dw, d * h, additions(rows) + 2, "dw"), (db, d, additions(rows), "db")):
        off = (got.double() - terms.sum(0)).abs() - 1.01 * steps * 2.0 ** -24 * terms.abs().sum(0)
        assert float(off.max()) <= 0, f"{name}: column {int(off.argmax())} is {float(off.max())} beyond the bound"
