"""Layer norm of finite rows whose sums or squares pass binary32: what is
stored where, and the bits of every NaN."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from tests.test_gpu_embedding import QUIET, TYPES, bits  # noqa: E402

DEV = "cuda:0"


@pytest.fixture(scope="module")
def gb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_all_reduce_amd as lib
    return lib


# the largest bfloat16 is 1/256 below binary32's largest: a deviation passes that in rows of up to 255 columns
@pytest.mark.parametrize("kind,cols", [("f32", 3), ("f32", 64), ("f32", 300), ("f32", 5000), ("f32", 20_001),
                                       ("bf16", 3), ("bf16", 8), ("bf16", 100), ("bf16", 255)])
def test_forward_of_finite_rows_beyond_binary32(gb, kind, cols):
    t = TYPES[kind]
    big = torch.finfo(t).max
    g = torch.Generator(device=DEV).manual_seed(cols)
    x = torch.randn(9, cols, generator=g, device=DEV).to(t)
    w, b = (torch.randn(cols, generator=g, device=DEV) for _ in range(2))
    clean, y = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(9, device=DEV), torch.empty(9, device=DEV)
    gb.gb_layer_norm_forward(clean, x, w, b)
    # the sum is -big, the mean -big / cols, and the first deviation beyond binary32
    x[1] = 0
    x[1, :3] = torch.tensor([big, -big, -big], device=DEV).to(t)
    # squares beyond binary32, deviations far from it
    x[3] = 0
    x[3, 0], x[3, 1] = 1e20, -1e20
    # a sum beyond binary32
    x[5] = big
    # a NaN among large values
    x[7] = big / 4
    x[7, cols - 1] = float("nan")
    gb.gb_layer_norm_forward(y, x, w, b, mean=mean, rstd=rstd)
    assert torch.equal(y[::2], clean[::2])
    assert bool(torch.isfinite(mean[[1, 3]]).all()) and bool((rstd[[1, 3]] == 0).all())
    assert abs(float(mean[1]) * cols / big + 1) < 1e-5
    bias = b.to(t)
    assert torch.equal(y[1, 1:], bias[1:]) and torch.equal(y[3], bias)
    assert (bits(y[1, :1]) == QUIET[kind]).all()
    assert float(mean[5]) == float("inf") and (bits(y[5]) == QUIET[kind]).all()
    assert (bits(y[7]) == QUIET[kind]).all() and (bits(mean[7:8]) == 0x7FC00000).all()
    assert (bits(rstd[7:8]) == 0x7FC00000).all()
