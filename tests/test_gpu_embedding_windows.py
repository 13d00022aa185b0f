"""The table's gradient where runs of every length around one and two folds
begin at every place of the 16-token windows, behind both sorts, over several
slabs of columns, written and added: bit for bit with the oracle."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from oracle import layers as Y  # noqa: E402
from tests.test_gpu_embedding import TYPES, f32, same  # noqa: E402

DEV = "cuda:0"
LENGTHS = [1, 62, 63, 64, 65, 66, 127, 128, 129, 130, 2, 192, 193, 1, 1, 64, 64, 65, 65, 5, 300]
# (tokens ahead of the first run, repeats of the lengths); the lengths add up to 1787, 11 more than a multiple of 16
SMALL, LARGE = [(p, 4) for p in (0, 12, 8, 4)], [(0, 16)]


@pytest.fixture(scope="module")
def gb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_all_reduce_amd as lib
    return lib


def runs(ahead, repeats):
    return [ahead] * (ahead > 0) + LENGTHS * repeats


@pytest.mark.parametrize("pieces", [SMALL, LARGE])
def test_every_length_begins_at_every_place(pieces):
    places = {n: set() for n in LENGTHS}
    for ahead, repeats in pieces:
        lengths = runs(ahead, repeats)
        starts = np.cumsum([0] + lengths)
        assert (starts[-1] <= 8192) == (pieces is SMALL)  # one workgroup sorts up to 8192 tokens
        for n, start in list(zip(lengths, starts))[ahead > 0:]:
            places[n].add(int(start) % 16)
    assert all(p == set(range(16)) for p in places.values())


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dim", [6, 520])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("ahead,repeats", SMALL + LARGE)
def test_runs_at_every_place(gb, ahead, repeats, kind, dim, accumulate):
    lengths = runs(ahead, repeats)
    numbers = np.concatenate([np.full(n, r) for r, n in enumerate(lengths)])
    vocab = len(lengths) + 3
    rng = np.random.default_rng(len(numbers) + dim)
    dout = torch.from_numpy(rng.standard_normal((len(numbers), dim), dtype=np.float32)).to(DEV).to(TYPES[kind])
    old = torch.from_numpy(rng.standard_normal((vocab, dim), dtype=np.float32)).to(DEV)
    ws = torch.empty(gb.gb_embedding_workspace_bytes(len(numbers), vocab, dim), dtype=torch.uint8, device=DEV)
    for order in (np.arange(len(numbers)), rng.permutation(len(numbers))):
        out = old.clone()
        gb.gb_embedding_backward(out, dout, torch.from_numpy(numbers[order]).to(DEV), scale=0.75,
                                 accumulate=accumulate, workspace=ws)
        want, _ = Y.table_gradient(f32(dout), numbers[order], vocab, 0.75, old=f32(old) if accumulate else None)
        same(out, want, "f32", f"{ahead} ahead, {dim} columns")
