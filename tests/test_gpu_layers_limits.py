"""The embedding calls at their largest vocabularies and numbers of tokens on
the GPU, where a call's work takes several launches."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def gb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_all_reduce_amd as lib
    return lib


def workspace(gb, tokens, vocab, dim):
    return torch.empty(gb.gb_embedding_workspace_bytes(tokens, vocab, dim), dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("vocab", [1 << 30, (1 << 30) + 1, 2_147_483_647])
@pytest.mark.parametrize("tokens", [6, 9006])
def test_gradient_of_the_largest_vocabularies(gb, vocab, tokens):
    """Rows of one value, named at both ends of the table and in the middle;
    every other row is cleared."""
    rows = torch.tensor([0, 1, vocab // 2, vocab - 2, vocab - 1], device=DEV)
    which = torch.arange(tokens, device=DEV) % 6
    ids = torch.where(which < 5, rows[which.clamp(max=4)], vocab)  # the last of six lies beyond the table
    dout = (1 + which).to(torch.float16)[:, None]
    grad = torch.full((vocab, 1), 7.0, dtype=torch.float16, device=DEV)
    gb.gb_embedding_backward(grad, dout, ids, workspace=workspace(gb, tokens, vocab, 1))
    # sums of equal whole numbers up to 5 x 1501: exact in any order, rounded once
    want = ((tokens // 6) * torch.arange(1.0, 6.0, device=DEV)).half()
    assert torch.equal(grad[rows, 0], want)
    grad[rows] = 0
    assert int(torch.count_nonzero(grad)) == 0


@pytest.mark.parametrize("accumulate", [False, True])
def test_the_largest_number_of_tokens(gb, accumulate):
    """2^30 tokens of the value 1 in three rows and one id beyond the table: a
    row's 2^28 tokens are summed over five levels, at each of them 64 equal
    powers of two in turn (16 at the last), so every sum is exact."""
    tokens, vocab = 1 << 30, 3
    ids = torch.arange(tokens, dtype=torch.int32, device=DEV) % 4
    grad = torch.full((vocab, 1), 2.0 ** 24, device=DEV)
    gb.gb_embedding_backward(grad, torch.ones(tokens, 1, dtype=torch.float16, device=DEV), ids, accumulate=accumulate,
                             workspace=workspace(gb, tokens, vocab, 1))
    assert grad[:, 0].tolist() == [2.0 ** 28 + (2.0 ** 24 if accumulate else 0.0)] * 3


def test_lookup_of_the_largest_number_of_tokens(gb):
    tokens = 1 << 30
    ids = torch.arange(tokens, dtype=torch.int32, device=DEV) % 4
    out = torch.full((tokens, 1), 7.0, dtype=torch.float16, device=DEV)
    gb.gb_embedding_forward(out, torch.tensor([[1.0], [2.0], [3.0]], device=DEV), ids, scale=2.0)
    four = out.view(-1, 4)
    for column, value in enumerate((2.0, 4.0, 6.0, 0.0)):
        assert bool((four[:, column] == value).all()), column
