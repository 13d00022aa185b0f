"""The embedding lookup and the table's gradient on the GPU, bit for bit with
the oracle's binary32 arithmetic: every type, odd widths, views with guards,
ids outside the table, runs of one token to many folds, and each path of the
sort."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from oracle import layers as Y  # noqa: E402

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
IDS = {"i32": torch.int32, "i64": torch.int64}
QUIET = {"f32": 0x7FC00000, "f16": 0x7E00, "bf16": 0x7FC0}
I64 = np.iinfo(np.int64)


@pytest.fixture(scope="module")
def gb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_all_reduce_amd as lib
    return lib


def f32(t):
    torch.cuda.synchronize()
    return t.detach().cpu().float().numpy()


def bits(t):
    torch.cuda.synchronize()
    t = t.detach().cpu().contiguous()
    return t.view(torch.int32 if t.element_size() == 4 else torch.int16).numpy()


def same(got, want, kind, what=""):
    """got, a tensor, against float32 values rounded to its type; torch's
    conversion of a NaN has bits of its own, the library's the quiet NaN's."""
    want = torch.from_numpy(np.ascontiguousarray(want))
    nan, want = torch.isnan(want).numpy(), want.to(TYPES[kind])
    a, b = bits(got), bits(want)
    b = np.where(nan, np.array(QUIET[kind], b.dtype), b)
    bad = np.argwhere(a != b)
    assert len(bad) == 0, f"{what}: {len(bad)} of {a.size} differ, first at {bad[0]}: {got[tuple(bad[0])]} " \
                          f"and {want[tuple(bad[0])]}"


class Guarded:
    """A rows x cols view `shift` values into a buffer, `gap` values between
    its rows, everything around it filled."""

    def __init__(self, rows, cols, dtype, shift=0, gap=0, fill=7.0):
        self.fill = fill
        self.buf = torch.full((shift + rows * (cols + gap) + 24,), fill, dtype=dtype, device=DEV)
        self.view = self.buf.as_strided((rows, cols), (cols + gap, 1), shift)

    def check(self):
        self.view.fill_(self.fill)
        assert bool((self.buf == self.fill).all()), "a value outside the view was written"


def draw_ids(rng, tokens, low, high, how):
    if how == "same":
        return np.full(tokens, (low + high) // 2)
    if how == "words":  # the one of rank r about 1 / r times as often as the first
        return low + (np.exp(rng.random(tokens) * np.log(high - low + 1)).astype(np.int64) - 1).clip(0, high - low - 1)
    return rng.integers(low, high, tokens)


# ---------------------------------------------------------------------------
# Lookup
# ---------------------------------------------------------------------------
def look(gb, tokens, vocab, dim, table="f32", out="f32", ids="i64", scale=1.5, first=0, shift=0, gap=0, spread=0,
         seed=0):
    rng = np.random.default_rng(seed)
    t = Guarded(vocab, dim, TYPES[table], shift, gap)
    t.view.copy_(torch.from_numpy(rng.standard_normal((vocab, dim), dtype=np.float32)))
    o = Guarded(tokens, dim, TYPES[out], shift, gap)
    numbers = rng.integers(first - spread, first + vocab + spread, tokens)
    i = torch.from_numpy(numbers).to(IDS[ids]).to(DEV)
    gb.gb_embedding_forward(o.view, t.view, i, scale=scale, first=first)
    same(o.view, Y.lookup(f32(t.view), numbers, scale, first), out, "out")
    o.check()


@pytest.mark.parametrize("dim", [1, 2, 3, 7, 8, 9, 63, 64, 65, 255, 1001, 4099])
@pytest.mark.parametrize("table,out", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16"),
                                       ("bf16", "f32"), ("f16", "f32"), ("f32", "f16"), ("f16", "bf16"),
                                       ("bf16", "f16")])
def test_lookup_widths_and_types(gb, dim, table, out):
    look(gb, 37, 29, dim, table, out, ids="i32" if dim % 2 else "i64", scale=dim ** 0.5, seed=dim)


@pytest.mark.parametrize("tokens", [1, 2, 63, 257, 5000])
@pytest.mark.parametrize("shift,gap", [(0, 0), (1, 0), (3, 5), (0, 1)])
def test_lookup_of_views_and_shards(gb, tokens, shift, gap):
    for kind, ids in (("f32", "i64"), ("bf16", "i32"), ("f16", "i64")):
        look(gb, tokens, 101, 77, kind, kind, ids, first=1000, shift=shift, gap=gap, spread=200, seed=tokens)


@pytest.mark.parametrize("scale", [0.0, -2.0, 1e-30, 3e38])
def test_lookup_scales(gb, scale):
    look(gb, 50, 40, 33, "f32", "f32", scale=scale)
    look(gb, 50, 40, 33, "f16", "f16", scale=min(scale, 100.0))


def test_lookup_without_tokens_rows_or_width(gb):
    out = torch.full((4, 8), 7.0, device=DEV)
    gb.gb_embedding_forward(out[:0], torch.zeros(3, 8, device=DEV), torch.zeros(0, dtype=torch.int64, device=DEV))
    assert bool((out == 7).all())
    gb.gb_embedding_forward(out, torch.zeros(0, 8, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV))
    assert bool((out == 0).all())
    gb.gb_embedding_forward(out[:, :0], torch.zeros(3, 0, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV))


def extreme_ids(first, vocab):
    return np.array([first, first - 1, first + vocab - 1, first + vocab, I64.min, I64.max, 0, -1, I64.max - 1,
                     -(1 << 32), 1 << 32, (1 << 32) + first, first + 1])


@pytest.mark.parametrize("first", [0, 5, -(1 << 62), I64.max - 20, I64.min])
def test_ids_at_the_ends_of_their_type(gb, first):
    vocab, dim = 11, 9
    first = int(first)
    numbers = np.array([v for v in (int(x) for x in extreme_ids(first, vocab)) if I64.min <= v <= I64.max], np.int64) \
        if first in (0, 5) else np.array([first, first + 1, first + vocab - 1, first + vocab, 0, -1, I64.max, I64.min],
                                         dtype=object).astype(np.int64)
    rng = np.random.default_rng(1)
    table = torch.from_numpy(rng.standard_normal((vocab, dim), dtype=np.float32)).to(DEV)
    out = torch.full((len(numbers), dim), 7.0, device=DEV)
    i = torch.from_numpy(numbers).to(DEV)
    gb.gb_embedding_forward(out, table, i, scale=2.0, first=first)
    same(out, Y.lookup(f32(table), numbers, 2.0, first), "f32")
    grad = torch.full((vocab, dim), 7.0, device=DEV)
    ws = torch.empty(gb.gb_embedding_workspace_bytes(len(numbers), vocab, dim), dtype=torch.uint8, device=DEV)
    gb.gb_embedding_backward(grad, out.fill_(1.0), i, scale=2.0, first=first, padding=first + 1, workspace=ws)
    want, _ = Y.table_gradient(np.ones((len(numbers), dim), np.float32), numbers, vocab, 2.0, first, first + 1)
    same(grad, want, "f32")


def test_values_that_are_not_finite(gb):
    inf, nan = np.inf, np.nan
    table = torch.tensor([[inf, -inf, nan, -0.0], [1.0, 2.0, 3.0, 4.0]], device=DEV)
    i = torch.tensor([0, 1, 9, 0], device=DEV)
    for kind in TYPES:
        t, out = table.to(TYPES[kind]), torch.empty(4, 4, dtype=TYPES[kind], device=DEV)
        gb.gb_embedding_forward(out, t, i, scale=0.0)
        same(out, Y.lookup(f32(t), i.cpu().numpy(), 0.0), kind)
        # rows of an id left out are not looked at, whatever they hold
        dout = torch.tensor([[inf, nan, 1.0, -0.0], [inf, -inf, nan, 5.0], [nan] * 4, [-inf, 1.0, 1.0, -0.0]],
                            dtype=TYPES[kind], device=DEV)
        grad = torch.empty(2, 4, dtype=TYPES[kind], device=DEV)
        ws = torch.empty(gb.gb_embedding_workspace_bytes(4, 2, 4), dtype=torch.uint8, device=DEV)
        gb.gb_embedding_backward(grad, dout, i, padding=1, workspace=ws)
        want, _ = Y.table_gradient(f32(dout), i.cpu().numpy(), 2, 1.0, padding=1)
        same(grad, want, kind)


# ---------------------------------------------------------------------------
# The table's gradient
# ---------------------------------------------------------------------------
def grad(gb, tokens, vocab, dim, how="words", kind="f32", into="f32", ids="i64", scale=0.75, first=0, padding=-1,
         accumulate=False, shift=0, gap=0, spread=0, seed=0):
    rng = np.random.default_rng(seed + tokens)
    d = Guarded(tokens, dim, TYPES[kind], shift, gap)
    d.view.copy_(torch.from_numpy(rng.standard_normal((tokens, dim), dtype=np.float32)))
    t = Guarded(vocab, dim, TYPES[into], shift, gap)
    t.view.copy_(torch.from_numpy(rng.standard_normal((vocab, dim), dtype=np.float32)))
    old = f32(t.view)
    numbers = draw_ids(rng, tokens, first - spread, first + vocab + spread, how)
    i = torch.from_numpy(numbers).to(IDS[ids]).to(DEV)
    need = gb.gb_embedding_workspace_bytes(tokens, vocab, dim)
    ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    gb.gb_embedding_backward(t.view, d.view, i, scale=scale, first=first, padding=padding, accumulate=accumulate,
                             workspace=ws[:need])
    want, _ = Y.table_gradient(f32(d.view), numbers, vocab, scale, first, padding, old if accumulate else None)
    same(t.view, want, into, f"{tokens} tokens, {vocab} rows of {dim}, {how}")
    t.check()
    assert bool((ws[need:] == 0xA5).all()), "the workspace's end was passed"


@pytest.mark.parametrize("how", ["uniform", "same", "words"])
@pytest.mark.parametrize("tokens", [1, 2, 3, 63, 64, 65, 66, 127, 128, 129, 130, 191, 1000, 4095, 4096, 4097, 8191,
                                    8192, 8193, 12289])
def test_gradient_lengths(gb, tokens, how):
    grad(gb, tokens, 300, 5, how, accumulate=tokens % 2 == 1)


@pytest.mark.parametrize("vocab", [1, 2, 3, 64, 1023, 1024, 1025, 70_001, 1 << 20, (1 << 20) + 1])
@pytest.mark.parametrize("tokens", [500, 9000])
def test_gradient_vocabularies(gb, vocab, tokens):
    grad(gb, tokens, vocab, 3, "uniform" if vocab > 4 else "words")


@pytest.mark.parametrize("dim", [1, 2, 7, 8, 9, 255, 256, 257, 511, 513, 1030])
@pytest.mark.parametrize("kind,into", [("f32", "f32"), ("bf16", "f32"), ("f16", "f32"), ("bf16", "bf16"),
                                       ("f16", "f16"), ("f32", "bf16"), ("f32", "f16"), ("f16", "bf16"),
                                       ("bf16", "f16")])
def test_gradient_widths_and_types(gb, dim, kind, into):
    for accumulate in (False, True):
        grad(gb, 400, 50, dim, "words", kind, into, "i32", accumulate=accumulate, seed=dim)


@pytest.mark.parametrize("shift,gap", [(1, 0), (3, 5), (0, 1), (2, 64)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_of_views_shards_and_padding(gb, shift, gap, accumulate):
    for kind, into in (("f32", "f32"), ("bf16", "f32"), ("f16", "f16")):
        for tokens in (200, 9001):
            grad(gb, tokens, 90, 77, "uniform", kind, into, first=500, padding=530, spread=40, shift=shift, gap=gap,
                 accumulate=accumulate)


@pytest.mark.parametrize("tokens", [4096, 4097, 64 * 64 * 3 + 5, 262_144, 262_145, 300_001])
def test_gradient_of_one_row_over_several_levels(gb, tokens):
    """262,144 = 64^3 tokens of one row: the sums of sums of sums."""
    grad(gb, tokens, 2, 3, "same")
    grad(gb, tokens, 2, 3, "words", kind="bf16", accumulate=True)


def test_gradient_runs_against_the_windows(gb):
    """Runs of every length around one and two folds, so that each begins at
    every place of a window."""
    lengths = [1, 62, 63, 64, 65, 66, 127, 128, 129, 130, 2, 192, 193, 1, 1, 64, 64, 65, 65, 5, 300]
    numbers = np.concatenate([np.full(n, r) for r, n in enumerate(lengths * 4)])
    vocab, dim = len(lengths) * 4 + 3, 6
    rng = np.random.default_rng(3)
    dout = rng.standard_normal((len(numbers), dim), dtype=np.float32)
    ws = torch.empty(gb.gb_embedding_workspace_bytes(len(numbers), vocab, dim), dtype=torch.uint8, device=DEV)
    for order in (np.arange(len(numbers)), rng.permutation(len(numbers))):
        out = torch.full((vocab, dim), 7.0, device=DEV)
        gb.gb_embedding_backward(out, torch.from_numpy(dout).to(DEV), torch.from_numpy(numbers[order]).to(DEV),
                                 workspace=ws)
        same(out, Y.table_gradient(dout, numbers[order], vocab, 1.0)[0], "f32")


def test_gradient_without_tokens(gb):
    out = torch.full((300, 17), 7.0, device=DEV)
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    gb.gb_embedding_backward(out, torch.zeros(0, 17, device=DEV), none, accumulate=True)
    assert bool((out == 7).all())
    gb.gb_embedding_backward(out, torch.zeros(0, 17, device=DEV), none)
    assert bool((out == 0).all())
    # all tokens left out
    out.fill_(7.0)
    ids = torch.full((9000,), 4, dtype=torch.int32, device=DEV)
    ws = torch.empty(gb.gb_embedding_workspace_bytes(9000, 300, 17), dtype=torch.uint8, device=DEV)
    gb.gb_embedding_backward(out, torch.ones(9000, 17, device=DEV), ids, padding=4, accumulate=True, workspace=ws)
    assert bool((out == 7).all())
    gb.gb_embedding_backward(out, torch.ones(9000, 17, device=DEV), ids, padding=4, workspace=ws)
    assert bool((out == 0).all())


def test_gradient_of_a_broadcast_input(gb):
    """One row of dout for every token (a stride of 0)."""
    ids = torch.tensor([1, 1, 2, 1], device=DEV)
    out = torch.empty(3, 40, device=DEV)
    ws = torch.empty(gb.gb_embedding_workspace_bytes(4, 3, 40), dtype=torch.uint8, device=DEV)
    gb.gb_embedding_backward(out, torch.ones(1, 40, device=DEV).expand(4, 40), ids, workspace=ws)
    assert out[:, 0].tolist() == [0.0, 3.0, 1.0] and bool((out == out[:, :1]).all())


def test_offsets_beyond_32_bits(gb):
    """A table of more than 2^32 values, its last rows looked up and given
    gradients, and zeros in all rows between."""
    vocab, dim = (1 << 20) + 3, 4100
    table = torch.zeros(vocab, dim, dtype=torch.bfloat16, device=DEV)
    table[-2:] = 3.0
    ids = torch.tensor([vocab - 1, vocab - 2, 0, vocab], device=DEV)
    out = torch.empty(4, dim, dtype=torch.bfloat16, device=DEV)
    gb.gb_embedding_forward(out, table, ids, scale=2.0)
    assert out[:, 0].tolist() == [6.0, 6.0, 0.0, 0.0] and bool((out == out[:, :1]).all())
    ws = torch.empty(gb.gb_embedding_workspace_bytes(4, vocab, dim), dtype=torch.uint8, device=DEV)
    gb.gb_embedding_backward(table, out, ids, accumulate=True, workspace=ws)
    assert table[-3:, 0].tolist() == [0.0, 9.0, 9.0] and bool((table[-2:] == 9.0).all())
    gb.gb_embedding_backward(table, out, ids, workspace=ws)
    assert table[-3:, -1].tolist() == [0.0, 6.0, 6.0]
    assert int(torch.count_nonzero(table[:-2])) == 0
