"""The token-sum layers as a program uses them: together in a model whose
gradients land in a bucket, against binary64 and against differences; on
another stream, two calls at once, captured and replayed, and over the
gradients of the same tokens in several micro-batches."""
import math
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

DEV = "cuda:0"


@pytest.fixture(scope="module")
def gb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_all_reduce_amd as lib
    return lib


def plain_loss(p, batches, ex):
    """The example's model in binary64 on the CPU: the sum of the losses."""
    total = 0.0
    for ids, targets in batches:
        x = p["table"][ids] * math.sqrt(ex.WIDTH)

        def norm(x, gain, bias):
            mean = x.mean(-1, keepdim=True)
            var = ((x - mean) ** 2).mean(-1, keepdim=True)
            return (x - mean) / torch.sqrt(var + 1e-5) * gain + bias

        x = x + torch.nn.functional.gelu(norm(x, p["gain1"], p["bias1"]) @ p["mix"].t())
        scores = torch.log_softmax(norm(x, p["gain2"], p["bias2"]) @ p["head"].t(), -1)
        scores = scores.gather(-1, targets[..., None])[..., 0]
        here = targets != ex.PADDING
        total = total - (scores * here).sum() / here.sum()
    return total


def test_a_models_gradients_in_its_bucket(gb):
    """Two micro-batches added up in one flat bucket whose views start at odd
    places.  Every gradient is a chain of about ten operations in binary32,
    each a sum of at most a few hundred terms (off by at most 86 u = 5.1e-6 of
    the terms' magnitudes in the library's order, torch's products likewise),
    so 1e-4 of a tensor's largest gradient covers it; bfloat16 would not pass."""
    import ddp_tokens as ex
    flat = ex.make_parameters(DEV)
    bucket = torch.full_like(flat, 9.0)
    data = torch.Generator(device=DEV).manual_seed(5)
    batches = [ex.make_batch(data, torch.device(DEV)) for _ in range(2)]
    losses = [ex.micro_batch(ex.views(flat), ex.views(bucket), *b, accumulate=m > 0) for m, b in enumerate(batches)]
    leaf = flat.cpu().double().requires_grad_()
    host = [(i.cpu(), t.cpu()) for i, t in batches]
    # rows of padding are looked up as any other and take no gradient
    want_loss = plain_loss(ex.views(leaf), host, ex)
    want, = torch.autograd.grad(want_loss, leaf)
    assert abs(float(sum(losses)) - float(want_loss.detach())) < 1e-4 * float(want_loss.detach())
    for (name, g), w in zip(ex.views(bucket.cpu().double()).items(), ex.views(want).values()):
        if name == "table":
            assert bool((g[ex.PADDING] == 0).all())
            w = w.clone()
            w[ex.PADDING] = 0
        assert float((g - w).abs().max()) <= 1e-4 * float(w.abs().max()), name
    # along a direction: the gradient against a difference of the loss in binary64, whose error is of second order
    d = torch.randn(flat.numel(), generator=torch.Generator().manual_seed(2), dtype=torch.float64)
    ex.views(d)["table"][ex.PADDING] = 0
    d /= d.norm()
    step, at = 1e-3, leaf.detach()
    slope = float(plain_loss(ex.views(at + step * d), host, ex) - plain_loss(ex.views(at - step * d), host, ex))
    slope /= 2 * step
    assert abs(float(bucket.cpu().double() @ d) - slope) <= 1e-4 * float(bucket.double().norm())


def test_the_example_runs(gb):
    import ddp_tokens as ex
    for codec in ("none", "fp8"):
        flat, losses = ex.train(codec, 6)
        assert len(losses) == 6 and np.isfinite(losses).all() and bool(torch.isfinite(flat).all())


class Calls:
    """One of each call with inputs and outputs of its own."""

    def __init__(self, gb, seed, rows=1500, cols=700, vocab=900, kind=torch.bfloat16):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.gb, self.g, self.vocab = gb, g, vocab
        self.table = torch.empty(vocab, cols, device=DEV)
        self.ids = torch.empty(rows, dtype=torch.int64, device=DEV)
        self.w, self.b = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
        self.dy = torch.empty(rows, cols, dtype=kind, device=DEV)
        self.x, self.y, self.dx = (torch.empty(rows, cols, dtype=kind, device=DEV) for _ in range(3))
        self.mean, self.rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        self.dw, self.db, self.dtable = (torch.empty_like(t) for t in (self.w, self.b, self.table))
        self.ws1 = torch.empty(gb.gb_layer_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
        self.ws2 = torch.empty(gb.gb_embedding_workspace_bytes(rows, vocab, cols), dtype=torch.uint8, device=DEV)
        self.fresh()

    def fresh(self):
        for t in (self.table, self.w, self.b):
            t.normal_(generator=self.g)
        self.dy.copy_(torch.randn(self.dy.shape, generator=self.g, device=DEV))
        self.ids.copy_(torch.randint(0, self.vocab, self.ids.shape, generator=self.g, device=DEV) ** 2 // self.vocab)
        for t in (self.dw, self.db, self.dtable):
            t.zero_()

    def run(self, stream=None, accumulate=True):
        gb = self.gb
        gb.gb_embedding_forward(self.x, self.table, self.ids, scale=3.0, stream=stream)
        gb.gb_layer_norm_forward(self.y, self.x, self.w, self.b, mean=self.mean, rstd=self.rstd, stream=stream)
        gb.gb_layer_norm_backward(self.dx, self.dw, self.db, self.dy, self.x, self.mean, self.rstd, self.w,
                                  accumulate=accumulate, workspace=self.ws1, stream=stream)
        gb.gb_embedding_backward(self.dtable, self.dx, self.ids, scale=3.0, padding=1, accumulate=accumulate,
                                 workspace=self.ws2, stream=stream)

    def results(self):
        return [t.clone() for t in (self.x, self.y, self.mean, self.rstd, self.dx, self.dw, self.db, self.dtable)]


def equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_stream_given_and_the_current_one(gb):
    c = Calls(gb, 0)
    c.run()
    want = c.results()
    for how in ("given", "current"):
        for t in (c.dw, c.db, c.dtable):
            t.zero_()
        for t in (c.x, c.y, c.dx):
            t.fill_(7.0)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        if how == "given":
            c.run(stream=s)
        else:
            with torch.cuda.stream(s):
                c.run()
        s.synchronize()
        assert equal(c.results(), want), how


def test_two_calls_at_once_with_workspaces_of_their_own(gb):
    calls = [Calls(gb, k, rows=9000 if k else 1500) for k in range(2)]
    want = []
    for c in calls:
        c.run()
        want.append(c.results())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for c in calls:
        for t in (c.dw, c.db, c.dtable):
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(calls, streams):
            c.run(stream=s, accumulate=False)
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        assert equal(c.results(), w)


@pytest.mark.parametrize("rows", [40, 1500, 9000])
def test_captured_once_and_replayed_with_new_inputs(gb, rows):
    """Each replay against the eager calls on the same inputs, with eager work
    and waits between."""
    c, eager = Calls(gb, 3, rows=rows), Calls(gb, 4, rows=rows)
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for k in range(4):
        c.fresh()
        if k == 2:
            c.ids.fill_(5)  # every token of one row
        for a, b in ((eager.table, c.table), (eager.w, c.w), (eager.b, c.b), (eager.dy, c.dy), (eager.ids, c.ids)):
            a.copy_(b)
        for t in (eager.dw, eager.db, eager.dtable):
            t.zero_()
        graph.replay()
        eager.run()
        torch.cuda.synchronize()
        assert equal(c.results(), eager.results()), k


def test_micro_batches_add_up(gb):
    """Integers: the gradients of three micro-batches are those of all tokens."""
    rows, cols, vocab = 3 * 700, 130, 50
    rng = np.random.default_rng(0)
    dout = torch.from_numpy(rng.integers(-4, 5, (rows, cols)).astype(np.float32)).to(DEV)
    ids = torch.from_numpy(rng.integers(0, vocab, rows)).to(DEV)
    ws = torch.empty(gb.gb_embedding_workspace_bytes(rows, vocab, cols), dtype=torch.uint8, device=DEV)
    whole, parts = (torch.full((vocab, cols), 3.0, device=DEV) for _ in range(2))
    gb.gb_embedding_backward(whole, dout, ids, workspace=ws)
    for k in range(3):
        gb.gb_embedding_backward(parts, dout[700 * k:700 * k + 700], ids[700 * k:700 * k + 700], accumulate=k > 0,
                                 workspace=ws)
    assert torch.equal(whole, parts)


def test_shards_of_a_vocabulary_add_up_to_the_whole(gb):
    vocab, dim, ranks = 1000, 40, 4
    table = torch.randn(vocab, dim, device=DEV)
    ids = torch.randint(0, vocab, (777,), device=DEV)
    whole = torch.empty(777, dim, device=DEV)
    gb.gb_embedding_forward(whole, table, ids, scale=2.0)
    outs = [torch.empty_like(whole) for _ in range(ranks)]
    for r, out in enumerate(outs):
        gb.gb_embedding_forward(out, table[250 * r:250 * r + 250], ids, scale=2.0, first=250 * r)
    total = torch.empty_like(whole)
    gb.gb_reduce_sum(total, outs)
    assert torch.equal(total, whole)
    ws = torch.empty(gb.gb_embedding_workspace_bytes(777, vocab, dim), dtype=torch.uint8, device=DEV)
    want, got = torch.empty_like(table), torch.empty_like(table)
    gb.gb_embedding_backward(want, whole, ids, workspace=ws)
    for r in range(ranks):
        gb.gb_embedding_backward(got[250 * r:250 * r + 250], whole, ids, first=250 * r, workspace=ws)
    assert torch.equal(got, want)
