"""The token model's layers as autograd sees them, without a GPU: the library's
calls are stood in for by plain ones."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def ex(monkeypatch):
    monkeypatch.syspath_prepend(os.path.join(ROOT, "examples"))
    import ddp_tokens
    yield ddp_tokens
    sys.modules.pop("ddp_tokens")


def test_the_lookup_is_not_copied_and_its_gradient_arrives(ex, monkeypatch):
    """The layer gives out the very buffer that the lookup wrote, and the
    backward pass reaches the table's call with the output's gradient."""
    seen = {}

    def forward(out, table, ids, scale):
        out.copy_(table[ids] * scale)
        seen["out"] = out.data_ptr()

    def backward(bucket, dout, ids, scale, padding, accumulate, workspace):
        seen["dout"], seen["accumulate"] = dout.clone(), accumulate
        bucket.index_add_(0, ids.flatten(), scale * dout.flatten(0, 1))

    monkeypatch.setattr(ex.gb, "gb_embedding_forward", forward)
    monkeypatch.setattr(ex.gb, "gb_embedding_backward", backward)
    table, bucket = torch.randn(10, 4), torch.zeros(10, 4)
    ids = torch.tensor([[1, 2, 2], [9, 0, 1]])
    anchor = torch.zeros((), requires_grad=True)
    x = ex.Embedding.apply(anchor, table, ids, bucket, True)
    assert x.data_ptr() == seen["out"] and x.requires_grad
    weights = torch.randn(2, 3, 4)
    d, = torch.autograd.grad((x * weights).sum(), anchor)
    assert float(d) == 0.0 and torch.equal(seen["dout"], weights) and seen["accumulate"] is True
    leaf = table.clone().requires_grad_()
    want, = torch.autograd.grad(((leaf[ids] * 2.0) * weights).sum(), leaf)
    assert torch.allclose(bucket, want)
