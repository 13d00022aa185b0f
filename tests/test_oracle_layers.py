"""The token-sum layers' oracle against independent formulas, without a GPU:
torch's own layer norm and its gradients in binary64, the order of the table's
sums by hand, and the bounds against a binary32 computation in numpy."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import layers as Y  # noqa: E402


def rows(seed, m, n):
    return np.random.default_rng(seed).standard_normal((m, n), dtype=np.float32)


@pytest.mark.parametrize("m,n", [(3, 1), (5, 7), (20, 300)])
def test_norm_and_its_gradients_are_torchs(m, n):
    x, dy, w, b = rows(1, m, n), rows(2, m, n), rows(3, 1, n)[0], rows(4, 1, n)[0]
    leaves = [torch.from_numpy(v).double().requires_grad_() for v in (x, w, b)]
    y = torch.nn.functional.layer_norm(leaves[0], (n,), leaves[1], leaves[2], 1e-5)
    got, mean, rstd, e_y, e_m, e_r = Y.norm(x, w, b, 1e-5)
    assert np.allclose(got, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    dx, dw, db = torch.autograd.grad(y, leaves, torch.from_numpy(dy).double())
    got = Y.norm_gradients(dy, x, mean, rstd, w)
    for a, want in zip(got, (dx, dw, db)):
        assert np.allclose(a, want.numpy(), rtol=1e-9, atol=1e-9)
    assert all((e >= 0).all() and np.isfinite(e).all() for e in (e_y, e_m, e_r, *got[3:]))


@pytest.mark.parametrize("m,n", [(50, 3), (40, 64), (30, 1000)])
def test_a_binary32_computation_stays_within_the_bounds(m, n):
    """numpy's pairwise sums have fewer additions on a term's way than the
    bounds allow for."""
    f = np.float32
    x = rows(5, m, n) * np.exp(rows(6, m, 1)) + f(0.5)
    w, b, dy = rows(7, 1, n)[0], rows(8, 1, n)[0], rows(9, m, n)
    mean = x.mean(1, dtype=f)
    dev = x - mean[:, None]
    rstd = f(1) / np.sqrt((dev * dev).mean(1, dtype=f) + f(1e-5))
    y = dev * rstd[:, None] * w + b
    want, m64, r64, e_y, e_m, e_r = Y.norm(x, w, b, 1e-5)
    # the product and the sum of y round apart here, fused in the bound: one more rounding
    assert (np.abs(y - want) <= e_y + Y.U * np.abs(want - b) * 1.01).all()
    assert (np.abs(mean - m64) <= e_m).all() and (np.abs(rstd - r64) <= e_r).all()
    h, g = dev * rstd[:, None], dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - h * (g * h).mean(1, keepdims=True))
    wdx, wdw, wdb, e_dx, e_dw, e_db = Y.norm_gradients(dy, x, mean, rstd, w)
    assert (np.abs(dx - wdx) <= e_dx).all()
    assert (np.abs((dy * h).sum(0) - wdw) <= e_dw).all() and (np.abs(dy.sum(0) - wdb) <= e_db).all()


def test_the_order_of_the_sums():
    f = np.float32
    big = f(2.0 ** 24)
    # 64 in turn: ones added to 2^24 one by one are lost
    x = np.array([[big]] + [[f(1)]] * 63, dtype=f)
    assert Y.fold(x)[0] == big
    # the 65th begins the next sum, and 64 ones there count together
    x = np.array([[big]] + [[f(1)]] * 63 + [[f(1)]] * 64, dtype=f)
    assert Y.fold(x)[0] == big + f(64)
    # 64 sums of 64, then one more: sums of sums
    x = np.ones((64 * 64 + 1, 1), dtype=f)
    x[0] = big
    assert Y.fold(x)[0] == big + f(63 * 64)


def test_lookup_and_gradient_against_plain_sums():
    table, dout = rows(1, 12, 5), rows(2, 400, 5)
    ids = np.random.default_rng(3).integers(-3, 20, 400)
    out = Y.lookup(table, ids, 2.0, first=1)
    for t, i in enumerate(ids):
        assert (out[t] == (table[i - 1] * np.float32(2) if 1 <= i < 13 else 0)).all()
    got, named = Y.table_gradient(dout, ids, 12, 0.5, first=1, padding=4)
    want = np.zeros((12, 5))
    for t, i in enumerate(ids):
        if 1 <= i < 13 and i != 4:
            want[i - 1] += 0.5 * dout[t].astype(np.float64)
    assert np.allclose(got, want, rtol=1e-5, atol=1e-5) and (got[3] == 0).all()
    assert named.tolist() == [r for r in range(12) if r != 3]
    more, _ = Y.table_gradient(dout, ids, 12, 0.5, first=1, padding=4, old=table)
    assert np.allclose(more, table + want, rtol=1e-5, atol=1e-5) and (more[3] == table[3]).all()
