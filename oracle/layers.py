"""Oracle of the token-sum layers in plain numpy (test infrastructure only):
the embedding lookup and the table's gradient in binary32 with every operation
rounded on its own, and layer norm, forward and backward, in binary64 with
bounds on what binary32 arithmetic may lose.

Arrays are in host memory; values of other types come as float32 (exact), and
results that are rounded to another type are rounded by the caller.
"""
import numpy as np

F = np.float32
FOLD = 64
U = 2.0 ** -24  # half a step of binary32, relative


def canon(x):
    return np.where(np.isnan(x), np.uint32(0x7FC00000).view(F), x)


def rows_of(ids, first, vocab):
    """The row of each id, -1 for one outside [first, first + vocab)."""
    return np.array([i - first if 0 <= i - first < vocab else -1 for i in (int(v) for v in ids)], dtype=np.int64)


def lookup(table, ids, scale, first=0):
    rows = rows_of(ids, first, len(table))
    with np.errstate(all="ignore"):
        out = canon(table[np.maximum(rows, 0)] * F(scale)) if len(table) else np.zeros((len(rows), table.shape[1]), F)
    out[rows < 0] = 0
    return out


def fold(x):
    """Rows of x added 64 at a time in turn, then those sums, until one is left."""
    with np.errstate(all="ignore"):
        while len(x) > 1:
            sums = []
            for i in range(0, len(x), FOLD):
                s = x[i].copy()
                for v in x[i + 1:i + FOLD]:
                    s = s + v
                sums.append(s)
            x = np.stack(sums)
    return x[0]


def table_gradient(dout, ids, vocab, scale, first=0, padding=-1, old=None):
    """The gradient in binary32, and which rows have a token."""
    rows = rows_of(ids, first, vocab)
    rows[np.asarray(ids) == padding] = -1
    out = np.zeros((vocab, dout.shape[1]), F) if old is None else old.copy()
    order = np.argsort(rows, kind="stable")
    order = order[rows[order] >= 0]
    named, starts = np.unique(rows[order], return_index=True)
    for row, tokens in zip(named, np.split(order, starts[1:]) if len(named) else []):
        with np.errstate(all="ignore"):
            s = fold(dout[tokens]) * F(scale)
            out[row] = canon(s if old is None else old[row] + s)
    return out, named


# ---------------------------------------------------------------------------
# Layer norm.  Bounds: a sum of n terms added in any order with at most d
# additions on a term's way is off by at most d u times the sum of the terms'
# magnitudes (u = 2^-24, first order, which a factor of 1.01 covers here).
# ---------------------------------------------------------------------------
def depth(n):
    """Additions on a term's way in a row's sum: a lane holds at most 64 values
    of a row, or its share of a shorter one, then at most 6 + 16 for joining
    lanes and wavefronts."""
    return min(n, 64 + 22)


def norm(x, w, b, eps):
    """y, mean, rstd in binary64 and a bound on the binary32 error of each."""
    x, n = x.astype(np.float64), x.shape[1]
    w = np.ones(n) if w is None else w.astype(np.float64)
    b = np.zeros(n) if b is None else b.astype(np.float64)
    mean = x.mean(1)
    dev = x - mean[:, None]
    var = (dev * dev).mean(1)
    rstd = 1.0 / np.sqrt(var + eps)
    d = depth(n)
    e_mean = 1.01 * ((d + 1) * U * np.abs(x).mean(1))
    # each deviation is off by the mean's error and its own rounding; the
    # deviations sum to zero, so the mean's error enters the variance squared
    e_var = 1.01 * (e_mean ** 2 + (d + 5) * U * (var + e_mean ** 2))
    # rstd is 1 / sqrt of a sum of eps' binary32 value and the variance: three more roundings
    e_rstd = rstd * (0.505 * (e_var + 2 * U * (var + eps)) / (var + eps) + 3 * U)
    y = dev * rstd[:, None] * w + b
    e_dev = e_mean[:, None] + U * np.abs(dev)
    e_h = e_dev * rstd[:, None] + np.abs(dev) * e_rstd[:, None] + U * np.abs(dev * rstd[:, None])
    e_y = 1.01 * (np.abs(w) * e_h + U * np.abs(y) + U * np.abs(b))
    return y, mean, rstd, e_y, e_mean, e_rstd


def norm_gradients(dy, x, mean, rstd, w):
    """dx, dw, db in binary64 with a bound on the binary32 error of each; mean
    and rstd are taken as they are."""
    n, rows = x.shape[1], x.shape[0]
    dy, x = dy.astype(np.float64), x.astype(np.float64)
    w = np.ones(n) if w is None else w.astype(np.float64)
    m, s = mean.astype(np.float64)[:, None], rstd.astype(np.float64)[:, None]
    h = (x - m) * s
    g = dy * w
    c1, c2 = g.mean(1, keepdims=True), (g * h).mean(1, keepdims=True)
    dx = s * (g - c1 - h * c2)
    d = depth(n)
    # h has 2 roundings, g one, 1 / n and the factors 3 more
    e_c1 = (d + 5) * U * np.abs(g).mean(1, keepdims=True)
    e_c2 = (d + 8) * U * np.abs(g * h).mean(1, keepdims=True)
    e_dx = 1.01 * (s * (e_c1 + np.abs(h) * e_c2) + 6 * U * s * (np.abs(g) + np.abs(c1) + np.abs(h * c2)))
    # the terms' 3 roundings, then a sum over the rows in any order
    e_dw = 1.01 * (rows + 4) * U * np.abs(dy * h).sum(0)
    e_db = 1.01 * (rows + 1) * U * np.abs(dy).sum(0)
    return dx, (dy * h).sum(0), dy.sum(0), e_dx, e_dw, e_db


def rounding(y, kind):
    """Half a step of a type at y: what rounding a result to it may add."""
    half, least = {"f32": (2.0 ** -24, 2.0 ** -150), "f16": (2.0 ** -11, 2.0 ** -25),
                   "bf16": (2.0 ** -8, 2.0 ** -134)}[kind]
    return half * np.abs(y) + least
