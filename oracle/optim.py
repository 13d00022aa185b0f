"""Oracle of the optimizer step in plain numpy (test infrastructure only):
the gradient norm, AdamW in binary32 with every operation rounded on its own,
the dithered E4M3 rounding of the 8-bit moments, and AdamW in binary64 to
measure the binary32 one against.

Arrays are in host memory; gradients come as float32 values, whatever type
they were held in.
"""
import math

import numpy as np

BLOCK = 256
F = np.float32
GOLDEN = 0x9E3779B97F4A7C15
M64 = (1 << 64) - 1

# magnitudes of the codes 0..126 (S.1111.111 = NaN is not among them)
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])


def power(b, t):
    """b^t by squaring, in binary64."""
    r = 1.0
    while t > 0:
        if t & 1:
            r *= b
        b *= b
        t >>= 1
    return r


def grad_norm(grads, max_norm, inv_scale):
    """(norm, coef, skipped) of gradients given as float32 arrays."""
    total = math.fsum(math.fsum(np.square(g.astype(np.float64)).tolist()) for g in grads)
    norm = inv_scale * math.sqrt(total) if total >= 0 else math.nan
    with np.errstate(over="ignore"):
        f = F(norm)
    if not np.isfinite(f):
        return f, F(0), True
    return f, F(inv_scale * max_norm / norm if norm > max_norm else inv_scale), False


def rates(t, beta1, beta2):
    """The bias corrections of step t."""
    return F(1.0 / (1.0 - power(beta1, t))), F(1.0 / math.sqrt(1.0 - power(beta2, t)))


def canon(x):
    return np.where(np.isnan(x), np.uint32(0x7FC00000).view(F), x)


def adamw(p, g, m, v, t, coef, lr, lr_scale=1.0, wd=0.0, beta1=0.9, beta2=0.999, eps=1e-8):
    """p', m', v' and sqrt(v'), binary32."""
    with np.errstate(all="ignore"):
        r1, r2 = rates(t, beta1, beta2)
        gs = g * F(coef)
        m = F(beta1) * m + F(1.0 - beta1) * gs
        v = F(beta2) * v + F(1.0 - beta2) * (gs * gs)
        u = np.sqrt(v)
        d = u * r2 + F(eps)
        lr_t = F(F(lr) * F(lr_scale))
        p = p * F(F(1) - F(lr_t * F(wd))) - F(lr_t * r1) * (m / d)
    assert p.dtype == m.dtype == v.dtype == np.float32
    return canon(p), canon(m), canon(v), u


def adamw64(p, g, m, v, t, coef, lr, lr_scale=1.0, wd=0.0, beta1=0.9, beta2=0.999, eps=1e-8):
    """p', m', v' in binary64."""
    p, g, m, v = (x.astype(np.float64) for x in (p, g, m, v))
    gs = g * float(coef)
    m = beta1 * m + (1 - beta1) * gs
    v = beta2 * v + (1 - beta2) * gs * gs
    lr_t = float(lr) * lr_scale
    p = p - lr_t * wd * p - lr_t * (m / (1 - beta1 ** t)) / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    return p, m, v


def dither(seed, t, first, n):
    """20 dither bits of the values [first, first + n) of a plan, step t."""
    z = (seed + t * GOLDEN) & M64
    for _ in range(3):
        z = ((z ^ (z >> 32)) * GOLDEN) & M64
    key = z >> 32
    i = np.arange(first, first + n, dtype=np.uint64)
    low = np.uint64(0xFFFFFFFF)
    x = (i // np.uint64(2) * np.uint64(0x9E3779B9) + np.uint64(key)) & low
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x6A09E667)) & low
    x = x ^ (x >> np.uint64(16))
    return np.where(i % np.uint64(2) == 0, x >> np.uint64(12), (x & np.uint64(0xFFFF)) << np.uint64(4)).astype(np.int64)


def scales(x):
    """A block's scale: the smallest 2^e, e >= -126, with the block's largest
    finite magnitude a <= 448 * 2^e; 1 for a = 0."""
    out = np.empty((x.size + BLOCK - 1) // BLOCK, F)
    for b in range(out.size):
        y = np.abs(x[b * BLOCK:(b + 1) * BLOCK])
        y = y[np.isfinite(y)]
        a = float(y.max()) if y.size else 0.0
        e = -126
        while a > 448.0 * 2.0 ** e:
            e += 1
        out[b] = F(2.0 ** e) if a > 0 else F(1)
    return out


def encode(x, d, keep=False):
    """Codes and scales of x with the 20-bit dither d; keep: a value above 0
    takes at least the code 1."""
    s = scales(x)
    with np.errstate(all="ignore"):
        q = np.abs(x.astype(np.float64)) / np.repeat(s.astype(np.float64), BLOCK)[:x.size]
    bad = ~np.isfinite(x)
    q[bad] = 0.0
    lo = np.searchsorted(E4M3, q, side="right") - 1
    step = np.append(np.diff(E4M3), 32.0)[lo]
    # the bits below the code's last, of which 20 are kept
    frac = np.floor((q - E4M3[lo]) / step * (1 << 20)).astype(np.int64)
    code = lo + (frac + d >= (1 << 20))
    if keep:
        code = np.where(x > 0, np.maximum(code, 1), code)
    code = code | np.where(np.signbit(x), 0x80, 0)
    return np.where(bad, 0x7F, code).astype(np.uint8), s


def decode(codes, s):
    mag = np.append(E4M3, np.nan).astype(F)[codes & 0x7F]
    return np.where(codes & 0x80, -mag, mag) * np.repeat(s, BLOCK)[:codes.size]


def adamw_e4m3(p, g, mc, ms, uc, us, t, coef, lr, seed, first, **kw):
    """p' and the codes and scales of m' and sqrt(v'); first: the tensor's
    position in the plan."""
    with np.errstate(all="ignore"):
        m, u = decode(mc, ms), decode(uc, us)
        p, m, _, u = adamw(p, g, m, u * u, t, coef, lr, **kw)
    d = dither(seed, t, first, p.size)
    return (p, *encode(m, d), *encode(u, d, keep=True))
