"""The optimizer's oracle on the CPU: its binary32 step against binary64
within the derived bound, its gradient step against differences of the moving
averages' definition, the dithered rounding's neighbours, mean and fixed
points, and what the 8-bit moments are for: averages that stay right."""
import math

import numpy as np
import pytest

from oracle import optim as P
from oracle import oracle as O

U = 2.0 ** -24


def inputs(n, seed, sigma=1e-3):
    rng = np.random.default_rng(seed)
    p = rng.standard_normal(n, dtype=np.float32) * np.float32(0.02)
    g = rng.standard_normal(n, dtype=np.float32) * np.float32(sigma)
    m = rng.standard_normal(n, dtype=np.float32) * np.float32(sigma)
    v = (rng.standard_normal(n, dtype=np.float32) * np.float32(sigma)) ** 2
    return p, g, m, v


def bounds(p, g, m, v, t, coef, lr, lr_scale, wd, beta1=0.9, beta2=0.999, eps=1e-8):
    """Error bounds of p', m', v' from the roundings along each path (u = 2^-24
    each; constants, coef and the corrections count as one): m' 5u of the
    sum of magnitudes, v' 8u, the denominator 8u, the quotient 15u and the
    update 20u of that sum's quotient, p's own terms 5u; one more each for
    the products of errors."""
    p, g, m, v = (np.abs(x.astype(np.float64)) for x in (p, g, m, v))
    gs = g * float(coef)
    big = beta1 * m + (1 - beta1) * gs
    v1 = beta2 * v + (1 - beta2) * gs * gs
    d = np.sqrt(v1 / (1 - beta2 ** t)) + eps
    step = float(lr) * lr_scale / (1 - beta1 ** t)
    tiny = 2.0 ** -149
    return (6 * U * p * (1 + lr * lr_scale * wd) + 21 * U * step * big / d + tiny, 6 * U * big + tiny,
            9 * U * v1 + 4 * tiny)


@pytest.mark.parametrize("t", [1, 2, 1000, 10 ** 6])
@pytest.mark.parametrize("wd,lr_scale,coef", [(0.0, 1.0, 1.0), (0.1, 0.5, 1.0 / 1024)])
def test_binary32_step_against_binary64(t, wd, lr_scale, coef):
    p, g, m, v = inputs(4099, t % 97)
    g = g * np.float32(1 / coef)
    got = P.adamw(p, g, m, v, t, coef, 1e-3, lr_scale, wd)
    # the inputs that the step receives in binary32 are what binary64 starts from
    lr = float(np.float32(1e-3))
    want = P.adamw64(p, g, m, v, t, coef, lr, lr_scale, float(np.float32(wd)))
    for name, x, y, b in zip("pmv", got, want, bounds(p, g, m, v, t, coef, lr, lr_scale, wd)):
        assert (np.abs(x.astype(np.float64) - y) <= b).all(), (name, np.max(np.abs(x - y) / b))


def test_the_moments_are_the_averages_of_their_definition():
    """After t steps from zero, m / (1 - beta1^t) and v / (1 - beta2^t) are
    the weighted means of the gradients and of their squares."""
    rng = np.random.default_rng(5)
    gs = rng.standard_normal((40, 33))
    z = np.zeros(33)
    p, m, v = z, z, z
    for t in range(1, 41):
        p, m, v = P.adamw64(p, gs[t - 1], m, v, t, 1.0, 1e-3)
    w1 = 0.9 ** np.arange(39, -1, -1)
    w2 = 0.999 ** np.arange(39, -1, -1)
    np.testing.assert_allclose(m / (1 - 0.9 ** 40), w1 @ gs / w1.sum(), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(v / (1 - 0.999 ** 40), w2 @ gs ** 2 / w2.sum(), rtol=1e-12)


def test_first_step_moves_by_the_learning_rate():
    """From zero moments the first step is lr * sign(g) to within eps / |g|."""
    p, g, _, _ = inputs(1000, 3)
    z = np.zeros_like(p)
    got = P.adamw(p, g, z, z, 1, 1.0, 1e-3)[0]
    off = np.abs((p.astype(np.float64) - got) - 1e-3 * np.sign(g))
    # the quotient |g| / (|g| + eps) and 30 roundings of the terms
    assert (off <= 1e-3 * 1e-8 / (np.abs(g) + 1e-8) + 30 * U * (np.abs(p) + 1e-3)).all()


@pytest.mark.parametrize("b", [0.0, 0.9, 0.999, 0.99999])
def test_power_by_squaring(b):
    for t in (1, 2, 3, 64, 1000, 123457):
        # each of the at most 2 log2(t) products rounds once, and the base's error grows with the power
        assert P.power(b, t) == pytest.approx(b ** t, rel=2 * t * 2.0 ** -53 + 40 * 2.0 ** -53, abs=1e-300)


def test_norm_clip_and_skip():
    g = [np.array([3e20, 0], np.float32), np.array([4e20], np.float32)]
    norm, coef, skip = P.grad_norm(g, 1.0, 1.0)
    assert not skip and abs(norm / 5e20 - 1) < 2e-7 and abs(coef * 5e20 - 1) < 2e-7
    assert P.grad_norm([np.array([1e-30], np.float32)], 1.0, 1.0)[:2] == (np.float32(1e-30), np.float32(1))
    for bad in (np.inf, np.nan):
        assert P.grad_norm([np.array([1, bad], np.float32)], 1.0, 1.0)[1:] == (0, True)
    assert P.grad_norm([], 1.0, 0.5) == (0, np.float32(0.5), False)


def test_dither_is_even_and_changes_with_the_step():
    d = P.dither(7, 3, 0, 1 << 16).astype(np.float64) / (1 << 20)
    # the mean of 2^16 uniform values is within 5 sigma = 5 / sqrt(12 * 2^16) of 1/2
    assert abs(d.mean() - 0.5) < 5 / math.sqrt(12 * (1 << 16))
    counts, _ = np.histogram(d, 64, (0, 1))
    assert ((counts - 1024) ** 2 / 1024).sum() < 63 + 6 * math.sqrt(2 * 63)
    assert abs(np.corrcoef(d[::2], d[1::2])[0, 1]) < 5 / math.sqrt(1 << 15)
    assert abs(np.corrcoef(d[:-2], d[2:])[0, 1]) < 5 / math.sqrt(1 << 16)
    steps = np.array([P.dither(7, t, 512, 64) for t in range(1, 2001)]).astype(np.float64) / (1 << 20)
    assert (np.abs(steps.mean(0) - 0.5) < 6 / math.sqrt(12 * 2000)).all()
    lag = ((steps[1:] - 0.5) * (steps[:-1] - 0.5)).mean(0) * 12
    assert (np.abs(lag) < 6 / math.sqrt(2000)).all()
    assert (P.dither(7, 3, 512, 100) == P.dither(7, 3, 0, 612)[512:]).all()


def test_every_code_on_the_grid_stays_and_others_go_to_a_neighbour():
    x = np.resize(P.E4M3, 256).astype(np.float32)
    for d in (0, (1 << 20) - 1):
        c, s = P.encode(x, np.full(256, d))
        assert s[0] == 1 and (P.decode(c, s) == x).all()
    rng = np.random.default_rng(1)
    x = (rng.standard_normal(4096) * 10.0 ** rng.uniform(-6, 2, 4096)).astype(np.float32)
    d = rng.integers(0, 1 << 20, 4096)
    c, s = P.encode(x, d)
    q = np.abs(x) / np.repeat(s, 256)
    k = (c & 0x7F).astype(np.int64)
    assert (np.abs(P.E4M3[k] - q) < np.append(np.diff(P.E4M3), 32.0)[np.searchsorted(P.E4M3, q, side="right") - 1]).all()
    assert (np.signbit(x) == (c >= 128)).all()


def test_the_codes_are_payloads_of_the_fp8_codec():
    """Scales follow the power-of-two rule of the codec, and its decode gives
    the values back."""
    rng = np.random.default_rng(2)
    x = (rng.standard_normal(1000) * 1e-3).astype(np.float32)
    c, s = P.encode(x, rng.integers(0, 1 << 20, 1000))
    _, want = O.encode_fp8(x, O.SCALE_POW2)
    assert (s == want).all()
    assert (O.decode_accumulate([c], [s], O.CODEC_FP8) == P.decode(c, s)).all()


def test_rounding_is_right_on_average():
    x = np.full(256, 1.03, np.float32)
    x[0] = 448.0
    got = np.array([P.decode(*P.encode(x, P.dither(1, t, 0, 256)))[1:] for t in range(400)])
    # steps of 0.125: 255 * 400 draws of a two-point variable
    p = 0.03 / 0.125
    assert abs(got.mean() - 1.03) < 5 * 0.125 * math.sqrt(p * (1 - p) / got.size)


def test_a_root_above_zero_keeps_a_code_and_zero_stays_zero():
    x = np.zeros(256, np.float32)
    x[0], x[1], x[2] = 1.0, 1e-9, 2.0 ** -74
    c, s = P.encode(x, np.zeros(256, np.int64), keep=True)
    assert (c[:3] == [P.E4M3.searchsorted(256.0), 1, 1]).all() and not c[3:].any()
    c, s = P.encode(np.zeros(300, np.float32), np.full(300, (1 << 20) - 1), keep=True)
    assert not c.any() and (s == 1).all()


def test_not_finite_values_take_the_nan_code_and_leave_the_scale():
    x = np.ones(256, np.float32)
    x[[3, 7, 9]] = [np.inf, -np.inf, np.nan]
    c, s = P.encode(x, np.zeros(256, np.int64))
    assert (c[[3, 7, 9]] == 0x7F).all() and s[0] == 2.0 ** -8
    assert (P.decode(c, s)[[0, 1, 2]] == 1).all()


def test_eight_bit_root_follows_the_binary32_one():
    """3000 steps of a noisy gradient that shrinks tenfold halfway for every
    other value: the mean ratio of the roots stays within 3%, where rounding
    to the nearest code would leave them where the moving averages' small
    steps no longer reach the next code."""
    rng = np.random.default_rng(11)
    n, T = 2048, 3000
    sigma = np.exp(rng.standard_normal(n)) * 1e-3
    half = np.arange(n) % 2 == 0
    p = np.zeros(n, np.float32)
    mc = uc = np.zeros(n, np.uint8)
    ms = us = np.zeros(n // 256, np.float32)
    m, v = p, p
    ratio = []
    for t in range(1, T + 1):
        s = np.where(half & (t > T // 2), 0.1 * sigma, sigma)
        g = (s * (0.2 + rng.standard_normal(n))).astype(np.float32)
        _, m, v, u = P.adamw(p, g, m, v, t, 1.0, 1e-3)
        _, mc, ms, uc, us = P.adamw_e4m3(p, g, mc, ms, uc, us, t, 1.0, 1e-3, 9, 0)
        if t > T - 500 and t % 50 == 0:
            ratio.append(P.decode(uc, us) / u)
    ratio = np.array(ratio)
    assert abs(ratio[:, half].mean() - 1) < 0.03 and abs(ratio[:, ~half].mean() - 1) < 0.03
