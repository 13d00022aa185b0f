"""The optimizer step on the GPU.  The binary32 arithmetic, the codes, the
scales and the copies are compared bit for bit with the oracle's; the step
and the norm also with binary64, within bounds derived from the roundings."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from oracle import optim as P  # noqa: E402
from tests.test_oracle_optim import bounds  # noqa: E402

DEV = "cuda:0"
U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def gb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_all_reduce_amd as lib
    return lib


def host(t):
    torch.cuda.synchronize()
    return t.detach().cpu()


def f32(t):
    """float32 numpy values of a float tensor (exact)."""
    return host(t.float()).numpy()


def same(a, b, what):
    a, b = np.ascontiguousarray(a), np.ascontiguousarray(b)
    if a.dtype == np.float32:
        a, b = a.view(np.uint32), b.view(np.uint32)
    bad = np.flatnonzero(a != b)
    assert bad.size == 0, f"{what}: {bad.size} of {a.size} differ, first at {bad[0]}: {a[bad[0]]} and {b[bad[0]]}"


class Problem:
    """Tensors of given sizes with their host mirrors; `shift` values of room
    before each parameter, gradient and copy (their views then start off 16
    bytes), and a guard after."""

    def __init__(self, gb, spec, draw, shift=0, lr=1e-3, sigma=1e-3, **plan):
        rng = np.random.default_rng(draw)
        self.gb, self.entries, self.host, self.guards, at = gb, [], [], [], 0
        for k, (n, kind, state, copy) in enumerate(spec):
            dt = TYPES[kind]

            def room(dtype, count, pre, fill=7):
                buf = torch.full((pre + count + 16,), fill, dtype=dtype, device=DEV)
                self.guards.append((buf, pre, count, fill))
                return buf[pre:pre + count]

            p = room(torch.float32, n, shift)
            g = room(dt, n, shift)
            p.copy_(torch.from_numpy(rng.standard_normal(n, dtype=np.float32) * np.float32(0.02)))
            c = room(TYPES[copy] if isinstance(copy, str) else dt, n, shift) if copy else None
            blocks = -(-n // 256)
            if state == "e4m3":
                m, v = room(torch.uint8, n, 0), room(torch.uint8, n, 0)
                ms, vs = room(torch.float32, blocks, 0), room(torch.float32, blocks, 0)
            else:
                m, v, ms, vs = room(torch.float32, n, 0), room(torch.float32, n, 0), None, None
            for x in (m, v, ms, vs):
                if x is not None:
                    x.zero_()
            wd, scale = (0.1 if k % 2 == 0 else 0.0), (0.5 if k % 3 == 2 else 1.0)
            self.entries.append(gb.GbOptimTensor(p, g, m, v, ms, vs, c, scale, wd))
            self.host.append(dict(p=f32(p), m=host(m).numpy().copy(), v=host(v).numpy().copy(),
                                  ms=None if ms is None else f32(ms), vs=None if vs is None else f32(vs),
                                  at=at, n=n, wd=wd, scale=scale, state=state, sigma=sigma))
            at += blocks * 256
        self.ws = torch.full((gb.gb_optim_plan_bytes([s[0] for s in spec]),), 255, dtype=torch.uint8, device=DEV)
        self.hyper = dict(beta1=plan.get("beta1", 0.9), beta2=plan.get("beta2", 0.999), eps=plan.get("eps", 1e-8))
        self.seed, self.lr, self.t = plan.get("seed", 12345), lr, 0
        self.plan = gb.gb_optim_plan(self.entries, self.ws, seed=self.seed, **self.hyper)
        self.control = torch.zeros(64, dtype=torch.uint8, device=DEV)
        self.view = gb.gb_optim_control(self.control)
        self.view["lr"].fill_(lr)
        self.rng = rng

    def gradients(self, special=()):
        for e, h in zip(self.entries, self.host):
            g = self.rng.standard_normal(h["n"], dtype=np.float32) * np.float32(h["sigma"])
            for i, value in enumerate(special):
                if i < h["n"]:
                    g[i] = value
            e.grad.copy_(torch.from_numpy(g))

    def step(self, max_norm=None, inv_scale=1.0, stream=None):
        if max_norm is None:
            self.gb.gb_optim_begin(self.plan, self.control, inv_scale, stream=stream)
        else:
            self.gb.gb_optim_begin_clip(self.plan, self.control, max_norm, inv_scale, stream=stream)
        self.gb.gb_adamw_step(self.plan, self.control, stream=stream)

    def follow(self, max_norm=None, inv_scale=1.0):
        """The oracle's step on the host mirrors."""
        grads = [f32(e.grad) for e in self.entries]
        coef, skip = np.float32(inv_scale), False
        if max_norm is not None:
            norm, coef, skip = P.grad_norm(grads, max_norm, inv_scale)
            same(f32(self.view["norm"]), np.array([norm], np.float32), "norm")
        same(f32(self.view["coef"]), np.array([coef], np.float32), "coef")
        assert bool(host(self.view["skip"])) == skip
        self.t += not skip
        assert int(host(self.view["step"])) == self.t
        if skip:
            return
        for g, h in zip(grads, self.host):
            kw = dict(lr_scale=h["scale"], wd=h["wd"], **self.hyper)
            if h["state"] == "e4m3":
                h["p"], h["m"], h["ms"], h["v"], h["vs"] = P.adamw_e4m3(
                    h["p"], g, h["m"], h["ms"], h["v"], h["vs"], self.t, coef, self.lr, self.seed, h["at"], **kw)
            else:
                h["p"], h["m"], h["v"], _ = P.adamw(h["p"], g, h["m"], h["v"], self.t, coef, self.lr, **kw)

    def check(self):
        for k, (e, h) in enumerate(zip(self.entries, self.host)):
            same(f32(e.param), h["p"], f"param {k}")
            same(host(e.m).numpy(), h["m"], f"m {k}")
            same(host(e.v).numpy(), h["v"], f"v {k}")
            if h["state"] == "e4m3":
                same(f32(e.m_scale), h["ms"], f"m_scale {k}")
                same(f32(e.v_scale), h["vs"], f"v_scale {k}")
            if e.copy is not None:
                want = torch.from_numpy(h["p"]).to(e.copy.dtype).view(torch.int16).numpy()
                # the library's NaN in each type
                want = np.where(np.isnan(h["p"]), 0x7FC0 if e.copy.dtype == torch.bfloat16 else 0x7E00, want)
                same(host(e.copy).view(torch.int16).numpy(), want.astype(np.int16), f"copy {k}")
        for buf, pre, count, fill in self.guards:
            assert (buf[:pre] == fill).all() and (buf[pre + count:] == fill).all()


SIZES = [1, 2, 3, 255, 256, 257, 1023, 1024, 1025, 5000]


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("state", ["f32", "e4m3"])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_three_steps_bit_for_bit(gb, kind, state, shift):
    """Odd sizes together, aligned and one value off, clipped and not."""
    prob = Problem(gb, [(n, kind, state, kind != "f32" and n % 2 == 1) for n in SIZES], 17, shift=shift)
    for max_norm, inv in ((None, 1.0), (0.01, 0.125), (math.inf, 1.0)):
        prob.gradients()
        prob.step(max_norm, inv)
        prob.follow(max_norm, inv)
        prob.check()


@pytest.mark.parametrize("n", [1, 64, 300, 70001])
def test_one_tensor_many_steps(gb, n):
    """8-bit moments over 25 steps: every dithered code as the oracle's."""
    prob = Problem(gb, [(n, "f32", "e4m3", False)], n, seed=n * 977)
    for _ in range(25):
        prob.gradients()
        prob.step()
        prob.follow()
    prob.check()


def test_kinds_mixed_in_one_plan_with_empty_tensors(gb):
    spec = []
    for n in (700, 0, 33, 2049, 0, 1):
        for kind in ("f32", "f16", "bf16"):
            for state in ("f32", "e4m3"):
                spec.append((n, kind, state, kind == "bf16"))
    prob = Problem(gb, spec, 4)
    for _ in range(2):
        prob.gradients()
        prob.step(1.0)
        prob.follow(1.0)
        prob.check()


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_copies_of_either_type_beside_every_gradient_type(gb, state):
    """A bfloat16 model trained on float32 gradients, and the other pairs."""
    spec = [(n, kind, state, copy) for n in (1, 255, 3001) for kind in ("f32", "f16", "bf16") for copy in ("f16", "bf16")]
    prob = Problem(gb, spec, 60, shift=1)
    for _ in range(2):
        prob.gradients()
        prob.step(1.0)
        prob.follow(1.0)
        prob.check()


def test_many_tensors(gb):
    """More tensors than one upload of the tables carries."""
    rng = np.random.default_rng(8)
    spec = [(int(rng.integers(0, 900)), ("f32", "bf16")[i % 2], ("e4m3", "f32")[i % 3 == 0], False)
            for i in range(400)]
    prob = Problem(gb, spec, 5)
    for _ in range(2):
        prob.gradients()
        prob.step(0.05)
        prob.follow(0.05)
        prob.check()


def test_a_plan_of_nothing(gb):
    for spec in ([], [(0, "f32", "f32", False)]):
        prob = Problem(gb, spec, 1)
        prob.step()
        prob.step(1.0, 0.5)
        assert int(host(prob.view["step"])) == 2 and float(host(prob.view["norm"])) == 0.0
        assert float(host(prob.view["coef"])) == 0.5 and int(host(prob.view["skip"])) == 0


@pytest.mark.parametrize("sigma", [1e-3, 1e3, 1e-12])
def test_float32_step_against_binary64(gb, sigma):
    prob = Problem(gb, [(20011, "f32", "f32", False)], 23, sigma=sigma)
    prob.gradients()
    prob.step()
    prob.follow()
    h, e = prob.host[0], prob.entries[0]
    old = (f32(e.param), f32(e.grad), f32(e.m), f32(e.v))
    prob.gradients()
    g = f32(e.grad)
    prob.step(inv_scale=0.25)
    lr, w = float(np.float32(1e-3)), float(np.float32(0.1))
    want = P.adamw64(old[0], g, old[2], old[3], 2, 0.25, lr, 1.0, w)
    for name, x, y, b in zip("pmv", (e.param, e.m, e.v), want,
                             bounds(old[0], g, old[2], old[3], 2, 0.25, lr, 1.0, w)):
        assert (np.abs(f32(x).astype(np.float64) - y) <= b).all(), name
    assert h["n"] == 20011


def code_step(q):
    """Distance of the E4M3 codes around magnitudes q (the larger one at a border)."""
    return np.exp2(np.maximum(np.floor(np.log2(np.maximum(q, 2.0 ** -20))), -6) - 3)


@pytest.mark.parametrize("sigma", [1e-3, 1e3, 1e-12])
def test_8_bit_step_against_binary64(gb, sigma):
    """p' within the float32 step's bounds of binary64 from the decoded
    moments; m' and the root at most one code's distance from binary64's."""
    n = 20011
    prob = Problem(gb, [(n, "f32", "e4m3", False)], 24, sigma=sigma)
    for _ in range(3):
        prob.gradients()
        prob.step()
        prob.follow()
    h, e = prob.host[0], prob.entries[0]
    p, m, u = f32(e.param), P.decode(h["m"], h["ms"]), P.decode(h["v"], h["vs"])
    # u * u is rounded once before it is v: one more rounding of v
    v = u.astype(np.float64) ** 2
    prob.gradients()
    g = f32(e.grad)
    prob.step(inv_scale=0.5)
    lr, w = float(np.float32(1e-3)), float(np.float32(0.1))
    want = P.adamw64(p, g, m, v, 4, 0.5, lr, 1.0, w)
    bp, bm, bv = bounds(p, g, m, v, 4, 0.5, lr, 1.0, w)
    assert (np.abs(f32(e.param) - want[0]) <= bp).all()
    mags = np.append(P.E4M3, np.nan)
    for codes, scale, exact, err in ((e.m, e.m_scale, want[1], bm), (e.v, e.v_scale, np.sqrt(want[2]), np.sqrt(bv))):
        c, sc = host(codes).numpy(), np.repeat(f32(scale).astype(np.float64), 256)[:n]
        got = np.where(c & 0x80, -mags[c & 0x7F], mags[c & 0x7F]) * sc
        near = code_step(np.maximum(np.abs(got), np.abs(exact)) / sc) * sc
        assert (np.abs(got - exact) <= near + err).all()


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("sizes", [[1], [5], [1024 * 2048 + 77], [3, 1025, 100000, 7]])
def test_norm_against_binary64(gb, kind, sizes):
    prob = Problem(gb, [(n, kind, "f32", False) for n in sizes], 31, sigma=0.3)
    prob.gradients()
    gb.gb_optim_begin_clip(prob.plan, prob.control, 0.5, 0.01)
    total = math.fsum(float(np.square(f32(e.grad).astype(np.float64)).sum()) for e in prob.entries)
    norm = 0.01 * math.sqrt(total)
    # one rounding to binary32; the binary64 sums are far below it
    assert abs(float(host(prob.view["norm"])) - norm) <= norm * U * 1.001
    coef = 0.01 * min(1.0, 0.5 / norm)
    assert abs(float(host(prob.view["coef"])) - coef) <= coef * U * 1.001


@pytest.mark.parametrize("values", [[3e38, 3e38], [1e-45, 1e-40], [0.0, -0.0], [1e30, 1e-30]])
def test_norm_of_extreme_gradients(gb, values):
    prob = Problem(gb, [(2, "f32", "f32", False)], 1)
    prob.entries[0].grad.copy_(torch.tensor(values))
    prob.step(1.0, 0.5)
    prob.follow(1.0, 0.5)
    prob.check()


@pytest.mark.parametrize("state", ["f32", "e4m3"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_a_gradient_that_is_not_finite_skips_the_step(gb, kind, bad, state):
    prob = Problem(gb, [(1000, kind, state, kind != "f32"), (3000, kind, state, False)], 2)
    prob.gradients()
    prob.step(1.0)
    prob.follow(1.0)
    prob.gradients()
    prob.entries[1].grad[2999] = bad
    prob.step(1.0)
    norm = float(host(prob.view["norm"]))
    assert not math.isfinite(norm) and float(host(prob.view["coef"])) == 0.0
    assert int(host(prob.view["skip"])) == 1 and int(host(prob.view["skipped"])) == 1
    assert int(host(prob.view["step"])) == 1
    prob.check()  # everything as after the first step
    prob.gradients()
    prob.step(1.0)
    prob.follow(1.0)
    prob.check()
    assert int(host(prob.view["skipped"])) == 1


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_special_gradients_without_a_norm(gb, state):
    """Infinities, NaN, zeros, subnormals and the largest values reach the
    moments when no norm guards the step."""
    special = [0.0, -0.0, math.inf, -math.inf, math.nan, 1e-45, -1e-40, 3.4e38, -3.4e38, 1e19, 1e-20, 1e25]
    prob = Problem(gb, [(900, "f32", state, False), (300, "bf16", state, True)], 6)
    for k in range(3):
        prob.gradients(special if k == 0 else ())
        prob.step()
        prob.follow()
        if k == 0:
            for h in prob.host:
                assert np.isnan(h["p"][4])
        prob.check()


def test_moments_of_zero_and_tiny_gradients_in_8_bits(gb):
    """Blocks of zeros, of one value, and of a range wider than the codes."""
    prob = Problem(gb, [(256 * 6, "f32", "e4m3", False)], 9)
    g = np.zeros(256 * 6, np.float32)
    g[256] = 1.0
    g[512:768] = np.exp2(np.linspace(0, -60, 256))
    g[768:1024] = np.float32(1e-38)
    g[1024:1280] = np.exp2(np.linspace(-100, 20, 256))
    g[1280:] = -1e-3
    for _ in range(4):
        prob.entries[0].grad.copy_(torch.from_numpy(g))
        prob.step()
        prob.follow()
        prob.check()
    codes = host(prob.entries[0].v).numpy()
    assert not codes[:256].any() and not codes[257:512].any() and codes[512:768].all()


def test_the_codes_decode_through_the_library(gb):
    """gb_decode_sum reads the moments' payloads."""
    prob = Problem(gb, [(5000, "f32", "e4m3", False)], 14)
    for _ in range(3):
        prob.gradients()
        prob.step()
        prob.follow()
    e, h = prob.entries[0], prob.host[0]
    out = torch.empty(5000, device=DEV)
    for codes, scale, want in ((e.m, e.m_scale, P.decode(h["m"], h["ms"])), (e.v, e.v_scale, P.decode(h["v"], h["vs"]))):
        gb.gb_decode_sum(out, [codes], [scale], gb.GB_CODEC_FP8_E4M3_B256)
        assert (f32(out) == want).all()


@pytest.mark.parametrize("beta1,beta2,eps", [(0.0, 0.0, 1e-8), (0.95, 0.95, 1e-15), (0.9, 0.9999, 1e-3)])
@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_other_constants_and_a_late_step(gb, state, beta1, beta2, eps):
    prob = Problem(gb, [(3001, "f32", state, False)], 21, beta1=beta1, beta2=beta2, eps=eps)
    prob.view["step"].fill_(123456)
    prob.t = 123456
    for _ in range(2):
        prob.gradients()
        prob.step(1.0)
        prob.follow(1.0)
        prob.check()


def test_a_schedule_changes_the_rate_on_the_device(gb):
    prob = Problem(gb, [(2000, "f32", "f32", False)], 22)
    for lr in (1e-3, 5e-4, 0.0):
        prob.view["lr"].fill_(lr)
        prob.lr = lr
        prob.gradients()
        prob.step()
        prob.follow()
        prob.check()


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_captured_steps_replayed_between_eager_ones(gb, state):
    """Begin and step in a HIP graph, replayed with eager steps and
    synchronizations between the replays: the same bits as the oracle's."""
    prob = Problem(gb, [(40000, "bf16", state, True), (77, "f32", state, False)], 33)
    prob.gradients()
    prob.step(0.02)
    prob.follow(0.02)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        prob.step(0.02)
    for k in range(6):
        prob.gradients()
        torch.cuda.synchronize()
        if k % 3 == 2:
            prob.step(0.02)
        else:
            graph.replay()
        prob.follow(0.02)
        prob.check()


def test_on_another_stream(gb):
    prob = Problem(gb, [(30000, "f32", "e4m3", False)], 40)
    prob.gradients()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    prob.step(0.5, stream=side)
    side.synchronize()
    prob.follow(0.5)
    prob.check()


def test_runs_repeat_bit_for_bit(gb):
    """The norm's order is fixed by the plan: the same bits on every run."""
    got = set()
    for _ in range(5):
        prob = Problem(gb, [(3_000_001, "f32", "f32", False)], 50, sigma=0.37)
        prob.gradients()
        prob.step(1.0)
        torch.cuda.synchronize()
        got.add((float(host(prob.view["norm"])), host(prob.entries[0].param).numpy().tobytes()))
    assert len(got) == 1


@pytest.mark.parametrize("bits", [32, 33])
def test_a_tensor_beyond_32_bit_offsets(gb, bits):
    """2^32 + 517 values, and 2^33 + 517, which take a second launch: the
    last ones are updated as the oracle says, the dither counting from their
    position."""
    n = (1 << bits) + 517
    tail = 517 + 256 * 5
    p = torch.zeros(n, device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    m, v = (torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2))
    ms, vs = (torch.zeros(-(-n // 256), device=DEV) for _ in range(2))
    rng = np.random.default_rng(3)
    hg = (rng.standard_normal(tail) * 1e-3).astype(np.float32)
    g[n - tail:] = torch.from_numpy(hg).to(DEV)
    hg = f32(g[n - tail:])
    ws = torch.empty(gb.gb_optim_plan_bytes([n]), dtype=torch.uint8, device=DEV)
    plan = gb.gb_optim_plan([gb.GbOptimTensor(p, g, m, v, ms, vs)], ws, seed=5)
    control = torch.zeros(64, dtype=torch.uint8, device=DEV)
    view = gb.gb_optim_control(control)
    view["lr"].fill_(1e-3)
    z, zb = np.zeros(tail, np.float32), np.zeros(tail, np.uint8)
    hp, hm, hms, hv, hvs = z, zb, z[:-(-tail // 256)], zb, z[:-(-tail // 256)]
    for t in (1, 2):
        gb.gb_optim_begin_clip(plan, control, math.inf)
        gb.gb_adamw_step(plan, control)
        hp, hm, hms, hv, hvs = P.adamw_e4m3(hp, hg, hm, hms, hv, hvs, t, 1.0, 1e-3, 5, n - tail)
    same(f32(view["norm"]), np.array([P.grad_norm([hg], math.inf, 1.0)[0]]), "norm")
    same(f32(p[n - tail:]), hp, "param")
    same(host(m[n - tail:]).numpy(), hm, "m")
    same(host(v[n - tail:]).numpy(), hv, "v")
    same(f32(ms[-hms.size:]), hms, "m_scale")
    same(f32(vs[-hvs.size:]), hvs, "v_scale")
    assert not bool(p[:n - tail].any()) and not bool(m[:n - tail].any())


def test_the_binding_refuses_what_does_not_fit(gb):
    """Each with nothing enqueued: wrong types, sizes, strides and devices."""
    n = 1000
    f = lambda k=n, dt=torch.float32: torch.zeros(k, dtype=dt, device=DEV)  # noqa: E731
    ws = f(gb.gb_optim_plan_bytes([n]), torch.uint8)
    good = gb.GbOptimTensor(f(), f(), f(), f())
    coded = gb.GbOptimTensor(f(), f(), f(n, torch.uint8), f(n, torch.uint8), f(4), f(4))
    for bad, error, text in (
            (good._replace(param=f(n, torch.float16)), TypeError, "param must be torch.float32"),
            (good._replace(grad=f(n, torch.float64)), TypeError, "grad must be"),
            (good._replace(grad=f(n - 1)), ValueError, "grad has 999 elements"),
            (good._replace(m=f(n + 1)), ValueError, r"\.m has 1001 elements"),
            (good._replace(v=f(2 * n)[::2]), ValueError, r"\.v must be contiguous"),
            (good._replace(m=f(n, torch.bfloat16)), TypeError, r"\.m must be torch.float32"),
            (good._replace(param=torch.zeros(n)), ValueError, "param must be in device memory"),
            (good._replace(param=None), TypeError, "param must be a torch.Tensor"),
            (good._replace(copy=f(n, torch.float64)), TypeError, "copy must be torch.float16 or"),
            (good._replace(copy=f(n - 1, torch.float16)), ValueError, "copy has 999 elements"),
            (good._replace(m_scale=f(4)), gb.GbError, "scales, but float32"),
            (coded._replace(v=f()), TypeError, r"\.v must be torch.uint8"),
            (coded._replace(v_scale=None), TypeError, "v_scale must be a torch.Tensor"),
            (coded._replace(m_scale=f(3)), ValueError, "m_scale has 3 elements, expected 4")):
        with pytest.raises(error, match=text):
            gb.gb_optim_plan([bad], ws)
    with pytest.raises(gb.GbError, match="workspace"):
        gb.gb_optim_plan([good], ws[:256])
    with pytest.raises(gb.GbError, match="overlaps"):
        gb.gb_optim_plan([good._replace(grad=good.param)], ws)
    plan = gb.gb_optim_plan([good, coded], f(gb.gb_optim_plan_bytes([n, n]), torch.uint8))
    control = torch.zeros(64, dtype=torch.uint8, device=DEV)
    for bad, error in ((control[:32], ValueError), (control.view(torch.float32), TypeError), (control.cpu(), ValueError),
                       (None, TypeError)):
        with pytest.raises(error):
            gb.gb_adamw_step(plan, bad)
    with pytest.raises(gb.GbError, match="inv_scale"):
        gb.gb_optim_begin(plan, control, 0.0)
    with pytest.raises(gb.GbError, match="max_norm"):
        gb.gb_optim_begin_clip(plan, control, -1.0)
    assert not bool(host(control).any())


def test_a_norm_beyond_binary32_skips_the_step_too(gb):
    """Finite gradients whose norm is not: four of 3e38."""
    prob = Problem(gb, [(4, "f32", "f32", False)], 3)
    prob.entries[0].grad.fill_(3e38)
    prob.step(1.0)
    prob.follow(1.0)
    assert int(host(prob.view["skip"])) == 1 and int(host(prob.view["step"])) == 0
    prob.check()
    prob.step(1.0, 0.25)  # scaled by the loss scale's reciprocal it fits
    prob.follow(1.0, 0.25)
    assert int(host(prob.view["skip"])) == 0 and int(host(prob.view["step"])) == 1
    prob.check()
