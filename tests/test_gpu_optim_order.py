"""The optimizer step where it takes another path than a small plan does:
- the permuted order of the step's workgroups, from 8,192 of them (2^21
  values), and the norm over more chunks than it has wavefronts (4,096), both
  against the oracle bit for bit;
- the float32 step's launch from 2^27 values, which reserves more LDS, bit for
  bit against the same step over slices that keep the index order;
- the norm over more gradients than it leaves in the last-level cache;
- the 8-bit step over more than 2^33 values, where every block leaves a mark.

Every block has values that the step changes, so one that no workgroup took, or
that two took, shows as a difference.  Sizes end in a ragged tail that is not
a whole number of runs of the permutation."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from tests.test_gpu_optim import DEV, U, Problem, f32, host, same  # noqa: E402

BLOCK = 256


@pytest.fixture(scope="module")
def gb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_all_reduce_amd as lib
    return lib


def every_block_changed(before, after):
    """Whether each block of 256 values has one whose bits changed."""
    changed = before.view(np.uint32) != after.view(np.uint32)
    return np.logical_or.reduceat(changed, np.arange(0, changed.size, BLOCK)).all()


def two_clipped_steps(prob):
    for _ in range(2):
        prob.gradients()
        before = [h["p"] for h in prob.host]
        prob.step(0.5, 0.25)
        prob.follow(0.5, 0.25)
        assert all(every_block_changed(b, h["p"]) for b, h in zip(before, prob.host))
        prob.check()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("state", ["f32", "e4m3"])
@pytest.mark.parametrize("n", [(1 << 21) + 8193, 5_000_001])
def test_one_tensor_in_the_permuted_order(gb, n, state, kind):
    two_clipped_steps(Problem(gb, [(n, kind, state, kind == "bf16")], 70, shift=n % 2))


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_many_tensors_in_the_permuted_order(gb, state):
    """Runs of the permutation across ragged tensors, and a second launch of
    another gradient type in the plan."""
    rng = np.random.default_rng(71)
    spec = [(int(n), "f32", state, False) for n in rng.integers(1, 120_000, 60)]
    spec += [(int(n), "f16", state, True) for n in rng.integers(1, 120_000, 55)]
    assert all(sum(n for n, kind, _, _ in spec if kind == k) > 1 << 21 for k in ("f32", "f16"))
    two_clipped_steps(Problem(gb, spec, 72))


@pytest.mark.parametrize("n", [(1 << 24) + 4097, (1 << 27) + 517])
def test_a_large_float32_step_is_that_of_its_slices(gb, n):
    step = 2_000_000 // BLOCK * BLOCK  # below 2^21: index order
    gen = torch.Generator(device=DEV).manual_seed(73)

    def normal(sigma):
        return torch.randn(n, generator=gen, device=DEV).mul_(sigma)

    p, g, m, v = normal(0.02), normal(1e-3), normal(1e-4), normal(1e-3).square_()
    whole, parts = [p.clone(), m.clone(), v.clone()], [p.clone(), m.clone(), v.clone()]

    def run(pmv, ranges):
        for s, e in ranges:
            control = torch.zeros(64, dtype=torch.uint8, device=DEV)
            gb.gb_optim_control(control)["lr"].fill_(1e-3)
            a, b, c = (x[s:e] for x in pmv)
            ws = torch.empty(gb.gb_optim_plan_bytes([e - s]), dtype=torch.uint8, device=DEV)
            plan = gb.gb_optim_plan([gb.GbOptimTensor(a, g[s:e], b, c, weight_decay=0.1)], ws)
            for _ in range(2):
                gb.gb_optim_begin(plan, control, 0.5)
                gb.gb_adamw_step(plan, control)
            torch.cuda.synchronize()

    run(whole, [(0, n)])
    run(parts, [(s, min(s + step, n)) for s in range(0, n, step)])
    for name, x, y, start in zip("pmv", whole, parts, (p, m, v)):
        assert torch.equal(x.view(torch.int32), y.view(torch.int32)), name
        moved = torch.nn.functional.pad(x != start, (0, -n % BLOCK)).view(-1, BLOCK).any(1)
        assert bool(moved.all()), name


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_the_norm_of_more_than_the_cache_holds(gb, kind):
    n = 180_000_011 if kind is torch.float32 else 360_000_011  # above 640 MiB of gradients
    gen = torch.Generator(device=DEV).manual_seed(74)
    g = torch.randn(n, generator=gen, device=DEV).mul_(0.3).to(kind)
    p, m, v = (torch.zeros(n, device=DEV) for _ in range(3))
    ws = torch.empty(gb.gb_optim_plan_bytes([n]), dtype=torch.uint8, device=DEV)
    plan = gb.gb_optim_plan([gb.GbOptimTensor(p, g, m, v)], ws)
    control = torch.zeros(64, dtype=torch.uint8, device=DEV)
    gb.gb_optim_begin_clip(plan, control, math.inf)
    norm = math.sqrt(sum(float(x.double().square().sum()) for x in g.split(1 << 24)))
    # one rounding to binary32; the binary64 sums are far below it
    assert abs(float(host(gb.gb_optim_control(control)["norm"])) - norm) <= norm * U * 1.001


def test_no_block_is_left_out_beyond_2_33_values(gb):
    """Scales start at 0; a block of zeros that was stepped stores 1."""
    n = (1 << 33) + 517
    p = torch.zeros(n, device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    m, v = (torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2))
    ms, vs = (torch.zeros(-(-n // BLOCK), device=DEV) for _ in range(2))
    ws = torch.empty(gb.gb_optim_plan_bytes([n]), dtype=torch.uint8, device=DEV)
    plan = gb.gb_optim_plan([gb.GbOptimTensor(p, g, m, v, ms, vs)], ws)
    control = torch.zeros(64, dtype=torch.uint8, device=DEV)
    gb.gb_optim_begin(plan, control)
    gb.gb_adamw_step(plan, control)
    assert bool((ms == 1).all()) and bool((vs == 1).all())
