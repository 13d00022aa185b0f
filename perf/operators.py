"""What is measured of the optimizer operators: the global gradient norm with
clipping, and the AdamW step over many tensors with its two moments held in
32 bits or in 8.

A case is one of three passes:
  clip    the norm of all gradients together and the factor that scales them
          (gb_optim_begin_clip);
  adamw   a training step's update with float32 moments (gb_optim_begin, or
          gb_optim_begin_clip where the case clips, then gb_adamw_step);
  adamw8  the same with the moments in 8 bits.

The tensors of a case lie in flat buffers, each tensor starting at a multiple
of 256 values and the gap after its last value holding zeros, which every
formula here maps to zeros.  So the plain form works on whole buffers, while
the framework gets the separate tensors.

The formulas, in binary32 with every operation rounded on its own:
  t = step + 1, r_i = 1 - beta_i^t (binary64), gs = g * coef
  m' = beta1 m + (1 - beta1) gs          v' = beta2 v + (1 - beta2) gs^2
  p' = p (1 - lr_t wd) - (lr_t / r_1) * m' / (sqrt(v') / sqrt(r_2) + eps)
with lr_t = lr * lr_scale of the tensor.  The 8-bit moments are m and
u = sqrt(v), as E4M3 codes with one power-of-two scale per 256 values, rounded
up or down by a dither made from the seed, the step and the value's position
(so that the averages stay right although a step moves them by less than the
distance of two codes); a root above zero keeps a code above zero.
"""
import random

import torch

own = False

BLOCK = 256
BETA1, BETA2, EPS, LR = 0.9, 0.999, 1e-8, 1e-3
MAX_NORM, INV_SCALE = 1.0, 1.0 / 1024.0
START_STEP = 1000
SEED = 20240
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}

DDP_N = 1_000_000_000  # the model of the repository's bucket-stream benchmark
BUCKET = 6_553_600  # its 25 MiB buckets
SHARD_BUCKET = 819_200  # one GPU's 1/8 share of such a bucket


def listed():
    return [
        # a few tiny tensors (a bias, a gain, a small head): the call's latency
        {"name": "clip_tiny_f32", "kind": "clip", "type": "f32", "layout": "mixed", "count": 6, "low": 1, "high": 4097,
         "sizes_seed": 1},
        # the ragged parameter list of a model held in bfloat16
        {"name": "clip_mixed_bf16", "kind": "clip", "type": "bf16", "layout": "mixed", "count": 300, "low": 1,
         "high": 1 << 20, "sizes_seed": 2},
        # every gradient of a 1e9-parameter model in 25 MiB buckets, after the all-reduce
        {"name": "clip_ddp_f32", "kind": "clip", "type": "f32", "layout": "buckets", "n": DDP_N, "bucket": BUCKET},
        # a few tiny tensors: the latency of a whole unclipped step
        {"name": "adamw_tiny_f32", "kind": "adamw", "type": "f32", "layout": "mixed", "count": 6, "low": 1,
         "high": 4097, "sizes_seed": 3, "clip": False, "copy": False},
        # a model's ragged parameter list, clipped: float32 training
        {"name": "adamw_mixed_f32", "kind": "adamw", "type": "f32", "layout": "mixed", "count": 300, "low": 1,
         "high": 1 << 20, "sizes_seed": 4, "clip": True, "copy": False},
        # one large tensor (an embedding) in mixed precision: bfloat16 gradient and model copy, float32 master
        {"name": "adamw_one_bf16", "kind": "adamw", "type": "bf16", "layout": "buckets", "n": 1 << 26,
         "bucket": 1 << 26, "clip": False, "copy": True},
        # the whole 1e9-parameter step on float32 buckets, clipped
        {"name": "adamw_ddp_f32", "kind": "adamw", "type": "f32", "layout": "buckets", "n": DDP_N, "bucket": BUCKET,
         "clip": True, "copy": False},
        # a few tiny tensors of float16 training with a loss scale
        {"name": "adamw8_tiny_f16", "kind": "adamw8", "type": "f16", "layout": "mixed", "count": 6, "low": 1,
         "high": 4097, "sizes_seed": 5, "clip": True, "copy": True},
        # a model's ragged parameter list with 8-bit moments
        {"name": "adamw8_mixed_f32", "kind": "adamw8", "type": "f32", "layout": "mixed", "count": 300, "low": 1,
         "high": 1 << 20, "sizes_seed": 6, "clip": False, "copy": False},
        # one GPU's eighth of the 1e9-parameter model: a sharded optimizer
        {"name": "adamw8_shard_bf16", "kind": "adamw8", "type": "bf16", "layout": "buckets", "n": DDP_N // 8,
         "bucket": SHARD_BUCKET, "clip": False, "copy": True},
        # the whole 1e9-parameter step, mixed precision, clipped, 8-bit moments
        {"name": "adamw8_ddp_bf16", "kind": "adamw8", "type": "bf16", "layout": "buckets", "n": DDP_N,
         "bucket": BUCKET, "clip": True, "copy": True},
    ]


def draw(rng):
    case = {"kind": rng.choice(["clip", "adamw", "adamw8"]), "type": rng.choice(["f32", "f16", "bf16"])}
    if rng.random() < 0.5:
        n = int(2 ** rng.uniform(8.0, 29.0)) | 1
        case |= {"layout": "buckets", "n": n, "bucket": max(256, int(2 ** rng.uniform(12.0, 24.0)), n // 500)}
    else:
        case |= {"layout": "mixed", "count": int(2 ** rng.uniform(0.0, 9.0)), "low": 1,
                 "high": int(2 ** rng.uniform(8.0, 22.0)) + 1, "sizes_seed": rng.randrange(1 << 20)}
    if case["kind"] != "clip":
        case |= {"clip": rng.random() < 0.5, "copy": case["type"] != "f32" and rng.random() < 0.7}
    return case


def sizes(case):
    """Values of each tensor of a case."""
    if case["layout"] == "buckets":
        return [min(case["bucket"], case["n"] - s) for s in range(0, case["n"], case["bucket"])]
    r = random.Random(case["sizes_seed"])
    span = case["high"] / case["low"]
    return [max(1, min(case["high"], int(case["low"] * span ** r.random()))) for _ in range(case["count"])]


def work(case):
    ns = sizes(case)
    n, blocks, e = sum(ns), sum(-(-v // BLOCK) for v in ns), SIZE[case["type"]]
    if case["kind"] == "clip":
        return {"bytes": n * e + 8, "flops": 2 * n}
    moments = 16 * n if case["kind"] == "adamw" else 4 * n + 16 * blocks
    return {"bytes": 8 * n + n * e * (2 if case["copy"] else 1) + moments,
            "flops": n * ((16 if case["clip"] else 14) + (16 if case["kind"] == "adamw8" else 0))}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _pow2_scale(a):
    """The smallest 2^e, e >= -126, with a <= 448 * 2^e; 1 for a = 0."""
    frac, exp = torch.frexp(a)
    e = torch.where(frac <= 0.875, exp - 9, exp - 8).clamp(min=-126)
    s = ((e + 127) << 23).to(torch.int32).view(torch.float32)
    return torch.where(a == 0, torch.ones_like(a), s)


def _nearest8(x):
    """Codes and scales of x as a state that some earlier step left behind."""
    x = x.view(-1, BLOCK)
    s = _pow2_scale(x.abs().amax(1))
    return (x / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(-1), s


def prepare(case, seed):
    dev = torch.device("cuda")
    ns = sizes(case)
    starts, at = [], 0
    for n in ns:
        starts.append(at)
        at += -(-n // BLOCK) * BLOCK
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    in_tensor = torch.ones(at, dtype=torch.bool, device=dev)
    for s, n in zip(starts, ns):
        if n % BLOCK:
            in_tensor[s + n:s + -(-n // BLOCK) * BLOCK] = False

    def normal(sigma):
        return torch.randn(at, generator=gen, device=dev).mul_(sigma).mul_(in_tensor)

    # gradients N(0, 1e-3) with 1% outliers a hundred times as large, under a loss scale of 1024
    g = normal(1e-3 / INV_SCALE)
    g.mul_(torch.where(torch.rand(at, generator=gen, device=dev) < 0.01, 100.0, 1.0))
    s = {"case": case, "g": g.to(TYPES[case["type"]])}
    del g
    control = torch.zeros(64, dtype=torch.uint8, device=dev)
    s |= {"control": control, "step": control[0:8].view(torch.int64), "lr": control[16:20].view(torch.float32),
          "norm": control[20:24].view(torch.float32), "coef": control[24:28].view(torch.float32)}
    s["step"].fill_(START_STEP)
    s["lr"].fill_(LR)
    blocks = at // BLOCK
    # weight decay on every other tensor and a smaller rate on every third, as parameter groups have them
    s["wd"] = [0.1 if i % 2 == 0 else 0.0 for i in range(len(ns))]
    s["rate"] = [0.5 if i % 3 == 2 else 1.0 for i in range(len(ns))]
    per = torch.tensor([-(-n // BLOCK) for n in ns], device=dev)
    of = lambda v: torch.repeat_interleave(torch.tensor(v, device=dev), per, output_size=blocks)[:, None]  # noqa: E731
    s["wd_of"], s["rate_of"] = of(s["wd"]), of(s["rate"])
    s["p"] = normal(0.02)
    m, u = normal(3e-4), normal(1e-3).abs_().add_(2e-4).mul_(in_tensor)
    if case["kind"] == "adamw8":
        (s["m"], s["ms"]), (s["v"], s["vs"]) = _nearest8(m), _nearest8(u)
    else:
        s["m"], s["v"] = m, u.square_()
    s["copy"] = s["p"].to(TYPES[case["type"]]) if case.get("copy") else None
    if own:
        import gradient_all_reduce_amd as gb

        def part(name, i):
            if s.get(name) is None:
                return None
            if name in ("ms", "vs"):
                return s[name][starts[i] // BLOCK:starts[i] // BLOCK + -(-ns[i] // BLOCK)]
            return s[name][starts[i]:starts[i] + ns[i]]

        tensors = [gb.GbOptimTensor(part("p", i), part("g", i), part("m", i), part("v", i), part("ms", i),
                                    part("vs", i), part("copy", i), lr_scale=s["rate"][i], weight_decay=s["wd"][i])
                   for i in range(len(ns))]
        s["workspace"] = torch.empty(gb.gb_optim_plan_bytes(ns), dtype=torch.uint8, device=dev)
        s["plan"] = gb.gb_optim_plan(tensors, s["workspace"], beta1=BETA1, beta2=BETA2, eps=EPS, seed=SEED)
        s["gb"] = gb
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    case = s["case"]
    clip = case["kind"] == "clip" or case["clip"]
    if own:
        gb = s["gb"]
        if clip:
            gb.gb_optim_begin_clip(s["plan"], s["control"], MAX_NORM, INV_SCALE)
        else:
            gb.gb_optim_begin(s["plan"], s["control"], INV_SCALE)
        if case["kind"] != "clip":
            gb.gb_adamw_step(s["plan"], s["control"])
        out = {"norm": s["norm"], "coef": s["coef"]} if clip else {}
    else:
        out = _plain_clip(s) if clip else {}
        coef = out["coef"] if clip else torch.full((1,), INV_SCALE, device=s["g"].device)
        s["step"] += 1
        if case["kind"] != "clip":
            _plain_adamw(s, coef)
    out["step"] = s["step"]
    if case["kind"] != "clip":
        out["p"] = s["p"]
        if case["kind"] == "adamw8":
            # the codes as the E4M3 values they are, with their scales
            out |= {"m": s["m"].view(torch.float8_e4m3fn), "m_scale": s["ms"],
                    "u": s["v"].view(torch.float8_e4m3fn), "u_scale": s["vs"]}
        else:
            out |= {"m": s["m"], "v": s["v"]}
        if s["copy"] is not None:
            out["copy"] = s["copy"]
    return out


def _plain_clip(s):
    norm = INV_SCALE * s["g"].double().square_().sum().sqrt().view(1)  # a long sum: 64 bits
    coef = torch.where(norm > MAX_NORM, INV_SCALE * MAX_NORM / norm, INV_SCALE)
    return {"norm": norm.float(), "coef": coef.float()}


def _plain_adamw(s, coef):
    case, t = s["case"], s["step"].double()
    r1 = (1.0 / (1.0 - BETA1 ** t)).float()
    r2 = (1.0 / (1.0 - BETA2 ** t).sqrt()).float()
    gs = s["g"].float() * coef
    if case["kind"] == "adamw8":
        m = (s["m"].view(torch.float8_e4m3fn).float().view(-1, BLOCK) * s["ms"][:, None]).view(-1)
        u = (s["v"].view(torch.float8_e4m3fn).float().view(-1, BLOCK) * s["vs"][:, None]).view(-1)
        v = u * u
    else:
        m, v = s["m"], s["v"]
    m = BETA1 * m + (1.0 - BETA1) * gs
    v = BETA2 * v + (1.0 - BETA2) * (gs * gs)
    del gs
    u = v.sqrt()
    update = m / (u * r2 + EPS)
    lr = s["lr"] * s["rate_of"]
    p = s["p"].view(-1, BLOCK)
    p.copy_(p * (1.0 - lr * s["wd_of"]) - (lr * r1) * update.view(-1, BLOCK))
    del update
    if case["kind"] == "adamw8":
        dither = _plain_dither(s["step"], s["p"].numel())
        codes, scale = _plain_encode(m, dither)
        s["m"].copy_(codes + (m.view(torch.int32) < 0) * 128)
        s["ms"].copy_(scale)
        codes, scale = _plain_encode(u, dither)
        s["v"].copy_(torch.where(u > 0, codes.clamp(min=1), codes))
        s["vs"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    if s["copy"] is not None:
        s["copy"].copy_(s["p"])


def _plain_encode(x, dither):
    """E4M3 magnitudes of x over its block's power of two: the 20 bits of the
    significand below the code's last are added to the dither, and what
    carries rounds up."""
    x = x.view(-1, BLOCK)
    scale = _pow2_scale(x.abs().amax(1))
    q = (x.abs() / scale[:, None]).view(-1)
    small = q < 2.0 ** -6
    fine = (torch.where(small, q, 0.0) * 2.0 ** 29).to(torch.int32)
    return torch.where(small, (fine + dither) >> 20, ((q.view(torch.int32) + dither) >> 20) - 960), scale


def _plain_dither(step, n):
    """20 bits for each of n values, two values to a 32-bit word."""
    golden, low = 0x9E3779B97F4A7C15 - (1 << 64), 0xFFFFFFFF
    z = SEED + step * golden
    for _ in range(3):
        z = (z ^ ((z >> 32) & low)) * golden
    x = (torch.arange(n // 2, device=step.device) * 0x9E3779B9 + ((z >> 32) & low)) & low
    x = ((x ^ (x >> 15)) * 0x6A09E667) & low
    x = x ^ (x >> 16)
    return torch.stack([x >> 12, (x << 4) & 0xFFFF0], 1).view(-1).to(torch.int32)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _value64(codes, scales):
    """What E4M3 codes and their blocks' scales stand for."""
    c = codes.to(torch.int64)
    exp, frac = (c >> 3) & 15, (c & 7).double()
    size = torch.where(exp > 0, (8.0 + frac) * torch.exp2((exp - 10).double()), frac * 2.0 ** -9)
    return torch.where(c > 127, -size, size).view(-1, BLOCK) * scales.double()[:, None]


def exact(case, seed):
    s = prepare(case, seed)
    t, f = START_STEP + 1, INV_SCALE
    g = s["g"].double()
    out = {"step": None}
    if case["kind"] == "clip" or case["clip"]:
        total = torch.linalg.vector_norm(g) * INV_SCALE
        f = INV_SCALE * min(1.0, MAX_NORM / float(total))
        out |= {"norm": total.view(1), "coef": torch.tensor([f], dtype=torch.float64)}
    if case["kind"] == "clip":
        return out
    g = (g * f).view(-1, BLOCK)
    if case["kind"] == "adamw8":
        m, v = _value64(s["m"], s["ms"]), _value64(s["v"], s["vs"]) ** 2
    else:
        m, v = s["m"].double().view(-1, BLOCK), s["v"].double().view(-1, BLOCK)
    m = m + (1.0 - BETA1) * (g - m)
    v = v + (1.0 - BETA2) * (g ** 2 - v)
    lr = LR * s["rate_of"].double()
    p = s["p"].double().view(-1, BLOCK)
    p = p - lr * s["wd_of"].double() * p - lr * (m / (1.0 - BETA1 ** t)) / ((v / (1.0 - BETA2 ** t)) ** 0.5 + EPS)
    out["p"] = p.view(-1)
    if case["kind"] == "adamw8":
        out |= {"m": None, "m_scale": None, "u": None, "u_scale": None}  # rounded by the dither: no such value
    else:
        out |= {"m": m.view(-1), "v": v.view(-1)}
    if s["copy"] is not None:
        out["copy"] = p.view(-1)
    return out
