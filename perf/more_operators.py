"""What is measured of the token-sum operators: the two layers of a language
model whose parameters' gradients are sums over tokens, with those sums
delivered where the gradient buckets want them.

A case is one of four passes:
  norm       layer norm, forward (gb_layer_norm_forward)
  norm_grad  its gradients: of the input, and of weight and bias summed over
             all rows (gb_layer_norm_backward)
  look       embedding lookup with scaling (gb_embedding_forward)
  look_grad  the table's gradient: the rows of every token summed by id
             (gb_embedding_backward)

The formulas, every sum in 32 bits, each output rounded once to its type:
  norm       mean = sum x / n, rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
             y = (x - mean) rstd w + b
  norm_grad  h = (x - mean) rstd, g = dy w
             dx = rstd (g - sum g / n - h sum(g h) / n)
             dw = [dw +] sum over rows of dy h, db = [db +] sum over rows of dy
  look       out[t] = scale table[ids[t] - first], zeros for an id outside
             [first, first + vocab)
  look_grad  dtable[v] = [dtable[v] +] scale (sum of dout[t] with ids[t] = first + v),
             an id equal to padding left out
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
IDS = {"i32": torch.int32, "i64": torch.int64}
EPS = 1e-5


def listed():
    return [
        # four sequences generating one token each: the call's latency
        {"name": "norm_decode_bf16", "kind": "norm", "rows": 4, "cols": 4096, "type": "bf16", "param": "bf16",
         "bias": True, "stats": False, "wider": 0},
        # a norm over each head's 128 values, read out of a wider projection: many short rows
        {"name": "norm_heads_f16", "kind": "norm", "rows": 65_536, "cols": 128, "type": "f16", "param": "f32",
         "bias": False, "stats": True, "wider": 256},
        # a training batch of 16,384 tokens in mixed precision, float32 parameters
        {"name": "norm_train_bf16", "kind": "norm", "rows": 16_384, "cols": 8192, "type": "bf16", "param": "f32",
         "bias": True, "stats": True, "wider": 0},
        # a small float32 model with an odd width, gradients written anew
        {"name": "norm_grad_small_f32", "kind": "norm_grad", "rows": 512, "cols": 771, "type": "f32", "param": "f32",
         "grad": "f32", "bias": True, "accumulate": False},
        # a training batch in mixed precision, a micro-batch's share added to float32 buckets
        {"name": "norm_grad_train_bf16", "kind": "norm_grad", "rows": 16_384, "cols": 4096, "type": "bf16",
         "param": "f32", "grad": "f32", "bias": True, "accumulate": True},
        # long ragged rows of a wide float16 model, gradients in the model's type
        {"name": "norm_grad_wide_f16", "kind": "norm_grad", "rows": 5003, "cols": 12_289, "type": "f16",
         "param": "f16", "grad": "f16", "bias": False, "accumulate": False},
        # eight sequences generating one token each: the call's latency
        {"name": "look_decode_bf16", "kind": "look", "tokens": 8, "vocab": 131_072, "dim": 4096, "table": "bf16",
         "out": "bf16", "ids": "i64", "first": 0, "ranks": 1},
        # one GPU's quarter of a vocabulary of 50,003: most ids belong to other GPUs and give zeros
        {"name": "look_shard_f16", "kind": "look", "tokens": 7001, "vocab": 12_501, "dim": 1001, "table": "f16",
         "out": "f16", "ids": "i32", "first": 12_501, "ranks": 4},
        # a training batch out of a float32 master table into bfloat16 activations
        {"name": "look_train_f32", "kind": "look", "tokens": 32_768, "vocab": 131_072, "dim": 4096, "table": "f32",
         "out": "bf16", "ids": "i64", "first": 0, "ranks": 1},
        # a small float32 model: few tokens, a small table
        {"name": "look_grad_small_f32", "kind": "look_grad", "tokens": 512, "vocab": 2000, "dim": 257, "type": "f32",
         "grad": "f32", "ids": "i64", "accumulate": False, "padding": 0},
        # a micro-batch's share added to the bucket of a table: only the rows it names are touched
        {"name": "look_grad_micro_bf16", "kind": "look_grad", "tokens": 98_304, "vocab": 50_003, "dim": 1024,
         "type": "bf16", "grad": "f32", "ids": "i32", "accumulate": True, "padding": -1},
        # the whole table's gradient written into its bucket, most rows of it zeros
        {"name": "look_grad_table_bf16", "kind": "look_grad", "tokens": 16_384, "vocab": 131_072, "dim": 4096,
         "type": "bf16", "grad": "f32", "ids": "i64", "accumulate": False, "padding": -1},
    ]


def draw(rng):
    def spread(low, high):
        return max(low, min(high, int(2 ** rng.uniform(math.log2(low), math.log2(high + 1)))))

    kind = rng.choice(["norm", "norm_grad", "look", "look_grad"])
    t, u = rng.choice(list(TYPES)), rng.choice(list(TYPES))
    most = max(work(c)["bytes"] for c in listed() if c["kind"] == kind)
    while True:
        if kind in ("norm", "norm_grad"):
            case = {"kind": kind, "rows": spread(1, 131_072), "cols": spread(16, 16_384), "type": t,
                    "param": rng.choice([t, "f32"]), "bias": rng.random() < 0.7}
            if kind == "norm":
                case |= {"stats": rng.random() < 0.7, "wider": rng.choice([0, 0, 0, 1, 64, 1000])}
            else:
                case |= {"grad": rng.choice([t, "f32"]), "accumulate": rng.random() < 0.5}
        else:
            case = {"kind": kind, "tokens": spread(1, 131_072), "vocab": spread(16, 262_144), "dim": spread(16, 8192),
                    "ids": rng.choice(list(IDS))}
            if kind == "look":
                ranks = rng.choice([1, 1, 2, 8])
                case |= {"table": t, "out": u, "first": rng.randrange(ranks) * case["vocab"], "ranks": ranks}
            else:
                case |= {"type": t, "grad": rng.choice([t, "f32"]), "accumulate": rng.random() < 0.5,
                         "padding": rng.choice([-1, -1, 0])}
        if work(case)["bytes"] <= most and case.get("vocab", 0) * case.get("dim", 0) <= 1 << 29:
            return case


def rows_named(case):
    """How many different rows of a table the ids of a case name, as a mean over seeds."""
    if "vocab" not in case:
        return 0
    span, n = case["vocab"] * case.get("ranks", 1), case["tokens"]
    low, high = case.get("first", 0) + 1, case.get("first", 0) + case["vocab"]
    total, at = 0.0, low
    while at <= high:  # ids 2^j .. 2^(j + 1) are alike enough to be counted together
        to = min(high, max(at, 2 * at - 1))
        p = math.log((to + 1) / at) / math.log(span + 1) / (to + 1 - at)
        total += (to + 1 - at) * (1.0 - (1.0 - p) ** n)
        at = to + 1
    return total


def work(case):
    if case["kind"] in ("norm", "norm_grad"):
        m, n, e, p = case["rows"], case["cols"], SIZE[case["type"]], SIZE[case["param"]]
        if case["kind"] == "norm":
            return {"bytes": 2 * m * n * e + n * p * (2 if case["bias"] else 1) + (8 * m if case["stats"] else 0),
                    "flops": 8 * m * n}
        grads = n * SIZE[case["grad"]] * (2 if case["bias"] else 1) * (2 if case["accumulate"] else 1)
        return {"bytes": 3 * m * n * e + 8 * m + n * p + grads, "flops": 16 * m * n}
    t, d, i = case["tokens"], case["dim"], 4 if case["ids"] == "i32" else 8
    if case["kind"] == "look":
        return {"bytes": int(rows_named(case) * d * SIZE[case["table"]]) + t * d * SIZE[case["out"]] + t * i,
                "flops": t * d}
    rows = 2 * rows_named(case) if case["accumulate"] else case["vocab"]
    return {"bytes": t * d * SIZE[case["type"]] + t * i + int(rows * d * SIZE[case["grad"]]), "flops": t * d}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = {"case": case}
    if case["kind"] in ("norm", "norm_grad"):
        m, n, t = case["rows"], case["cols"], TYPES[case["type"]]
        # a residual stream: rows of different size, a few channels far larger than the others
        x = normal(m, n).mul_(normal(m, 1).exp_())
        x.mul_(torch.where(torch.rand(n, generator=gen, device=dev) < 0.004, 20.0, 1.0)).add_(0.1 * normal(n))
        wide = torch.zeros(m, n + case.get("wider", 0), dtype=t, device=dev)
        wide[:, :n] = x
        s["x"] = wide[:, :n]
        del x
        s["w"] = (1.0 + 0.1 * normal(n)).to(TYPES[case["param"]])
        s["b"] = (0.1 * normal(n)).to(TYPES[case["param"]]) if case["bias"] else None
        if case["kind"] == "norm":
            s["y"] = torch.empty(m, n, dtype=t, device=dev)
            s["mean"], s["rstd"] = (torch.empty(m, device=dev) if case["stats"] else None for _ in range(2))
        else:
            var, mean = torch.var_mean(s["x"].double(), 1, correction=0)
            s["mean"], s["rstd"] = mean.float(), (var + EPS).rsqrt().float()
            s["dy"] = (1e-3 * normal(m, n)).to(t)
            s["dx"] = torch.empty(m, n, dtype=t, device=dev)
            s["dw"], s["db"] = (1e-2 * normal(n)).to(TYPES[case["grad"]]), None
            if case["bias"]:
                s["db"] = (1e-2 * normal(n)).to(TYPES[case["grad"]])
    else:
        # ids as frequent as words are: the one of rank r about 1 / r times as often as the first
        span = case["vocab"] * case.get("ranks", 1)
        u = torch.rand(case["tokens"], generator=gen, device=dev, dtype=torch.float64)
        ids = torch.exp(u * math.log(span + 1)).long() - 1
        s["ids"] = ids.clamp_(0, span - 1).to(IDS[case["ids"]])
        s["scale"] = math.sqrt(case["dim"])
        if case["kind"] == "look":
            s["table"] = (0.02 * normal(case["vocab"], case["dim"])).to(TYPES[case["table"]])
            s["out"] = torch.empty(case["tokens"], case["dim"], dtype=TYPES[case["out"]], device=dev)
        else:
            s["dout"] = (1e-3 * normal(case["tokens"], case["dim"])).to(TYPES[case["type"]])
            s["dtable"] = (1e-2 * normal(case["vocab"], case["dim"])).to(TYPES[case["grad"]])
    if own:
        import gradient_all_reduce_amd as gb
        s["gb"], need = gb, 0
        if case["kind"] == "norm_grad":
            need = gb.gb_layer_norm_workspace_bytes(case["rows"], case["cols"])
        if case["kind"] == "look_grad":
            need = gb.gb_embedding_workspace_bytes(case["tokens"], case["vocab"], case["dim"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    return _PASS[s["case"]["kind"]](s)


def _norm(s):
    if own:
        s["gb"].gb_layer_norm_forward(s["y"], s["x"], s["w"], s["b"], eps=EPS, mean=s["mean"], rstd=s["rstd"])
        y, mean, rstd = s["y"], s["mean"], s["rstd"]
    else:
        x = s["x"].float()
        mean = x.sum(1) / x.shape[1]
        x = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((x * x).sum(1) / x.shape[1] + EPS)
        y = x * rstd[:, None] * s["w"].float()
        if s["b"] is not None:
            y = y + s["b"].float()
        y = y.to(s["x"].dtype)
    return {"y": y, "mean": mean, "rstd": rstd} if s["case"]["stats"] else {"y": y}


def _norm_grad(s):
    if own:
        s["gb"].gb_layer_norm_backward(s["dx"], s["dw"], s["db"], s["dy"], s["x"], s["mean"], s["rstd"], s["w"],
                                       accumulate=s["case"]["accumulate"], workspace=s["workspace"])
        out = {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
    else:
        n = s["x"].shape[1]
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        h = (s["x"].float() - s["mean"][:, None]) * rstd
        g = dy * s["w"].float()
        dx = rstd * (g - g.sum(1, keepdim=True) / n - h * ((g * h).sum(1, keepdim=True) / n))
        out = {"dx": dx.to(s["x"].dtype), "dw": _into(s, "dw", (dy * h).sum(0)), "db": None}
        if s["db"] is not None:
            out["db"] = _into(s, "db", dy.sum(0))
    return {k: v for k, v in out.items() if v is not None}


def _into(s, name, total):
    """A gradient's sum in its buffer: added to what is there, or in its place."""
    s[name].copy_(s[name].float() + total if s["case"]["accumulate"] else total)
    return s[name]


def _look(s):
    first, vocab = s["case"]["first"], s["case"]["vocab"]
    if own:
        s["gb"].gb_embedding_forward(s["out"], s["table"], s["ids"], scale=s["scale"], first=first)
        return {"out": s["out"]}
    row = s["ids"].long() - first
    here = (row >= 0) & (row < vocab)
    out = s["table"][torch.where(here, row, 0)].float() * s["scale"]
    return {"out": torch.where(here[:, None], out, 0.0).to(s["out"].dtype)}


def _look_grad(s):
    case = s["case"]
    if own:
        s["gb"].gb_embedding_backward(s["dtable"], s["dout"], s["ids"], scale=s["scale"], padding=case["padding"],
                                      accumulate=case["accumulate"], workspace=s["workspace"])
        return {"dtable": s["dtable"]}
    dout = s["dout"].float()
    if case["padding"] >= 0:
        dout = torch.where((s["ids"] != case["padding"])[:, None], dout, 0.0)
    total = torch.zeros(case["vocab"], case["dim"], device=dout.device).index_add_(0, s["ids"].long(), dout)
    return {"dtable": _into(s, "dtable", total * s["scale"])}


_PASS = {"norm": _norm, "norm_grad": _norm_grad, "look": _look, "look_grad": _look_grad}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "norm":
        x, w = s["x"].double(), s["w"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        y = (x - mean) / (var + EPS) ** 0.5 * w
        if case["bias"]:
            y += s["b"].double()
        if not case["stats"]:
            return {"y": y}
        return {"y": y, "mean": mean[:, 0], "rstd": (var[:, 0] + EPS) ** -0.5}
    if case["kind"] == "norm_grad":
        # dx as (I - 1 1' / n - h h' / n) applied to g, from the saved statistics
        rstd = s["rstd"].double().view(-1, 1)
        h = s["x"].double().sub_(s["mean"].double().view(-1, 1)).mul_(rstd)
        dy = s["dy"].double()
        old = 1.0 if case["accumulate"] else 0.0
        dw = torch.mul(dy, h).sum(dim=0).add_(s["dw"].double(), alpha=old)
        db = dy.sum(dim=0).add_(s["db"].double(), alpha=old) if case["bias"] else None
        dy *= s["w"].double()
        along = torch.mul(dy, h).mean(dim=1, keepdim=True)
        dy -= dy.mean(dim=1, keepdim=True)
        dy.addcmul_(h, along, value=-1.0).mul_(rstd)
        return {"dx": dy, "dw": dw} | ({"db": db} if case["bias"] else {})
    if case["kind"] == "look":
        ids = s["ids"].long()
        out = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device=ids.device)
        mine = torch.nonzero((ids >= case["first"]) & (ids < case["first"] + case["vocab"]))[:, 0]
        out[mine] = s["table"].double().index_select(0, ids[mine] - case["first"]) * s["scale"]
        return {"out": out}
    # tokens put in the order of their ids: a row's sum is a difference of running sums in 64 bits,
    # taken over a few columns at a time
    order = torch.argsort(s["ids"].long(), stable=True)
    ids = s["ids"].long()[order]
    ends = torch.searchsorted(ids, torch.arange(case["vocab"] + 1, device=ids.device))
    out = torch.empty(case["vocab"], case["dim"], dtype=torch.float64, device=ids.device)
    for c in range(0, case["dim"], 1024):
        run_sum = torch.zeros(case["tokens"] + 1, min(1024, case["dim"] - c), dtype=torch.float64, device=ids.device)
        torch.cumsum(s["dout"][:, c:c + 1024][order].double(), 0, out=run_sum[1:])
        out[:, c:c + 1024] = run_sum[ends[1:]] - run_sum[ends[:-1]]
    if case["padding"] >= 0:
        out[case["padding"]] = 0.0
    out *= s["scale"]
    return {"dtable": out.add_(s["dtable"]) if case["accumulate"] else out}


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(4)]:
        print(c, work(c))
