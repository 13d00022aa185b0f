"""Data-parallel training of a small token model on one GPU: the embedding's
and the layer norms' gradients are summed over tokens straight into each
rank's bucket, micro-batch by micro-batch, the buckets are reduced through the
bridge codec, and AdamW updates the parameters.

  python examples/ddp_tokens.py [--codec none|bf16|fp8] [--steps N]

The ranks are simulated: each takes its own sequences.  Autograd runs the
model; the two layers below are its functions over the library's calls, and
leave their parameters' gradients in the bucket instead of a .grad.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gradient_all_reduce_amd as gb  # noqa: E402

CODECS = {"none": gb.GB_CODEC_NONE, "bf16": gb.GB_CODEC_BF16, "fp8": gb.GB_CODEC_FP8_E4M3_B256}
RANKS, MICRO, BATCH, LENGTH = 2, 2, 8, 33
VOCAB, WIDTH = 1009, 96
PADDING = 0  # the id that fills short sequences: its row has no gradient


class Embedding(torch.autograd.Function):
    """Rows of the table times sqrt(width); the gradient goes to `bucket`.  The
    anchor's value is not used: that it wants a gradient makes autograd come
    back here."""

    @staticmethod
    def forward(ctx, anchor, table, ids, bucket, accumulate):
        out = torch.empty(*ids.shape, table.shape[1], dtype=table.dtype, device=table.device)
        gb.gb_embedding_forward(out, table, ids, scale=math.sqrt(table.shape[1]))
        ctx.save_for_backward(ids)
        ctx.bucket, ctx.accumulate = bucket, accumulate
        return out

    @staticmethod
    def backward(ctx, dout):
        ids, = ctx.saved_tensors
        vocab, dim = ctx.bucket.shape
        workspace = torch.empty(gb.gb_embedding_workspace_bytes(ids.numel(), vocab, dim), dtype=torch.uint8,
                                device=ids.device)
        gb.gb_embedding_backward(ctx.bucket, dout.contiguous(), ids, scale=math.sqrt(dim), padding=PADDING,
                                 accumulate=ctx.accumulate, workspace=workspace)
        return torch.zeros((), dtype=dout.dtype, device=dout.device), None, None, None, None


class LayerNorm(torch.autograd.Function):
    """Layer norm; the parameters' gradients go to `buckets`."""

    @staticmethod
    def forward(ctx, x, weight, bias, buckets, accumulate):
        y, rows = torch.empty_like(x), x.numel() // x.shape[-1]
        mean, rstd = (torch.empty(rows, device=x.device) for _ in range(2))
        gb.gb_layer_norm_forward(y, x, weight, bias, mean=mean, rstd=rstd)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.buckets, ctx.accumulate = buckets, accumulate
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        workspace = torch.empty(gb.gb_layer_norm_workspace_bytes(mean.numel(), x.shape[-1]), dtype=torch.uint8,
                                device=x.device)
        dx = torch.empty_like(x)
        gb.gb_layer_norm_backward(dx, *ctx.buckets, dy.contiguous(), x, mean, rstd, weight, accumulate=ctx.accumulate,
                                  workspace=workspace)
        return dx, None, None, None, None


SHAPES = {"table": (VOCAB, WIDTH), "gain1": (WIDTH,), "bias1": (WIDTH,), "mix": (WIDTH, WIDTH), "gain2": (WIDTH,),
          "bias2": (WIDTH,), "head": (VOCAB, WIDTH)}


def views(flat):
    """The parameters' views of a flat buffer; they start at any value."""
    out, at = {}, 0
    for name, shape in SHAPES.items():
        n = math.prod(shape)
        out[name] = flat[at:at + n].view(shape)
        at += n
    return out


def make_parameters(device, seed=0):
    flat = torch.zeros(sum(math.prod(s) for s in SHAPES.values()), device=device)
    g = torch.Generator(device=device).manual_seed(seed)
    for name, p in views(flat).items():
        if p.dim() == 2:
            p.copy_(torch.randn(p.shape, generator=g, device=device) / math.sqrt(WIDTH))
        elif name.startswith("gain"):
            p.fill_(1.0)
    return flat


def make_batch(generator, device):
    """Sequences that count upwards from their first token by their second,
    some of them ended early by padding; the next token is the target."""
    start, by = (torch.randint(1, VOCAB, (BATCH, 1), generator=generator, device=device) for _ in range(2))
    ids = 1 + (start + by * torch.arange(LENGTH + 1, device=device)) % (VOCAB - 1)
    length = torch.randint(LENGTH // 2, LENGTH + 2, (BATCH, 1), generator=generator, device=device)
    ids = torch.where(torch.arange(LENGTH + 1, device=device) < length, ids, PADDING)
    return ids[:, :-1].contiguous(), ids[:, 1:].contiguous()


def micro_batch(params, bucket, ids, targets, accumulate):
    """Forward and backward of one micro-batch; the loss.  Every gradient is in
    the bucket afterwards."""
    anchor = torch.zeros((), dtype=params["table"].dtype, device=ids.device, requires_grad=True)
    mix, head = (params[n].detach().requires_grad_() for n in ("mix", "head"))
    x = Embedding.apply(anchor, params["table"], ids, bucket["table"], accumulate)
    h = LayerNorm.apply(x, params["gain1"], params["bias1"], (bucket["gain1"], bucket["bias1"]), accumulate)
    x = x + torch.nn.functional.gelu(h @ mix.t())
    h = LayerNorm.apply(x, params["gain2"], params["bias2"], (bucket["gain2"], bucket["bias2"]), accumulate)
    scores = torch.log_softmax((h @ head.t()).float(), -1).gather(-1, targets[..., None])[..., 0]
    here = targets != PADDING
    loss = -(scores * here).sum() / here.sum()
    dmix, dhead, _ = torch.autograd.grad(loss, (mix, head, anchor))
    for name, d in (("mix", dmix), ("head", dhead)):
        bucket[name].add_(d) if accumulate else bucket[name].copy_(d)
    return loss.detach()


def train(codec="fp8", steps=100, lr=2e-3, device="cuda", report=None):
    """Train; the parameters and the loss of every step."""
    device = torch.device(device, 0) if device == "cuda" else torch.device(device)
    flat = make_parameters(device)
    params, n, codec = views(flat), flat.numel(), CODECS[codec]
    ranks = [torch.zeros(n, device=device) for _ in range(RANKS)]
    buckets = [views(r) for r in ranks]
    reduced = torch.zeros(n, device=device)
    bridge = torch.empty(max(1, gb.gb_bucket_batch_workspace_bytes(codec, RANKS, [n])), dtype=torch.uint8,
                         device=device)
    moments = {name: [torch.zeros_like(p).view(-1) for _ in range(2)] for name, p in params.items()}
    tensors = [gb.GbOptimTensor(p.view(-1), g.view(-1), *moments[name], weight_decay=0.01 if p.dim() == 2 else 0.0)
               for (name, p), g in zip(params.items(), views(reduced).values())]
    numels = [p.numel() for p in params.values()]
    plan = gb.gb_optim_plan(tensors, torch.empty(gb.gb_optim_plan_bytes(numels), dtype=torch.uint8, device=device))
    control = torch.zeros(gb.GB_OPTIM_CONTROL_BYTES, dtype=torch.uint8, device=device)
    fields = gb.gb_optim_control(control)
    fields["lr"].fill_(lr)
    data, losses = torch.Generator(device=device).manual_seed(1), []
    for step in range(steps):
        total = 0.0
        for bucket in buckets:
            for m in range(MICRO):
                total += float(micro_batch(params, bucket, *make_batch(data, device), accumulate=m > 0))
        gb.gb_bucket_allreduce_local_batch([reduced], [ranks], codec, workspace=bridge, divisor=RANKS)
        gb.gb_optim_begin_clip(plan, control, max_norm=1.0, inv_scale=1.0 / MICRO)
        gb.gb_adamw_step(plan, control)
        losses.append(total / (RANKS * MICRO))
        if report is not None and (step % 20 == 0 or step == steps - 1):
            report(f"step {int(fields['step'])}: loss {losses[-1]:.4f}, gradient norm {float(fields['norm']):.4f}")
    return flat, losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--codec", choices=tuple(CODECS), default="fp8")
    ap.add_argument("--steps", type=int, default=100)
    a = ap.parse_args()
    train(a.codec, a.steps, report=print)
