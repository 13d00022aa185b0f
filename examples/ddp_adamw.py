"""A data-parallel training step on one GPU: k ranks' gradients are reduced
through the bridge codec, their norm is clipped, and AdamW updates a bfloat16
model from float32 master parameters, with the moments in 32 or in 8 bits.

  python examples/ddp_adamw.py [--state f32|e4m3] [--codec none|bf16|fp8] [--steps N]

The ranks are simulated: each takes its own batch of a synthetic regression
and leaves its gradients in its own bucket.  What follows the backward passes
(all-reduce, norm, AdamW) is captured in a HIP graph once and replayed: the
step count, the learning rate and the norm live in the control block on the
device, so nothing in it waits for the host.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gradient_all_reduce_amd as gb  # noqa: E402

CODECS = {"none": gb.GB_CODEC_NONE, "bf16": gb.GB_CODEC_BF16, "fp8": gb.GB_CODEC_FP8_E4M3_B256}
RANKS, BATCH, WIDTH, HIDDEN = 4, 256, 96, 257  # odd on purpose: ragged buckets


def make_model(device, seed=0):
    """Master parameters (float32) and the bfloat16 copies the model runs on."""
    g = torch.Generator(device=device).manual_seed(seed)
    shapes = [(HIDDEN, WIDTH), (HIDDEN,), (HIDDEN, HIDDEN), (HIDDEN,), (1, HIDDEN), (1,)]
    masters = [torch.randn(s, generator=g, device=device) / math.sqrt(s[-1]) if len(s) == 2
               else torch.zeros(s, device=device) for s in shapes]
    return masters, [m.bfloat16().requires_grad_() for m in masters]


def forward(params, x):
    for w, b in zip(params[0:4:2], params[1:4:2]):
        x = torch.nn.functional.silu(torch.addmm(b, x, w.t()))
    return torch.addmm(params[5], x, params[4].t()).squeeze(1)



def train(state="e4m3", codec="fp8", steps=200, lr=3e-3, max_norm=1.0, device="cuda", report=None):
    """Train and return the loss of every step."""
    device = torch.device(device, 0) if device == "cuda" else torch.device(device)
    masters, params = make_model(device)
    numels = [m.numel() for m in masters]

    # each rank's gradients, and the reduced ones that the optimizer reads
    ranks = [[torch.zeros(n, device=device) for _ in range(RANKS)] for n in numels]
    reduced = [torch.zeros(n, device=device) for n in numels]
    codec = CODECS[codec]
    bridge = torch.empty(max(1, gb.gb_bucket_batch_workspace_bytes(codec, RANKS, numels)), dtype=torch.uint8,
                         device=device)

    # moments, all zero before the first step; no decay on the biases
    def moments(n):
        if state == "f32":
            return [torch.zeros(n, device=device) for _ in range(2)] + [None, None]
        blocks = -(-n // gb.GB_BLOCK)
        return ([torch.zeros(n, dtype=torch.uint8, device=device) for _ in range(2)]
                + [torch.zeros(blocks, device=device) for _ in range(2)])

    # the step writes the bfloat16 model beside the masters it updates
    tensors = [gb.GbOptimTensor(m.view(-1), g, *moments(m.numel()), copy=p.detach().view(-1),
                                weight_decay=0.01 if m.dim() == 2 else 0.0)
               for m, g, p in zip(masters, reduced, params)]
    workspace = torch.empty(gb.gb_optim_plan_bytes(numels), dtype=torch.uint8, device=device)
    plan = gb.gb_optim_plan(tensors, workspace, beta1=0.9, beta2=0.99, seed=1)
    control = torch.zeros(gb.GB_OPTIM_CONTROL_BYTES, dtype=torch.uint8, device=device)
    fields = gb.gb_optim_control(control)

    def reduce_and_step():
        gb.gb_bucket_allreduce_local_batch(reduced, ranks, codec, workspace=bridge, divisor=RANKS)
        gb.gb_optim_begin_clip(plan, control, max_norm)
        gb.gb_adamw_step(plan, control)

    data = torch.Generator(device=device).manual_seed(1)
    teacher = torch.randn(WIDTH, generator=data, device=device) / math.sqrt(WIDTH)
    graph, losses = None, []
    for step in range(steps):
        fields["lr"].fill_(lr * (1 - step / steps))  # a schedule, in stream order
        total = 0.0
        for r in range(RANKS):
            x = torch.randn(BATCH, WIDTH, generator=data, device=device)
            y = torch.sin(x @ teacher)
            loss = (forward(params, x.bfloat16()).float() - y).square().mean()
            for bucket, grad in zip(ranks, torch.autograd.grad(loss, params)):
                bucket[r].copy_(grad.reshape(-1))
            total += loss.item() / RANKS
        if step == 0:
            reduce_and_step()  # the first one eager
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    reduce_and_step()
            graph.replay()
        losses.append(total)
        if report is not None and (step % 20 == 0 or step == steps - 1):
            report(f"step {int(fields['step'])}: loss {total:.4f}, gradient norm {float(fields['norm']):.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--state", choices=("f32", "e4m3"), default="e4m3")
    ap.add_argument("--codec", choices=tuple(CODECS), default="fp8")
    ap.add_argument("--steps", type=int, default=200)
    a = ap.parse_args()
    train(a.state, a.codec, a.steps, report=print)
