"""Benchmark of libgbreduce on one GPU: effective HBM GB/s of the leader-side
arithmetic of reduce-bridge-broadcast (fixed-order fp32 sum, bf16 / fp8
bridge codecs).

    python bench.py [--steps K] [--warmup W] [--workload NAME] [--no-cpu-baseline]

Prints ONE JSON line.  A step is one pass of the workload's path over its
synthetic inputs, which are resident in device memory before timing starts.
`value` is algorithmic bytes per step / measured time per step (GB/s, 1e9).
Algorithmic bytes are the least reads and writes the step needs: every input
value read once, every payload byte and every output value written once
(and, where a call reads a payload back, read once).

Workloads (inputs from workloads.py):
  ddp_1b_buckets   (default) k=4 ranks x 1.0e9 fp32 gradients in 153 buckets
                   of 25 MiB; per bucket: fp8 E4M3 encode of every rank with
                   one absmax/448 scale per 256 values, decode and add in rank
                   order, fp32 sum written out.  One gb_bucket_allreduce_local
                   call over the whole stream per step (one launch; buckets
                   start on block boundaries).  The same pass made as one call
                   per bucket, as a DDP hook would issue it, is reported too,
                   and the buckets as separate buffers through
                   gb_bucket_allreduce_local_batch (16 per launch).
                   --dtype f16|bf16|f64 runs the same stream over gradients
                   of that type (gb_bucket_allreduce_local_typed): values
                   taken to float32, encoded, the float32 total rounded once
                   to the type.
  gradients_256mib k=4 x 2^26 fp32; 4 x gb_encode_fp8_e4m3_blockscaled +
                   gb_decode_accumulate(fp8).
  gradients_64mib  k=4 x 2^24 fp32; 4 x gb_encode_bf16 + gb_decode_accumulate(bf16).
  two_island_sweep k=2, 19 sizes 2^8..2^26 fp32; gb_reduce_sum into a
                   separate output at every size.  --op avg|max|min uses
                   gb_reduce; --dtype f16|bf16|f64|i8|u8|i32|i64 runs the
                   sweep in that element type through gb_reduce_typed.
  two_rank_4mib    k=2 x 2^20 fp32; gb_reduce_sum, gb_encode_bf16 of the sum,
                   gb_decode_accumulate(bf16, k=1).  The same outputs from
                   gb_reduce_encode (sum and codes in one pass) + the decode
                   are reported too.
  staged_fp8_256mib the leader's staged (pipelined) bridge step on one GPU:
                   its 2^26-value fp32 island sum encoded to fp8 and copied to
                   pinned host memory in 4 MiB chunks (gb_encode_staged), then
                   the 4 leaders' payloads copied back from pinned host memory
                   in chunks and decoded-and-accumulated
                   (gb_decode_accumulate_staged).  Bound by the host link;
                   the same work done serially is reported too.
  ddp_1b_buckets_ef the ddp_1b_buckets stream with error feedback: each rank
                   keeps an fp32 residual, encodes gradient + residual and
                   writes the new residual (gb_bucket_allreduce_local_ef).

The roofline object reports the step's dominant kernel: its algorithmic bytes
per launch over its average launch time, timed with HIP events on the stream
the library launches on, against MI355X's 8 TB/s HBM peak.  The CPU baseline
is the oracle (oracle/, single-threaded C) on a bounded sample of the same
workload, on this host; the sample's GPU outputs are also checked against it.
"""
import argparse
import json
import os
import sys
import time

HBM_PEAK_GBS = 8000.0
METRIC = "effective HBM GB/s (and % of peak) for k-way reduce + bf16/fp8 encode/decode"


def parse():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--gpus", type=int, default=1)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--warmup", type=int, default=3)
    p.add_argument("--workload", default="ddp_1b_buckets",
                   choices=["ddp_1b_buckets", "gradients_256mib", "gradients_64mib",
                            "two_island_sweep", "two_rank_4mib", "ddp_1b_buckets_ef",
                            "staged_fp8_256mib"])
    p.add_argument("--scale-mode", type=int, default=0, choices=[0, 1],
                   help="fp8 scale: 0 absmax/448, 1 power of two")
    p.add_argument("--op", default="sum", choices=["sum", "avg", "max", "min"],
                   help="reduction of the two_island_sweep workload (avg divides by the "
                        "world size, 2 here)")
    p.add_argument("--codec", default="fp8", choices=["fp8", "bf16", "none"],
                   help="bridge codec of the ddp_1b_buckets stream")
    p.add_argument("--dtype", default="f32", choices=["f32", "f16", "bf16", "f64", "i8", "u8", "i32", "i64"],
                   help="element type of the two_island_sweep workload")
    p.add_argument("--shard", type=int, default=1,
                   help="run one GPU's share of the workload when it is split over G GPUs: every "
                        "bucket (or buffer) cut into G contiguous ranges aligned to 256 values, "
                        "GPU 0's range kept (ddp_1b_buckets, ddp_1b_buckets_ef, gradients_256mib, "
                        "gradients_64mib)")
    p.add_argument("--no-cpu-baseline", action="store_true")
    p.add_argument("--no-memory-ceiling", action="store_true",
                   help="skip the memory-ceiling program (gradient_all_reduce_amd/gb_ceiling)")
    p.add_argument("--no-other-workloads", action="store_true",
                   help="with the default workload, skip the summary of the four other workloads "
                        "(two_rank_4mib, two_island_sweep, gradients_64mib, gradients_256mib)")
    p.add_argument("--cpu-seconds", type=float, default=12.0,
                   help="rough budget of oracle CPU time for the baseline sample")
    p.add_argument("--calibrate-copy", action="store_true",
                   help="only run plain 1 GiB device copies (gb_reduce_sum with k=1, and torch "
                        "copy_), the known-size kernels that scale rocprofv3 FETCH_SIZE / "
                        "WRITE_SIZE readings")
    return p.parse_args()


def log(*a):
    print(*a, file=sys.stderr, flush=True)


class Workload:
    """Inputs resident on the device, a step, and the step's byte count."""
    name = ""
    config = {}

    def __init__(self, gb, torch, args):
        self.gb, self.torch, self.args = gb, torch, args
        self.dev = "cuda:0"
        self.stream = torch.cuda.current_stream()

    def timed_kernel(self):
        """(name, bytes per launch, callable doing `launches` launches)."""
        raise NotImplementedError


def nblocks(n):
    return (n + 255) // 256


def shard_len(length, g):
    """Values of GPU 0's range when `length` values are cut into g contiguous
    ranges aligned to 256 values (so no fp8 block straddles two GPUs)."""
    return min(length, -(-length // (256 * g)) * 256)


SHARDED = ("ddp_1b_buckets", "ddp_1b_buckets_ef", "gradients_256mib", "gradients_64mib")


def shard_note(g):
    return f"GPU 0 of {g}: each buffer cut into {g} contiguous ranges aligned to 256 values"


class Unit:
    """One independent piece of the CPU baseline: `compute` runs the oracle on
    inputs already copied to the host (the timed part), `check` compares its
    result with the GPU's output (untimed); `nbytes` counts the piece's
    algorithmic bytes by the workload's own formula."""

    def __init__(self, nbytes, compute, check):
        self.nbytes, self.compute, self.check = nbytes, compute, check
        self.result = None


def host_values(torch, t):
    """A device tensor's values on the host; 16-bit floats as raw codes."""
    import numpy as np
    if t.element_size() == 2 and t.is_floating_point():
        return t.view(torch.int16).cpu().numpy().view(np.uint16)
    return t.cpu().numpy()


def same_bits(got, want):
    """Bit-identical arrays, NaN included (every NaN the arithmetic delivers
    is the canonical one on both sides)."""
    return got.tobytes() == want.tobytes()


class DdpBuckets(Workload):
    name = "ddp_1b_buckets"

    def __init__(self, gb, torch, args):
        super().__init__(gb, torch, args)
        import workloads as W
        self.W = W
        self.k, self.n, self.bucket = 4, W.DDP_N, W.DDP_BUCKET
        if args.shard > 1:
            # each bucket is reduced across the GPUs on its own, so each is cut
            pieces = [shard_len(l, args.shard) for _, l in W.ddp_buckets()]
            self.bucket = shard_len(W.DDP_BUCKET, args.shard)
            assert all(p == self.bucket for p in pieces[:-1])
            self.n = sum(pieces)
        self.mode = args.scale_mode
        self.dt = args.dtype
        if self.dt not in ("f32", "f16", "bf16", "f64"):
            raise SystemExit("the bucket stream compresses floating-point gradients only")
        self.esize = {"f32": 4, "f16": 2, "bf16": 2, "f64": 8}[self.dt]
        self.codec = {"fp8": gb.GB_CODEC_FP8_E4M3_B256, "bf16": gb.GB_CODEC_BF16, "none": gb.GB_CODEC_NONE}[
            getattr(args, "codec", "fp8")]
        self.config = {"workload": self.name, "k": self.k, "n_per_rank": self.n,
                       "bucket_elems": self.bucket, "buckets": len(self.buckets()),
                       "codec": {2: "fp8_e4m3_b256", 1: "bf16", 0: "none"}[self.codec],
                       "scale_mode": ["absmax_div_448", "pow2"][self.mode],
                       "distribution": "N(0, sigma=1e-3)", "element_type": self.dt}
        if args.shard > 1:
            self.config["shard"] = shard_note(args.shard)

    def buckets(self):
        return self.W.ddp_buckets(self.n, self.bucket)

    def setup(self):
        torch, gb = self.torch, self.gb
        self.x = [self.W.device_gradients_typed(self.n, self.W.BASE_SEED + r, self.dev, self.dt)
                  for r in range(self.k)]
        self.out = torch.empty(self.n, dtype=self.x[0].dtype, device=self.dev)
        self.lay = gb.gb_bucket_workspace_layout(self.codec, self.k, self.n, self.bucket)
        self.ws = torch.empty(max(1, self.lay["total"]), dtype=torch.uint8, device=self.dev)

    def call(self, out, xs, ws):
        if self.dt == "f32":
            self.gb.gb_bucket_allreduce_local(out, xs, self.bucket, self.codec, self.mode, ws)
        else:
            self.gb.gb_bucket_allreduce_local_typed(out, xs, self.bucket, self.codec, self.mode, ws)

    def step(self):
        self.call(self.out, self.x, self.ws)

    def payload_bytes(self, n):
        return {2: n + 4 * nblocks(n), 1: 2 * n, 0: 0}[self.codec]

    def bytes_for(self, n):
        # every rank's gradients read, every payload written, the sum written
        return self.k * self.esize * n + self.k * self.payload_bytes(n) + self.esize * n

    def step_bytes(self):
        return sum(self.bytes_for(l) for _, l in self.buckets())

    def timed_kernel(self):
        et = self.gb.GB_DTYPE_OF[self.dt]
        # the four-rank float32 sum takes its wide kernel from 2^28 values per rank
        f32_sum = "reduce_sum4_wide_kernel" if self.n >= (1 << 28) else "reduce_sum_kernel<4,false>"
        # the fp8 pass over 4 ranks takes one block per 64-lane workgroup for
        # float32 gradients from 2^22 values per rank, and 128-lane workgroups
        # for float64 ones between 3 * 2^21 and 2^29
        n = self.n
        if et == 0 and n >= (1 << 22):
            fp8 = "fused_fp8_wave_kernel<4>"
        elif et == 3 and (3 << 21) <= n < (1 << 29):
            fp8 = "fused_fp8_half_kernel<4,3>"
        else:
            fp8 = f"fused_fp8_kernel<4,{et}>"
        # and the bf16 pass its 64-lane workgroups: float32 gradients over 3 or
        # more ranks, float16 and bfloat16 ones over 4 from 2^29 values
        wave = et == 0 or (et in (1, 2) and self.n >= (1 << 29))
        bf16 = f"fused_bf16_wave_kernel<4,{et}>" if wave else f"fused_bf16_kernel<4,{et}>"
        # (over four ranks the half-precision types take 8 values per lane
        # from 2^22 values)
        if et in (1, 2) and self.n >= (1 << 22):
            bf16 = f"fused_bf16_eight_kernel<{et}>"
        name = {2: fp8, 1: bf16,
                0: f32_sum if et == 0 else f"reduce_typed_kernel<{et},4,0>"}[self.codec]
        return (name, self.step_bytes(), 1, self.step)

    def per_bucket_step(self):
        for out, xs, ws in self.pb_args:
            self.call(out, xs, ws)

    def per_bucket_step_streams(self, m):
        """The per-bucket calls dealt round-robin over the current stream and
        m - 1 more (all at the default priority), forked from and joined back
        into the current stream, so m buckets are in flight at once."""
        torch = self.torch
        main = torch.cuda.current_stream()
        streams = [main] + self.side[:m - 1]
        for st in streams[1:]:
            st.wait_stream(main)
        for i, (out, xs, ws) in enumerate(self.pb_args):
            with torch.cuda.stream(streams[i % m]):
                self.call(out, xs, ws)
        for st in streams[1:]:
            main.wait_stream(st)

    def extra(self, time_region, reps):
        """Throughput of the same pass issued as one call per bucket, as a DDP
        hook would issue it, each bucket's payloads in its own slice of the
        workspace.  The 153 calls are captured once in a HIP graph and the
        graph is replayed, so the figure is the GPU's, not the Python
        binding's per-call cost; every replay's output is checked against the
        single-launch result.  The same calls are also timed dealt over two and
        over four streams inside one graph.  Leaves the workspace in the per-bucket
        layout."""
        torch, gb = self.torch, self.gb
        want = self.out.clone()
        ibits = {2: torch.int16, 4: torch.int32, 8: torch.int64}[self.esize]
        matches = lambda: bool(torch.equal(self.out.view(ibits), want.view(ibits)))
        self.pb_args = []
        off = 0
        for start, length in self.buckets():
            need = gb.gb_bucket_workspace_bytes(self.codec, self.k, length, self.bucket)
            self.pb_args.append((self.out[start:start + length],
                                 [t[start:start + length] for t in self.x],
                                 self.ws[off:off + need]))
            off += need
        self.per_bucket_step()  # eager, also warms up
        torch.cuda.synchronize()
        eager_ok = matches()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.per_bucket_step()
        self.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        replay_ok = matches()
        ms = time_region(graph.replay, reps) / reps
        replay_ok &= matches()
        eager_ms = time_region(self.per_bucket_step, reps) / reps
        del graph
        # the same calls over 2 and 4 streams: the buckets' workspace slices
        # and output slices are disjoint, so several calls may run at once
        self.side = [torch.cuda.Stream() for _ in range(3)]
        by_streams = {}
        for m in (2, 4):
            self.per_bucket_step_streams(m)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                self.per_bucket_step_streams(m)
            self.out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            replay_ok &= matches()
            ms_m = time_region(graph.replay, reps) / reps
            replay_ok &= matches()
            del graph
            by_streams[m] = ms_m
        # the same buckets through gb_bucket_allreduce_local_batch: up to 16
        # buckets, each its own buffer for the library, per launch
        outs = [a[0] for a in self.pb_args]
        srcs = [a[1] for a in self.pb_args]
        sizes = [o.numel() for o in outs]
        need = gb.gb_bucket_batch_workspace_bytes(self.codec, self.k, sizes)
        wsb = self.ws if need <= self.ws.numel() else torch.empty(need, dtype=torch.uint8, device=self.dev)
        batch = lambda: gb.gb_bucket_allreduce_local_batch(outs, srcs, self.codec, self.mode, wsb if need else None)
        batch()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            batch()
        self.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        batch_ok = matches()
        ms_batch = time_region(graph.replay, reps) / reps
        batch_ok &= matches()
        del graph
        gbs = lambda t: round(self.step_bytes() / (t * 1e-3) / 1e9, 2)
        return {"per_bucket_batched_graph_gbs": gbs(ms_batch),
                "per_bucket_batched_graph_ms": round(ms_batch, 4),
                "per_bucket_batched_outputs_match": batch_ok,
                "per_bucket_calls_graph_gbs": gbs(ms),
                "per_bucket_calls_graph_ms": round(ms, 4),
                "per_bucket_calls_two_streams_graph_gbs": gbs(by_streams[2]),
                "per_bucket_calls_four_streams_graph_gbs": gbs(by_streams[4]),
                "per_bucket_calls_four_streams_graph_ms": round(by_streams[4], 4),
                "per_bucket_calls_eager_ms": round(eager_ms, 4),
                "per_bucket_outputs_match": eager_ok and replay_ok}

    CPU_CHUNK = 1_638_400  # a quarter of a bucket (6,400 blocks)

    def cpu_units(self):
        """Quarter-bucket pieces of the stream, in order; each is the oracle's
        bucket stream over that piece (pieces start on block boundaries, so
        their blocks are the whole stream's)."""
        from oracle import oracle as O
        torch = self.torch

        def make(start, length):
            def factory():
                xs = [host_values(torch, t[start:start + length]) for t in self.x]
                if self.dt == "f32":
                    compute = lambda: O.bucket_allreduce(xs, self.bucket, self.codec, self.mode)
                else:
                    compute = lambda: O.bucket_allreduce_typed(xs, self.dt, self.bucket, self.codec, self.mode)

                def check(res):
                    want, codes, scales = res
                    ok = same_bits(host_values(torch, self.out[start:start + length]), want)
                    cb = {2: 1, 1: 2, 0: 0}[self.codec]  # code bytes per value
                    for r in range(self.k if cb else 0):
                        c0 = r * self.lay["codes_stride"] + cb * start
                        ok &= same_bits(self.ws[c0:c0 + cb * length].cpu().numpy(), codes[r].view("uint8"))
                        if self.codec == 2:
                            s0 = self.lay["scales_offset"] + r * self.lay["scales_stride"] + 4 * (start // 256)
                            ok &= same_bits(self.ws[s0:s0 + 4 * nblocks(length)].cpu().numpy(),
                                            scales[r].view("uint8"))
                    return ok
                return Unit(self.bytes_for(length), compute, check)
            return factory

        factories = [make(s + o, min(self.CPU_CHUNK, l - o))
                     for s, l in self.buckets() for o in range(0, l, self.CPU_CHUNK)]
        return factories, lambda m: (f"first {m} quarter-buckets ({m * self.CPU_CHUNK:,} values x {self.k} ranks) "
                                     f"of {len(factories)}")


class DdpBucketsEF(DdpBuckets):
    name = "ddp_1b_buckets_ef"

    def __init__(self, gb, torch, args):
        super().__init__(gb, torch, args)
        if self.codec == gb.GB_CODEC_NONE:
            raise SystemExit("error feedback runs with the bf16 or fp8 codec")
        self.config = dict(self.config, workload=self.name, error_feedback="fp32 residual per rank")

    def setup(self):
        super().setup()
        self.res = [self.torch.zeros(self.n, dtype=self.torch.float32, device=self.dev) for _ in range(self.k)]

    def step(self):
        if self.dt == "f32":
            self.gb.gb_bucket_allreduce_local_ef(self.out, self.x, self.res, self.bucket, self.codec, self.mode,
                                                 self.ws)
        else:
            self.gb.gb_bucket_allreduce_local_ef_typed(self.out, self.x, self.res, self.bucket, self.codec, self.mode,
                                                       self.ws)

    def bytes_for(self, n):
        # sources and (fp32) residuals read; payload, residuals and sum written
        return self.k * (self.esize + 4) * n + self.k * self.payload_bytes(n) + self.k * 4 * n + self.esize * n

    def timed_kernel(self):
        et = self.gb.GB_DTYPE_OF[self.dt]
        fp8 = self.codec == self.gb.GB_CODEC_FP8_E4M3_B256
        # the bf16 pass over four ranks takes 64-lane workgroups at every size,
        # for every gradient type
        bf16 = f"fused_bf16_ef_wave_kernel<4,{et}>"
        # the fp8 pass over four ranks of float32, float16 and bfloat16
        # gradients takes one block per 64-lane workgroup from 2^22 values
        wave = et in (0, 1, 2) and self.n >= (1 << 22)
        name = (f"fused_fp8_ef_wave_kernel<{et}>" if wave else f"fused_fp8_ef_kernel<4,{et}>") if fp8 else bf16
        return (name, self.step_bytes(), 1, self.step)

    def extra(self, time_region, reps):
        """The same step as one gb_bucket_allreduce_local_ef (or _ef_typed)
        call per bucket and through gb_bucket_allreduce_local_batch_ef (8
        buckets per launch), each captured in a HIP graph; the two give the
        same bits from the same residuals."""
        torch, gb = self.torch, self.gb
        buckets = list(self.buckets())
        outs = [self.out[s:s + n] for s, n in buckets]
        srcs = [[t[s:s + n] for t in self.x] for s, n in buckets]
        ress = [[t[s:s + n] for t in self.res] for s, n in buckets]
        wsl, off = [], 0
        for _, n in buckets:
            need = gb.gb_bucket_workspace_bytes(self.codec, self.k, n, self.bucket)
            wsl.append(self.ws[off:off + need])
            off += need

        call = gb.gb_bucket_allreduce_local_ef if self.dt == "f32" else gb.gb_bucket_allreduce_local_ef_typed

        def per_bucket():
            for o, xs, rs, w in zip(outs, srcs, ress, wsl):
                call(o, xs, rs, self.bucket, self.codec, self.mode, w)

        need = gb.gb_bucket_batch_workspace_bytes(self.codec, self.k, [n for _, n in buckets])
        wsb = self.ws if need <= self.ws.numel() else torch.empty(need, dtype=torch.uint8, device=self.dev)
        batch = lambda: gb.gb_bucket_allreduce_local_batch_ef(outs, srcs, ress, self.codec, self.mode, wsb)
        saved = [t.clone() for t in self.res]
        per_bucket()
        torch.cuda.synchronize()
        want, want_res = self.out.clone(), [t.clone() for t in self.res]
        for t, s0 in zip(self.res, saved):
            t.copy_(s0)
        batch()
        torch.cuda.synchronize()
        ibits = {2: torch.int16, 4: torch.int32, 8: torch.int64}[self.esize]
        ok = bool(torch.equal(self.out.view(ibits), want.view(ibits)))
        ok &= all(bool(torch.equal(a.view(torch.int32), b.view(torch.int32))) for a, b in zip(self.res, want_res))
        del saved, want, want_res
        ms = {}
        for name, fn in (("calls", per_bucket), ("batched", batch)):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                fn()
            ms[name] = time_region(graph.replay, reps) / reps
            del graph
        gbs = lambda t: round(self.step_bytes() / (t * 1e-3) / 1e9, 2)
        return {"per_bucket_calls_graph_gbs": gbs(ms["calls"]),
                "per_bucket_calls_graph_ms": round(ms["calls"], 4),
                "per_bucket_batched_graph_gbs": gbs(ms["batched"]),
                "per_bucket_batched_graph_ms": round(ms["batched"], 4),
                "per_bucket_batched_matches_calls": ok}

    def cpu_units(self):
        """One more step of the stream, checked against the oracle from the
        residuals it starts from, on the first quarter-buckets (their
        residuals are captured before that step)."""
        from oracle import oracle as O
        torch = self.torch
        pieces = []
        for s, l in self.buckets():
            for o in range(0, l, self.CPU_CHUNK):
                pieces.append((s + o, min(self.CPU_CHUNK, l - o)))
        pieces = pieces[:24]  # about 0.55 s of oracle work each
        before = [[r[s:s + l].cpu().numpy() for r in self.res] for s, l in pieces]
        self.step()
        torch.cuda.synchronize()

        def make(i):
            start, length = pieces[i]

            def factory():
                xs = [host_values(torch, t[start:start + length]) for t in self.x]
                compute = lambda: O.bucket_allreduce_ef_typed(xs, before[i], self.dt, self.bucket, self.codec,
                                                              self.mode)

                def check(res):
                    want, codes, scales, res1 = res
                    ok = same_bits(host_values(torch, self.out[start:start + length]), want)
                    cb = 1 if self.codec == self.gb.GB_CODEC_FP8_E4M3_B256 else 2  # code bytes per value
                    for r in range(self.k):
                        ok &= same_bits(self.res[r][start:start + length].cpu().numpy(), res1[r])
                        c0 = r * self.lay["codes_stride"] + cb * start
                        ok &= same_bits(self.ws[c0:c0 + cb * length].cpu().numpy(), codes[r].view("uint8"))
                    return ok
                return Unit(self.bytes_for(length), compute, check)
            return factory
        return [make(i) for i in range(len(pieces))], lambda m: f"one step of the first {m} quarter-buckets"


class Staged(Workload):
    name = "staged_fp8_256mib"
    CHUNK = (4 << 20) // 4  # 4 MiB of fp32 per chunk

    def __init__(self, gb, torch, args):
        super().__init__(gb, torch, args)
        import workloads as W
        self.W = W
        self.k, self.n = 4, W.GRAD256_N
        self.mode = args.scale_mode
        self.config = {"workload": self.name, "k": self.k, "n_per_rank": self.n, "chunk_elems": self.CHUNK,
                       "codec": "fp8_e4m3_b256", "scale_mode": ["absmax_div_448", "pow2"][self.mode],
                       "distribution": "N(0, sigma=1e-3), 1% outliers x100",
                       "path": "encode_staged (device -> pinned host) + decode_accumulate_staged "
                               "(pinned host -> device, k=4)"}

    def setup(self):
        torch, gb, n, k = self.torch, self.gb, self.n, self.k
        nb = nblocks(n)
        self.xh = self.W.gradient_ranks(k, n)
        self.x = [torch.from_numpy(a).to(self.dev) for a in self.xh]
        self.cd = torch.empty(n, dtype=torch.uint8, device=self.dev)
        self.sd = torch.empty(nb, dtype=torch.float32, device=self.dev)
        self.ch = torch.empty(n, dtype=torch.uint8, pin_memory=True)
        self.sh = torch.empty(nb, dtype=torch.float32, pin_memory=True)
        # the payloads of the k leaders as the bridge delivers them: pinned host memory
        self.rh, self.rsh = [], []
        for r in range(k):
            gb.gb_encode_fp8_e4m3_blockscaled(self.cd, self.sd, self.x[r], self.mode)
            self.rh.append(self.cd.cpu().pin_memory())
            self.rsh.append(self.sd.cpu().pin_memory())
        self.rd = [torch.empty(n, dtype=torch.uint8, device=self.dev) for _ in range(k)]
        self.rsd = [torch.empty(nb, dtype=torch.float32, device=self.dev) for _ in range(k)]
        self.acc = torch.empty(n, dtype=torch.float32, device=self.dev)

    def step(self):
        gb = self.gb
        gb.gb_encode_staged(gb.GB_CODEC_FP8_E4M3_B256, self.cd, self.sd, self.ch, self.sh, self.x[0], self.CHUNK,
                            self.mode)
        gb.gb_decode_accumulate_staged(self.acc, self.rh, self.rsh, self.rd, self.rsd,
                                       gb.GB_CODEC_FP8_E4M3_B256, self.CHUNK)

    def serial_step(self):
        gb = self.gb
        gb.gb_encode_fp8_e4m3_blockscaled(self.cd, self.sd, self.x[0], self.mode)
        self.ch.copy_(self.cd, non_blocking=True)
        self.sh.copy_(self.sd, non_blocking=True)
        for r in range(self.k):
            self.rd[r].copy_(self.rh[r], non_blocking=True)
            self.rsd[r].copy_(self.rsh[r], non_blocking=True)
        gb.gb_decode_accumulate(self.acc, self.rd, self.rsd, gb.GB_CODEC_FP8_E4M3_B256)

    def payload(self):
        return self.n + 4 * nblocks(self.n)

    def step_bytes(self):
        # HBM: encode (4n read, payload written), the D2H copy (payload read),
        # the H2D copies (k payloads written), decode (k payloads read, 4n written)
        return 4 * self.n + 2 * self.payload() + 2 * self.k * self.payload() + 4 * self.n

    def timed_kernel(self):
        n = self.n
        per = self.k * self.payload() + 4 * n
        return (decode_fp8_name(n), per, 1,
                lambda: self.gb.gb_decode_accumulate(self.acc, self.rd, self.rsd, self.gb.GB_CODEC_FP8_E4M3_B256))

    def extra(self, time_region, reps):
        self.serial_step()
        serial_ms = time_region(self.serial_step, reps) / reps
        staged_ms = time_region(self.step, reps) / reps
        sweep = {}
        default_chunk = self.CHUNK
        for chunk in (1 << 18, 1 << 20, 1 << 22, 1 << 24):
            self.CHUNK = chunk
            sweep[str(chunk)] = round(time_region(self.step, reps) / reps, 4)
        self.CHUNK = default_chunk
        link = (1 + self.k) * self.payload()
        d2h = self.torch.empty(self.payload(), dtype=self.torch.uint8, pin_memory=True)
        src = self.torch.empty(self.payload(), dtype=self.torch.uint8, device=self.dev)
        copy_ms = time_region(lambda: d2h.copy_(src, non_blocking=True), reps) / reps
        return {"link_payload_bytes_per_step": link,
                "link_gbs_staged": round(link / (staged_ms * 1e-3) / 1e9, 2),
                "staged_ms": round(staged_ms, 4), "serial_ms": round(serial_ms, 4),
                "overlap_speedup": round(serial_ms / staged_ms, 4),
                "staged_ms_by_chunk_elems": sweep,
                "d2h_copy_gbs_one_payload": round(self.payload() / (copy_ms * 1e-3) / 1e9, 2)}

    def cpu_units(self):
        """The staged step's arithmetic (rank 0's fp8 encode; decode-and-add of
        the four payloads) on 2^18-value pieces of the first 2^22 values."""
        from oracle import oracle as O
        self.step()
        self.torch.cuda.synchronize()
        piece = 1 << 18

        def make(start):
            def factory():
                xs = [a[start:start + piece] for a in self.xh]

                def compute():
                    enc = [O.encode_fp8(a, self.mode) for a in xs]
                    return enc, O.decode_accumulate([c for c, _ in enc], [s for _, s in enc], O.CODEC_FP8)

                def check(res):
                    enc, want = res
                    ok = same_bits(self.ch[start:start + piece].numpy(), enc[0][0])
                    ok &= same_bits(self.sh[start // 256:(start + piece) // 256].numpy(), enc[0][1])
                    return ok and same_bits(self.acc[start:start + piece].cpu().numpy(), want)
                p = piece + 4 * nblocks(piece)
                return Unit(4 * piece + 2 * p + 2 * self.k * p + 4 * piece, compute, check)
            return factory
        return [make(o) for o in range(0, 1 << 22, piece)], lambda m: f"first {m * piece:,} values of each rank"


def decode_fp8_name(n):
    """The kernel that decodes 4 fp8 payloads of n values into a float32
    total: one block per 64-lane workgroup from 2^24 values."""
    return "decode_fp8_wave_kernel<false>" if n >= (1 << 24) else "decode_fp8_kernel<4,false,0>"


def codec_extra(wl, time_region, reps, dec_name, dec_bytes):
    """Extras of the two gradient workloads (4 encodes, then the decode): the
    decode kernel timed alone, and the same arithmetic as one fused launch,
    gb_bucket_allreduce_local over the whole buffer (each rank's values read
    once, its payload written, decoded and added in rank order), whose
    output, codes and scales are checked bit for bit against the separate
    calls'."""
    torch, gb = wl.torch, wl.gb
    fp8 = hasattr(wl, "scales")
    codec = gb.GB_CODEC_FP8_E4M3_B256 if fp8 else gb.GB_CODEC_BF16
    wl.step()
    torch.cuda.synchronize()
    dec_ms = time_region(wl.decode, reps) / reps
    lay = gb.gb_bucket_workspace_layout(codec, wl.k, wl.n, wl.n)
    ws = torch.empty(lay["total"], dtype=torch.uint8, device=wl.dev)
    out = torch.empty_like(wl.out)
    fused = lambda: gb.gb_bucket_allreduce_local(out, wl.x, wl.n, codec, getattr(wl, "mode", 0), ws)
    fused()
    torch.cuda.synchronize()
    same = bool(torch.equal(out.view(torch.int32), wl.out.view(torch.int32)))
    cb = 1 if fp8 else 2
    for r in range(wl.k):
        c0 = r * lay["codes_stride"]
        same &= bool(torch.equal(ws[c0:c0 + cb * wl.n], wl.codes[r].view(torch.uint8)))
        if fp8:
            s0 = lay["scales_offset"] + r * lay["scales_stride"]
            same &= bool(torch.equal(ws[s0:s0 + 4 * nblocks(wl.n)], wl.scales[r].view(torch.uint8)))
    fused_ms = time_region(fused, reps) / reps
    del ws, out
    gbs = lambda b, t: round(b / (t * 1e-3) / 1e9, 1)
    return {"decode_kernel": dec_name, "decode_kernel_gbs": gbs(dec_bytes, dec_ms),
            "decode_kernel_frac": round(gbs(dec_bytes, dec_ms) / HBM_PEAK_GBS, 4),
            "fused_pass_kernel": "fused_fp8_wave_kernel<4>" if fp8 else "fused_bf16_wave_kernel<4,0>",
            "fused_pass_bytes": wl.fused_bytes(), "fused_pass_us": round(fused_ms * 1e3, 2),
            "fused_pass_gbs": gbs(wl.fused_bytes(), fused_ms),
            "fused_pass_frac": round(gbs(wl.fused_bytes(), fused_ms) / HBM_PEAK_GBS, 4),
            "fused_pass_same_bits_as_the_calls": same}


class Gradients256(Workload):
    name = "gradients_256mib"

    def __init__(self, gb, torch, args):
        super().__init__(gb, torch, args)
        import workloads as W
        self.W = W
        self.k, self.n = 4, shard_len(W.GRAD256_N, args.shard)
        self.mode = args.scale_mode
        self.config = {"workload": self.name, "k": self.k, "n_per_rank": self.n,
                       "codec": "fp8_e4m3_b256", "scale_mode": ["absmax_div_448", "pow2"][self.mode],
                       "distribution": "N(0, sigma=1e-3), 1% outliers x100",
                       "path": "4 x encode_fp8 + decode_accumulate"}
        if args.shard > 1:
            self.config["shard"] = shard_note(args.shard)

    def setup(self):
        torch = self.torch
        self.xh = self.W.gradient_ranks(self.k, self.n)
        self.x = [torch.from_numpy(a).to(self.dev) for a in self.xh]
        self.codes = [torch.empty(self.n, dtype=torch.uint8, device=self.dev) for _ in range(self.k)]
        self.scales = [torch.empty(nblocks(self.n), dtype=torch.float32, device=self.dev) for _ in range(self.k)]
        self.out = torch.empty(self.n, dtype=torch.float32, device=self.dev)

    def encode(self, r):
        self.gb.gb_encode_fp8_e4m3_blockscaled(self.codes[r], self.scales[r], self.x[r], self.mode)

    def step(self):
        for r in range(self.k):
            self.encode(r)
        self.gb.gb_decode_accumulate(self.out, self.codes, self.scales, self.gb.GB_CODEC_FP8_E4M3_B256)

    def step_bytes(self):
        p = self.n + 4 * nblocks(self.n)
        return self.k * (4 * self.n + p) + self.k * p + 4 * self.n

    def timed_kernel(self):
        per = 4 * self.n + self.n + 4 * nblocks(self.n)
        return ("encode_fp8_kernel<0>", per, self.k, lambda: [self.encode(r) for r in range(self.k)])

    def decode(self):
        self.gb.gb_decode_accumulate(self.out, self.codes, self.scales, self.gb.GB_CODEC_FP8_E4M3_B256)

    def fused_bytes(self):
        return self.k * (4 * self.n + self.n + 4 * nblocks(self.n)) + 4 * self.n

    def extra(self, time_region, reps):
        return codec_extra(self, time_region, reps, decode_fp8_name(self.n),
                           self.k * (self.n + 4 * nblocks(self.n)) + 4 * self.n)

    def cpu_units(self):
        """4 fp8 encodes and the decode-and-add on 2^18-value pieces of every
        rank, in order."""
        from oracle import oracle as O
        piece = 1 << 18

        def make(start):
            def factory():
                xs = [a[start:start + piece] for a in self.xh]

                def compute():
                    enc = [O.encode_fp8(a, self.mode) for a in xs]
                    return enc, O.decode_accumulate([c for c, _ in enc], [s for _, s in enc], O.CODEC_FP8)

                def check(res):
                    enc, want = res
                    ok = same_bits(self.out[start:start + piece].cpu().numpy(), want)
                    for r in range(self.k):
                        ok &= same_bits(self.codes[r][start:start + piece].cpu().numpy(), enc[r][0])
                        ok &= same_bits(self.scales[r][start // 256:(start + piece) // 256].cpu().numpy(), enc[r][1])
                    return ok
                p = piece + 4 * nblocks(piece)
                return Unit(self.k * (4 * piece + p) + self.k * p + 4 * piece, compute, check)
            return factory
        return ([make(o) for o in range(0, self.n, piece)],
                lambda m: f"first {m * piece:,} values of each of the {self.k} ranks")


class Gradients64(Workload):
    name = "gradients_64mib"

    def __init__(self, gb, torch, args):
        super().__init__(gb, torch, args)
        import workloads as W
        self.W = W
        self.k, self.n = 4, shard_len(W.GRAD64_N, args.shard)
        self.config = {"workload": self.name, "k": self.k, "n_per_rank": self.n, "codec": "bf16",
                       "distribution": "N(0, sigma=1e-3), 1% outliers x100",
                       "path": "4 x encode_bf16 + decode_accumulate"}
        if args.shard > 1:
            self.config["shard"] = shard_note(args.shard)

    def setup(self):
        torch = self.torch
        self.xh = self.W.gradient_ranks(self.k, self.n)
        self.x = [torch.from_numpy(a).to(self.dev) for a in self.xh]
        self.codes = [torch.empty(self.n, dtype=torch.uint16, device=self.dev) for _ in range(self.k)]
        self.out = torch.empty(self.n, dtype=torch.float32, device=self.dev)

    def encode(self, r):
        self.gb.gb_encode_bf16(self.codes[r], self.x[r])

    def step(self):
        for r in range(self.k):
            self.encode(r)
        self.gb.gb_decode_accumulate(self.out, self.codes, None, self.gb.GB_CODEC_BF16)

    def step_bytes(self):
        return self.k * 6 * self.n + self.k * 2 * self.n + 4 * self.n

    def timed_kernel(self):
        return ("encode_bf16_kernel<0,2>", 6 * self.n, self.k, lambda: [self.encode(r) for r in range(self.k)])

    def decode(self):
        self.gb.gb_decode_accumulate(self.out, self.codes, None, self.gb.GB_CODEC_BF16)

    def fused_bytes(self):
        return self.k * (4 * self.n + 2 * self.n) + 4 * self.n

    def extra(self, time_region, reps):
        return codec_extra(self, time_region, reps, "decode_bf16_kernel<4,false,0>", self.k * 2 * self.n + 4 * self.n)

    def cpu_units(self):
        """4 bf16 encodes and the decode-and-add on 2^18-value pieces."""
        from oracle import oracle as O
        torch = self.torch
        piece = 1 << 18

        def make(start):
            def factory():
                xs = [a[start:start + piece] for a in self.xh]

                def compute():
                    codes = [O.encode_bf16(a) for a in xs]
                    return codes, O.decode_accumulate(codes, None, O.CODEC_BF16)

                def check(res):
                    codes, want = res
                    ok = same_bits(self.out[start:start + piece].cpu().numpy(), want)
                    for r in range(self.k):
                        ok &= same_bits(host_values(torch, self.codes[r][start:start + piece].view(torch.int16))
                                        .view("uint16"), codes[r])
                    return ok
                return Unit(self.k * 8 * piece + 4 * piece, compute, check)
            return factory
        return ([make(o) for o in range(0, self.n, piece)],
                lambda m: f"first {m * piece:,} values of each of the {self.k} ranks")


class Sweep(Workload):
    name = "two_island_sweep"
    OPS = {"sum": 0, "avg": 1, "max": 2, "min": 3}
    ESIZE = {"f32": 4, "f16": 2, "bf16": 2, "f64": 8, "i8": 1, "u8": 1, "i32": 4, "i64": 8}

    def __init__(self, gb, torch, args):
        super().__init__(gb, torch, args)
        import workloads as W
        self.W = W
        self.sizes = W.SWEEP_SIZES
        self.op = self.OPS[args.op]
        self.dt = args.dtype
        self.esize = self.ESIZE[self.dt]
        if self.dt in ("i8", "u8", "i32", "i64") and self.op == 1:
            raise SystemExit("AVG is defined for floating-point element types only")
        dist = "N(0,1)" if self.dt in ("f32", "f16", "bf16", "f64") else "uniform over the type"
        self.config = {"workload": self.name, "k": 2, "sizes": f"2^8..2^26 values ({len(self.sizes)} sizes)",
                       "distribution": dist, "op": args.op, "element_type": self.dt,
                       "path": f"{args.op} of the two island results into a separate output"}

    def setup(self):
        torch = self.torch
        if self.dt == "f32":
            self.xh = {n: self.W.normal_ranks(2, n) for n in self.sizes}
            self.x = {n: [torch.from_numpy(a).to(self.dev) for a in xs] for n, xs in self.xh.items()}
            self.out = {n: torch.empty(n, dtype=torch.float32, device=self.dev) for n in self.sizes}
            return
        tdt = {"f16": torch.float16, "bf16": torch.bfloat16, "f64": torch.float64, "i8": torch.int8,
               "u8": torch.uint8, "i32": torch.int32, "i64": torch.int64}[self.dt]
        self.xh = {n: self.W.typed_ranks(2, n, self.dt) for n in self.sizes}

        def dev(a):
            if a.dtype == __import__("numpy").uint16:  # 16-bit float codes
                return torch.from_numpy(a.view("int16")).to(self.dev).view(tdt)
            return torch.from_numpy(a).to(self.dev)
        self.x = {n: [dev(a) for a in xs] for n, xs in self.xh.items()}
        self.out = {n: torch.empty(n, dtype=tdt, device=self.dev) for n in self.sizes}

    def reduce(self, n):
        if self.dt != "f32":
            self.gb.gb_reduce_typed(self.out[n], self.x[n], self.op, 2)
        elif self.op == 0:
            self.gb.gb_reduce_sum(self.out[n], self.x[n])
        else:
            self.gb.gb_reduce(self.out[n], self.x[n], self.op, 2)

    def step(self):
        for n in self.sizes:
            self.reduce(n)

    def step_bytes(self):
        return sum(3 * self.esize * n for n in self.sizes)

    def timed_kernel(self):
        n = self.sizes[-1]
        if self.dt != "f32":
            name = f"reduce_typed_kernel<{self.gb.GB_DTYPE_OF[self.dt]},2,{self.op}>"
        elif self.op == 0:
            name = "reduce_sum_kernel<2,false>"
        else:
            name = f"reduce_op_kernel<2,{self.op}>"
        return (name, 3 * self.esize * n, 1, lambda: self.reduce(n))

    def extra(self, time_region, reps):
        """Every size of the sweep timed alone: the median of `reps` calls, a
        1 GiB buffer rewritten (untimed) before each so that no call finds its
        inputs in the 256 MB last-level cache; microseconds and GB/s.  Small
        sizes are latency, the large ones bandwidth."""
        torch = self.torch
        scratch = torch.empty((1 << 30) // 4, dtype=torch.float32, device=self.dev)
        us, gbs = {}, {}
        for n in self.sizes:
            t = []
            for i in range(max(5, reps)):
                scratch.fill_(float(i))
                t.append(time_region(lambda: self.reduce(n), 1))
            t.sort()
            med = t[len(t) // 2]
            us[str(n)] = round(med * 1e3, 2)
            gbs[str(n)] = round(3 * self.esize * n / (med * 1e-3) / 1e9, 1)
        del scratch
        res = {"per_size_us_cache_flushed": us, "per_size_gbs_cache_flushed": gbs}
        if self.dt == "f32" and self.op == 0:
            res.update(self.copy_contrast(time_region, reps))
        return res

    def copy_contrast(self, time_region, reps):
        """The leader's total written once, straight into the output (the sum
        kernel's 12 bytes per value), against the unfused form: the sum made
        in place into the first island buffer, then a device-to-device copy
        (torch copy_, hipMemcpyAsync) into the output, 20 bytes per value.
        Back to back at the three largest sizes; both give the same bits."""
        torch, gb = self.torch, self.gb
        res = {}
        for n in self.sizes[-3:]:
            x0 = self.x[n][0].clone()
            fused = lambda: gb.gb_reduce_sum(self.out[n], self.x[n])
            tmp = torch.empty_like(x0)
            reset = lambda: tmp.copy_(x0)  # restores the first operand, untimed

            def pair():
                gb.gb_reduce_sum(tmp, [tmp, self.x[n][1]])
                self.out[n].copy_(tmp)
            fused()
            want = self.out[n].clone()
            reset()
            pair()
            torch.cuda.synchronize()
            same = bool(torch.equal(self.out[n].view(torch.int32), want.view(torch.int32)))
            f_ms = time_region(fused, reps) / reps
            tot = 0.0
            for _ in range(reps):
                reset()
                tot += time_region(pair, 1)
            u_ms = tot / reps
            res[str(n)] = {"fused_12n_us": round(f_ms * 1e3, 2), "inplace_plus_d2d_20n_us": round(u_ms * 1e3, 2),
                           "fused_gbs": round(12 * n / (f_ms * 1e-3) / 1e9, 1),
                           "inplace_plus_d2d_gbs_of_20n": round(20 * n / (u_ms * 1e-3) / 1e9, 1),
                           "speedup": round(u_ms / f_ms, 3), "same_bits": same}
            del x0, tmp, want
        return {"sum_written_once_vs_inplace_plus_copy": res}

    def cpu_units(self):
        """Every size of the sweep, the larger ones in 2^20-value pieces."""
        from oracle import oracle as O
        torch = self.torch
        piece = 1 << 20

        def make(n, start, length):
            def factory():
                xs = [a[start:start + length] for a in self.xh[n]]
                if self.dt == "f32":
                    compute = lambda: O.reduce(xs, self.op, 2)
                else:
                    compute = lambda: O.reduce_typed(xs, self.dt, self.op, 2)
                check = lambda want: same_bits(host_values(torch, self.out[n][start:start + length]), want)
                return Unit(3 * self.esize * length, compute, check)
            return factory
        factories = [make(n, o, min(piece, n - o)) for n in self.sizes for o in range(0, n, piece)]
        return factories, lambda m: "the whole sweep" if m == len(factories) else f"{m} of {len(factories)} pieces"


class TwoRank(Workload):
    name = "two_rank_4mib"

    def __init__(self, gb, torch, args):
        super().__init__(gb, torch, args)
        import workloads as W
        self.W = W
        self.n = W.TWO_RANK_N
        self.config = {"workload": self.name, "k": 2, "n_per_rank": self.n, "distribution": "N(0,1)",
                       "path": "reduce_sum, encode_bf16 of the sum, decode (k=1)",
                       "note": "24 MiB per step stays in the 256 MB last-level cache"}

    def setup(self):
        torch = self.torch
        self.xh = self.W.normal_ranks(2, self.n)
        self.x = [torch.from_numpy(a).to(self.dev) for a in self.xh]
        self.sum = torch.empty(self.n, dtype=torch.float32, device=self.dev)
        self.codes = torch.empty(self.n, dtype=torch.uint16, device=self.dev)
        self.dec = torch.empty(self.n, dtype=torch.float32, device=self.dev)

    def step(self):
        gb = self.gb
        gb.gb_reduce_sum(self.sum, self.x)
        gb.gb_encode_bf16(self.codes, self.sum)
        gb.gb_decode_accumulate(self.dec, [self.codes], None, gb.GB_CODEC_BF16)

    def step_bytes(self):
        return 12 * self.n + 6 * self.n + 6 * self.n

    def timed_kernel(self):
        return ("reduce_sum_kernel<2,false>", 12 * self.n, 1, lambda: self.gb.gb_reduce_sum(self.sum, self.x))

    def fused_step(self):
        gb = self.gb
        gb.gb_reduce_encode(gb.GB_CODEC_BF16, self.codes2, None, self.x, self.sum2)
        gb.gb_decode_accumulate(self.dec2, [self.codes2], None, gb.GB_CODEC_BF16)

    def extra(self, time_region, reps):
        """The same outputs (sum, bf16 codes of the sum, its decode) from two
        launches: gb_reduce_encode writes the sum and its codes in one pass
        (reads 8n, writes 4n + 2n), then the decode.  Checked bit for bit
        against the three-call path.  Both paths are also timed as replayed
        HIP graphs."""
        torch = self.torch
        self.sum2 = torch.empty_like(self.sum)
        self.codes2 = torch.empty_like(self.codes)
        self.dec2 = torch.empty_like(self.dec)
        reps = max(reps, 50)
        self.fused_step()
        torch.cuda.synchronize()
        same = (torch.equal(self.sum2.view(torch.int32), self.sum.view(torch.int32))
                and torch.equal(self.codes2.view(torch.int16), self.codes.view(torch.int16))
                and torch.equal(self.dec2.view(torch.int32), self.dec.view(torch.int32)))
        ms = time_region(self.fused_step, reps) / reps
        base = time_region(self.step, reps) / reps
        # Both paths captured once in a HIP graph and replayed: the launches'
        # host cost leaves the step, the device work stays.  Every replay's
        # outputs are checked against the eager three-call path's.
        graph_ms, graph_ok = {}, True
        for name, fn, outs in (("three_call", self.step, (self.sum, self.codes, self.dec)),
                               ("fused", self.fused_step, (self.sum2, self.codes2, self.dec2))):
            fn()
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                fn()
            for o in outs:
                o.view(torch.uint8).fill_(0xFF)
            g.replay()
            torch.cuda.synchronize()
            graph_ms[name] = time_region(g.replay, reps) / reps
            graph_ok &= (torch.equal(outs[0].view(torch.int32), self.sum2.view(torch.int32) if name == "three_call"
                                     else self.sum.view(torch.int32))
                         and torch.equal(outs[1].view(torch.int16), self.codes2.view(torch.int16)
                                         if name == "three_call" else self.codes.view(torch.int16))
                         and torch.equal(outs[2].view(torch.int32), self.dec2.view(torch.int32)
                                         if name == "three_call" else self.dec.view(torch.int32)))
            del g
        return {"fused_sum_encode_step_ms": round(ms, 4), "three_call_step_ms": round(base, 4),
                "fused_sum_encode_gbs": round(20 * self.n / (ms * 1e-3) / 1e9, 2),
                "three_call_graph_step_ms": round(graph_ms["three_call"], 4),
                "three_call_graph_gbs": round(24 * self.n / (graph_ms["three_call"] * 1e-3) / 1e9, 2),
                "fused_graph_step_ms": round(graph_ms["fused"], 4),
                "fused_graph_gbs": round(20 * self.n / (graph_ms["fused"] * 1e-3) / 1e9, 2),
                "fused_outputs_match": bool(same), "graph_outputs_match": bool(graph_ok)}

    def cpu_units(self):
        """Sum, bf16 encode of the sum and its decode, on 2^18-value pieces."""
        from oracle import oracle as O
        piece = 1 << 18

        def make(start):
            def factory():
                xs = [a[start:start + piece] for a in self.xh]

                def compute():
                    s = O.reduce_sum(xs)
                    return O.decode_accumulate([O.encode_bf16(s)], None, O.CODEC_BF16)
                check = lambda want: same_bits(self.dec[start:start + piece].cpu().numpy(), want)
                return Unit(24 * piece, compute, check)
            return factory
        return [make(o) for o in range(0, self.n, piece)], lambda m: f"first {m * piece:,} values of both ranks"


WORKLOADS = {c.name: c for c in (DdpBuckets, Gradients256, Gradients64, Sweep, TwoRank, DdpBucketsEF, Staged)}

ROOT = os.path.dirname(os.path.abspath(__file__))


def kernel_sources_sha256():
    """sha256 over the library's kernel sources (gb_device.h and every .hip
    file of the library that defines a kernel, by name in sorted order: each
    name, a NUL, its bytes, a NUL).  Host-only sources (the C ABI layer, the
    no-allocation entry point), the ceiling program, the optimizer step and
    the token-sum layers, whose kernels no workload here runs, are left out: a
    change there leaves the workloads' kernels and their counters as they were."""
    import glob
    import hashlib
    csrc = os.path.join(ROOT, "gradient_all_reduce_amd", "csrc")
    h = hashlib.sha256()
    srcs = [p for p in glob.glob(os.path.join(csrc, "*.hip"))
            if os.path.basename(p) not in ("gb_ceiling.hip", "gb_optim.hip", "gb_norm.hip", "gb_embed.hip")
            and "__global__" in open(p).read()]
    for path in sorted(srcs + [os.path.join(csrc, "gb_device.h")]):
        h.update(os.path.basename(path).encode() + b"\0" + open(path, "rb").read() + b"\0")
    return h.hexdigest()


def profiled_traffic(kernel, workload):
    """HBM bytes per launch of `kernel` on `workload` from the rocprofv3 counter
    summaries under profiles/, or None when none was taken on the kernel
    source as it is now (the summary records the source's sha256)."""
    import glob
    sha = kernel_sources_sha256()
    for path in sorted(glob.glob(os.path.join(ROOT, "profiles", "*.md"))):
        for line in open(path):
            if not line.startswith("traffic "):
                continue
            kv = dict(tok.split("=", 1) for tok in line.split()[1:])
            if (kv.get("kernel") == kernel and kv.get("workload") == workload
                    and kv.get("kernels_sha256") == sha):
                return int(float(kv["traffic_bytes"]))
    return None


def time_region(torch, stream, fn, reps):
    """Milliseconds for `reps` calls of fn, HIP events on `stream`."""
    start = torch.cuda.Event(enable_timing=True)
    end = torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    start.record(stream)
    for _ in range(reps):
        fn()
    end.record(stream)
    end.synchronize()
    return start.elapsed_time(end)


def cpu_model():
    try:
        for line in open("/proc/cpuinfo"):
            if line.startswith("model name"):
                return line.split(":", 1)[1].strip()
    except OSError:
        pass
    return "unknown"


def cpu_baseline(wl, budget):
    """The oracle on a bounded sample of the workload: units are taken in order
    (their inputs copied to the host untimed) until about `budget` seconds of
    single-threaded oracle work, then the same units are run again across the
    host's cores (the oracle is C; ctypes releases the GIL), and every unit's
    result is compared with the GPU's output."""
    import concurrent.futures as cf
    wl.torch.cuda.synchronize()
    factories, describe = wl.cpu_units()
    units, t_one = [], 0.0
    for factory in factories:
        u = factory()
        t0 = time.perf_counter()
        u.result = u.compute()
        t_one += time.perf_counter() - t0
        units.append(u)
        if t_one >= budget:
            break
    ok = all(bool(u.check(u.result)) for u in units)
    affinity = len(os.sched_getaffinity(0))
    # every core this process may run on, up to the 16 a one-GPU share of the
    # benchmark host holds
    cores = max(1, min(affinity, 16))
    with cf.ThreadPoolExecutor(cores) as ex:
        t0 = time.perf_counter()
        list(ex.map(lambda u: u.compute(), units))
        t_all = time.perf_counter() - t0
    nbytes = sum(u.nbytes for u in units)
    return {"value": round(nbytes / t_all / 1e9, 4), "unit": "GB/s", "cores": cores, "affinity_cores": affinity,
            "kind": "oracle",
            "sample": describe(len(units)), "seconds": round(t_all, 3),
            "single_core": {"value": round(nbytes / t_one / 1e9, 4), "seconds": round(t_one, 3)},
            "cpu_model": cpu_model(), "gpu_matches_oracle_on_sample": ok}


OTHER_WORKLOADS = ("two_rank_4mib", "two_island_sweep", "gradients_64mib", "gradients_256mib")


def graph_kernel_ms(torch, stream, fn, launches, calls=16, reps=5):
    """Milliseconds per launch of the dominant kernel with the host out of
    the way: `calls` calls of fn captured in one HIP graph, the graph
    replayed `reps` times back to back.  Each launch still pays the GPU's
    own boundary between kernels on one stream (about 1.6 us)."""
    fn()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(calls):
            fn()
    g.replay()
    torch.cuda.synchronize()
    ms = time_region(torch, stream, g.replay, reps) / (reps * calls * launches)
    del g
    return ms


def workload_summary(gb, torch, args, name, reps):
    """One of the smaller workloads, timed as its own --workload run times it
    but with fewer repetitions: the step's GB/s, its dominant kernel's GB/s
    and fraction of the HBM peak, the p10/p50/p90 of single steps with the
    last-level cache flushed, the workload's extras, and the oracle on the
    first pieces of its CPU sample (compared with the GPU's outputs).  The
    dominant kernel is timed twice: called from Python back to back (a short
    kernel is then bound by the host's launch rate) and replayed from a HIP
    graph."""
    a = argparse.Namespace(**vars(args))
    a.workload, a.shard, a.dtype, a.op, a.codec, a.scale_mode = name, 1, "f32", "sum", "fp8", 0
    wl = WORKLOADS[name](gb, torch, a)
    wl.setup()
    torch.cuda.synchronize()
    for _ in range(2):
        wl.step()
    ms = time_region(torch, wl.stream, wl.step, reps) / reps
    kname, kbytes, klaunches, kfn = wl.timed_kernel()
    kms = time_region(torch, wl.stream, kfn, reps) / (reps * klaunches)
    gms = graph_kernel_ms(torch, wl.stream, kfn, klaunches)
    dist = step_distribution(torch, wl.stream, wl.step, reps)
    extra = wl.extra(lambda fn, r: time_region(torch, wl.stream, fn, r), reps) if hasattr(wl, "extra") else {}
    torch.cuda.synchronize()
    factories, describe = wl.cpu_units()
    units = [f() for f in factories[:2]]
    ok = all(bool(u.check(u.compute())) for u in units)
    sb = wl.step_bytes()
    res = {"workload": wl.config, "step_ms": round(ms, 4), "step_gbs": round(sb / (ms * 1e-3) / 1e9, 1),
           "dominant_kernel": kname, "kernel_us_per_launch": round(kms * 1e3, 3),
           "kernel_gbs": round(kbytes / (kms * 1e-3) / 1e9, 1),
           "kernel_frac": round(kbytes / (kms * 1e-3) / 1e9 / HBM_PEAK_GBS, 4),
           "kernel_us_per_launch_graph": round(gms * 1e3, 3),
           "kernel_graph_gbs": round(kbytes / (gms * 1e-3) / 1e9, 1),
           "kernel_graph_frac": round(kbytes / (gms * 1e-3) / 1e9 / HBM_PEAK_GBS, 4),
           "step_p50_ms_cache_flushed": dist["p50_ms"],
           "step_gbs_cache_flushed_p50": round(sb / (dist["p50_ms"] * 1e-3) / 1e9, 1),
           "step_distribution": dist, "oracle_sample": describe(len(units)),
           "gpu_matches_oracle_on_sample": ok}
    res.update(extra)
    del wl, units
    torch.cuda.empty_cache()
    return res


def copy_ceiling(torch, gb, stream, reps=5):
    """GB/s of plain 1 GiB device copies of gradient-like values (HBM moves
    constant or zero data faster): the library's own streaming copy
    (gb_reduce_sum with one source) and the runtime's device-to-device copy
    (torch copy_, a hipMemcpyDtoD), each reading and writing 1 GiB."""
    import workloads as W
    n = (1 << 30) // 4
    src = W.device_gradients(n, W.BASE_SEED + 99, "cuda:0")
    dst = torch.empty_like(src)
    gb.gb_reduce_sum(dst, [src])
    dst.copy_(src)
    lib_ms = time_region(torch, stream, lambda: gb.gb_reduce_sum(dst, [src]), reps) / reps
    rt_ms = time_region(torch, stream, lambda: dst.copy_(src), reps) / reps
    del src, dst
    return {"library_copy_gbs": round(2 * 4 * n / (lib_ms * 1e-3) / 1e9, 1),
            "hipMemcpyDtoD_gbs": round(2 * 4 * n / (rt_ms * 1e-3) / 1e9, 1), "bytes_each_way": 4 * n}


def memory_ceiling(gib=4, reps=10):
    """The memory-ceiling program (gradient_all_reduce_amd/gb_ceiling, built
    with the library) run as a child process: median GB/s of plain copies
    (1, 2 and 4 vectors per lane; index order or 8 fronts; through LDS with
    global_load_lds_dwordx4), read-only and write-only streams, and a
    memory-only replicas of the fused fp8 pass with and without error
    feedback, on `gib`-GiB buffers of gradient-like values; and the
    median microseconds per launch of an empty kernel (1, 1,600 and 25,600
    workgroups) launched back to back from a stream and from a graph."""
    import subprocess
    prog = os.path.join(ROOT, "gradient_all_reduce_amd", "gb_ceiling")
    if not os.path.exists(prog):
        return {"error": "gb_ceiling is not built"}
    try:
        r = subprocess.run([prog, str(gib), str(reps)], capture_output=True, text=True, timeout=180)
    except subprocess.TimeoutExpired:
        return {"error": "gb_ceiling timed out"}
    if r.returncode != 0:
        return {"error": f"gb_ceiling exited with {r.returncode}: {r.stderr.strip()[-300:]}"}
    last = json.loads(r.stdout.strip().splitlines()[-1])
    res = last["median_gbs"]
    copies = {k: v for k, v in res.items() if k.startswith("copy")}
    best = max(copies, key=copies.get)
    return {"command": f"gradient_all_reduce_amd/gb_ceiling {gib} {reps}", "median_gbs": res,
            "best_copy": best, "best_copy_gbs": copies[best], "empty_launch_us": last["launch_us"]}


def replica_frac(achieved, mem_ceiling, wl):
    """For the float32 fp8 bucket stream, plain or with error feedback, over
    the whole 1e9-value buffer: the fused pass against the memory-only
    replica of its own access pattern, in the same run."""
    med = mem_ceiling.get("median_gbs", {})
    if getattr(wl, "dt", None) != "f32" or getattr(wl, "codec", None) != 2 or "shard" in wl.config:
        return {}
    rep = med.get("fused_fp8_ef_replica_4GiB") if type(wl) is DdpBucketsEF else (
        med.get("fused_fp8_replica_4GiB") if type(wl) is DdpBuckets else None)
    return {"frac_of_own_memory_pattern": round(achieved / rep, 4)} if rep else {}


def step_distribution(torch, stream, fn, reps):
    """Per-step milliseconds, each step timed alone with HIP events, a 1 GiB
    buffer rewritten (untimed) before each so no step starts from a warm
    last-level cache; p10 / p50 / p90."""
    scratch = torch.empty((1 << 30) // 4, dtype=torch.float32, device="cuda:0")
    times = []
    for i in range(reps):
        scratch.fill_(float(i))
        times.append(time_region(torch, stream, fn, 1))
    del scratch
    times.sort()
    q = lambda f: times[min(len(times) - 1, int(f * (len(times) - 1) + 0.5))]
    return {"reps": reps, "p10_ms": round(q(0.1), 4), "p50_ms": round(q(0.5), 4), "p90_ms": round(q(0.9), 4),
            "cache_flushed": True}


def main():
    args = parse()
    world = int(os.environ.get("WORLD_SIZE", "1"))
    if args.gpus != 1 or world != 1:
        print(f"bench.py measures one GPU: the leader arithmetic runs on a single device "
              f"(asked for --gpus {args.gpus}, WORLD_SIZE {world}); run it with --gpus 1",
              file=sys.stderr, flush=True)
        sys.exit(2)

    if args.shard < 1 or (args.shard > 1 and args.workload not in SHARDED):
        print(f"--shard G (G >= 1) applies to {', '.join(SHARDED)}; the sweep already spans the "
              f"smaller sizes", file=sys.stderr, flush=True)
        sys.exit(2)

    import torch
    import gradient_all_reduce_amd as gb

    if not torch.cuda.is_available():
        print("bench.py needs a GPU", file=sys.stderr)
        sys.exit(1)
    if args.calibrate_copy:
        # gb_reduce_sum with one source is a plain copy through the library's
        # own streaming kernel: it reads and writes exactly 1 GiB per launch.
        n = (1 << 30) // 4
        src = torch.ones(n, dtype=torch.float32, device="cuda:0")
        dst = torch.empty_like(src)
        for _ in range(3):
            gb.gb_reduce_sum(dst, [src])
        for _ in range(3):
            dst.copy_(src)
        torch.cuda.synchronize()
        log(f"[bench] copied {4 * n} bytes 3 times with gb_reduce_sum(k=1) and 3 times with torch copy_")
        return
    wl = WORKLOADS[args.workload](gb, torch, args)
    log(f"[bench] workload {wl.name}: allocating and drawing inputs")
    wl.setup()
    torch.cuda.synchronize()
    log(f"[bench] warmup {args.warmup} steps")
    for _ in range(args.warmup):
        wl.step()
    torch.cuda.synchronize()
    log(f"[bench] timing {args.steps} steps")
    ms = time_region(torch, wl.stream, wl.step, args.steps)
    ms_per_step = ms / args.steps
    step_bytes = wl.step_bytes()
    value = step_bytes / (ms_per_step * 1e-3) / 1e9

    kname, kbytes, klaunches, kfn = wl.timed_kernel()
    reps = max(3, args.steps)
    kms = time_region(torch, wl.stream, kfn, reps) / (reps * klaunches)
    achieved = kbytes / (kms * 1e-3) / 1e9
    log(f"[bench] step {ms_per_step:.3f} ms, {value:.1f} GB/s; {kname}: {kms * 1e3:.2f} us/launch, "
        f"{achieved:.1f} GB/s")

    dist = step_distribution(torch, wl.stream, wl.step, max(5, min(args.steps, 50)))
    log(f"[bench] per step (cache flushed): p10 {dist['p10_ms']} p50 {dist['p50_ms']} p90 {dist['p90_ms']} ms")

    cpu = None
    if not args.no_cpu_baseline:
        log("[bench] cpu baseline: oracle on a sample")
        cpu = cpu_baseline(wl, args.cpu_seconds)
        log(f"[bench] oracle {cpu['value']} GB/s on {cpu['cores']} cores ({cpu['single_core']['value']} on one) "
            f"over {cpu['sample']}; GPU output matches: {cpu['gpu_matches_oracle_on_sample']}")

    ceiling = copy_ceiling(torch, gb, wl.stream)
    log(f"[bench] copy ceiling: {ceiling}")
    mem_ceiling = {} if args.no_memory_ceiling else memory_ceiling()
    log(f"[bench] memory ceiling: {mem_ceiling}")

    extra = {}
    if hasattr(wl, "extra"):
        extra = wl.extra(lambda fn, reps: time_region(torch, wl.stream, fn, reps), max(3, args.steps // 2))
        log(f"[bench] extra: {extra}")
    if isinstance(wl, DdpBuckets) and not isinstance(wl, DdpBucketsEF):
        extra["headline"] = (f"value = one gb_bucket_allreduce_local call over the whole {wl.n:,}-value buffer of "
                             f"each rank: a single launch covering all {len(wl.buckets())} buckets (each starts on a "
                             f"256-value block boundary, so the result equals one call per bucket, bit for bit); "
                             f"one call per bucket, as a DDP hook issues them, is per_bucket_calls_*")

    if (args.workload == "ddp_1b_buckets" and args.shard == 1 and args.dtype == "f32" and args.codec == "fp8"
            and args.scale_mode == 0 and not args.no_other_workloads):
        for attr in ("pb_args", "x", "out", "ws"):  # the headline's 24 GB
            if hasattr(wl, attr):
                delattr(wl, attr)
        torch.cuda.empty_cache()
        others = {}
        for name in OTHER_WORKLOADS:
            log(f"[bench] other workload {name}")
            others[name] = workload_summary(gb, torch, args, name, max(5, min(args.steps, 20)))
            log(f"[bench] {name}: step {others[name]['step_gbs']} GB/s, {others[name]['dominant_kernel']} "
                f"{others[name]['kernel_gbs']} GB/s (frac {others[name]['kernel_frac']}), oracle sample "
                f"{others[name]['gpu_matches_oracle_on_sample']}")
        extra["other_workloads"] = others

    line = {
        "metric": METRIC,
        "value": round(value, 2),
        "unit": "GB/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms_per_step, 4),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": getattr(wl, "dt", "f32"),
        "data": "synthetic",
        "config": dict(wl.config, **extra),
        "roofline": {"bound": "hbm", "achieved": round(achieved, 2), "peak": HBM_PEAK_GBS, "unit": "GB/s",
                     "frac": round(achieved / HBM_PEAK_GBS, 4), "traffic": profiled_traffic(kname, wl.name if args.shard == 1 else f"{wl.name}_shard{args.shard}"),
                     "kernel": kname, "bytes_per_launch": int(kbytes), "us_per_launch": round(kms * 1e3, 3),
                     "frac_of_copy_ceiling": round(achieved / max(ceiling["library_copy_gbs"],
                                                                  ceiling["hipMemcpyDtoD_gbs"],
                                                                  mem_ceiling.get("best_copy_gbs", 0.0)), 4),
                     **replica_frac(achieved, mem_ceiling, wl)},
        "copy_ceiling": ceiling,
        "memory_ceiling": mem_ceiling,
        "step_distribution": dist,
        "cpu_baseline": cpu,
    }
    print(json.dumps(line), flush=True)


if __name__ == "__main__":
    main()
