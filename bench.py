"""Benchmark: routed-MoE layer tokens/s and achieved HBM GB/s on one MI355X.

A step is one moe_layer_forward call (router, top-k, bucketing, shared and
routed gate/up + SwiGLU, shared and routed down, combine) on one batch of
synthetic tokens already resident in HBM.  The default workload is the
Step-3.5-Flash-shaped layer on the MTP verify batch: 4 tokens (the last
accepted token and 3 drafts), hidden 4096, 288 routed experts, top-8, FFN
1280, routed gate/up/down in Q4_K, a Q8_0 shared expert (FFN 1280), F32
router.  Calls rotate over R independent layer instances so that no call
finds its weights in the 256 MB Infinity Cache left by the previous one.

Prints one JSON line.  `roofline` reports the dominant kernel against the
8 TB/s HBM peak: the routed gate/up stage (k_dual, which also streams the
shared down projection, for up to 16 tokens; the routed gate/up grouped
GEMM k_gemm for larger batches).  Its time comes from HIP events recorded by the library on
the launch stream; `layer_us` is the median (and spread) of per-call
event times in a second pass; for batches above 16 tokens `mfma` gives the
matrix-core utilisation; `cpu_baseline` times the CPU oracle on a bounded
sample (repeated layer calls, about 10 s on every host core and 10 s on
one core) on the host.

    python bench.py [--gpus 1] [--steps 200] [--warmup 20] [--instances 4]
                    [--events dominant|all] [--graph] [--copy-calibration MIB]
    python bench.py --summarize-counters FETCH_DIR WRITE_DIR [--copy-calibration MIB]
"""

from __future__ import annotations

import argparse
import hashlib
import json
import os
import sys
import time

import numpy as np

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

HBM_PEAK_GBS = 8000.0
DEFAULT_WORKLOAD = "step35_verify_m4"
# Dominant stage -> its kernel.  The staged path (up to 16 tokens) has three
# stages, the batched path five (its first is "route"); in both "gateup"
# moves the most bytes.
KERNEL_OF_STAGE = {"gateup": "k_dual"}
BATCHED_KERNEL = "k_gemm"


def traffic_file(kernel: str, workload: str) -> str:
    """Counter summary of `kernel` (a name, or a name with the start of its
    template arguments, e.g. "k_gemm<2, true") on `workload`."""
    return os.path.join(ROOT, "profiles", f"{kernel.split('<')[0]}_{workload}_hbm_counters.json")


def _bytes_per_row(dtype: str, cols: int) -> float:
    if dtype == "q8_0":
        return cols // 32 * 34
    return cols // 256 * {"q4_k": 144, "q2_k": 84, "q3_k": 114, "q6_k": 210}[dtype]


def layer_bytes(cfg, distinct: int, batched: bool = False) -> dict:
    """Algorithmic HBM bytes of one call: router, distinct experts, shared expert, x, y;
    and of the "gateup" stage of the staged (default) or batched path."""
    H, F, Fs, M, k = cfg.hidden, cfg.ffn, cfg.shared_ffn, cfg.n_tokens, cfg.top_k
    expert = 2 * F * _bytes_per_row(cfg.expert_type, H) + H * _bytes_per_row(cfg.routed_down_type, F)
    shared = 0
    if Fs:
        shared = 2 * Fs * _bytes_per_row(cfg.shared_type, H) + H * _bytes_per_row(cfg.shared_type, Fs)
    router = cfg.n_experts * H * 4
    xy = 2 * M * H * 4
    # Stage "gateup": routed gate/up (x in, h out) and shared down (hs in, s out).
    # Batched: the routed gate/up GEMM alone (split x in, split h out, both
    # four bytes per element).
    gateup = distinct * 2 * F * _bytes_per_row(cfg.expert_type, H) + M * H * 4 + M * k * F * 4
    if Fs and not batched:
        gateup += H * _bytes_per_row(cfg.shared_type, Fs) + M * Fs * 4 + M * H * 4
    total = router + distinct * expert + shared + xy
    return dict(total=total, layer=total, gateup=gateup)


BF16_PEAK_TFLOPS = 2500.0  # MI355X dense bf16 matrix-core peak


def mfma_utilisation(cfg, ids_per_instance, t_us: float) -> dict:
    """Matrix-core use of a batched call: the method's FLOP (routed and
    shared expert products and the router) over the call time, against the
    dense bf16 peak; and the issued fraction of the expert GEMMs, which
    pad each expert's tokens to tiles of 16 and run every product twice
    (bf16 hi and lo activation terms).  The all-ones MFMAs that give the
    activation sums are not counted."""
    H, F, Fs, M, k, E = (cfg.hidden, cfg.ffn, cfg.shared_ffn, cfg.n_tokens, cfg.top_k,
                         cfg.n_experts)
    routed = 2.0 * M * k * 3 * H * F
    shared = 2.0 * M * 3 * H * Fs
    router = 2.0 * M * E * H
    flop = routed + shared + router
    pads = []
    for ids in ids_per_instance:
        cnt = np.bincount(np.asarray(ids).reshape(-1), minlength=E)
        pads.append(float(np.sum((cnt + 15) // 16 * 16)) / (M * k))
    pad = float(np.mean(pads))
    issued = 2.0 * (routed * pad + shared * ((M + 15) // 16 * 16) / M)
    t = t_us * 1e-6
    peak = BF16_PEAK_TFLOPS * 1e12
    return {"flop": flop, "peak_tflops": BF16_PEAK_TFLOPS, "t_us": round(t_us, 2),
            "util": round(flop / (t * peak), 4),
            "issued_flop": issued, "issued_util": round(issued / (t * peak), 4),
            "token_tile_padding": round(pad, 4)}


# Sources of the operators beside the layer and verify/accept, which no
# counter profile covers.
OTHER_SOURCES = ("kv", "launch_attention", "logprobs")


def source_hash() -> str:
    h = hashlib.sha256()
    csrc = os.path.join(ROOT, "speculative_verify_router_amd", "csrc")
    for name in sorted(os.listdir(csrc)):
        if name.startswith(OTHER_SOURCES):
            continue
        with open(os.path.join(csrc, name), "rb") as f:
            h.update(name.encode() + f.read())
    return h.hexdigest()[:16]


def traffic_for(kernel: str, workload: str):
    """HBM bytes per launch of the dominant kernel from committed counter runs,
    or None if they were taken on other kernel sources."""
    try:
        with open(traffic_file(kernel, workload)) as f:
            t = json.load(f)
    except (OSError, ValueError):
        return None
    if t.get("source_hash") != source_hash() or t.get("workload") != workload:
        return None
    return t.get("bytes_per_launch")


def cpu_model() -> str:
    """The host CPU's model name from /proc/cpuinfo (empty if unreadable)."""
    try:
        with open("/proc/cpuinfo") as f:
            for line in f:
                if line.startswith("model name"):
                    return line.split(":", 1)[1].strip()
    except OSError:
        pass
    return ""


def host_cores() -> int:
    """Cores this process may run on (the machine's CPU share, not the machine's)."""
    try:
        return len(os.sched_getaffinity(0))
    except (AttributeError, OSError):
        return os.cpu_count() or 1


def _time_oracle_calls(cfg, inp, x, threads: int, budget_s: float, tokens=None):
    """Repeat layer calls of the oracle with `threads` threads (its expert
    loop) until about `budget_s` seconds are timed; `tokens` restricts the
    expert FFNs to those tokens (the routing is always computed for all)."""
    from oracle import moe_oracle as om
    from threadpoolctl import threadpool_limits
    kw = dict(top_k=cfg.top_k, ffn=cfg.ffn, expert_type=cfg.expert_type, down_type=cfg.down_type)
    if cfg.shared_ffn:
        kw.update(shared=(inp.shared_gate, inp.shared_up, inp.shared_down),
                  shared_ffn=cfg.shared_ffn, shared_type=cfg.shared_type)
    # One BLAS thread per oracle thread (the expert loop is what spreads over
    # the cores; nested BLAS pools would oversubscribe them).
    with threadpool_limits(1):
        calls, t0 = 0, time.perf_counter()
        while True:
            om.moe_layer(x, inp.router, inp.gate, inp.up, inp.down, workers=threads,
                         tokens=tokens, **kw)
            calls += 1
            dt = time.perf_counter() - t0
            if dt >= budget_s or calls >= 30:
                break
    return calls, dt


def cpu_baseline(cfg, inp, x) -> dict:
    """The oracle as it stands on whole layer calls of the workload: on every
    host core (its expert loop on that many threads), then on one core.  On
    one core a batch above 16 tokens is sampled: the FFNs of its first 16
    tokens (the routing of the whole batch is still computed)."""
    cores = host_cores()
    n_all, t_all = _time_oracle_calls(cfg, inp, x, cores, 10.0)
    one_tokens = None if cfg.n_tokens <= 16 else list(range(16))
    n_one, t_one = _time_oracle_calls(cfg, inp, x, 1, 10.0, tokens=one_tokens)
    per_call_one = cfg.n_tokens if one_tokens is None else len(one_tokens)
    one_what = "layer call(s)" if one_tokens is None else "calls on the first 16 tokens"
    return {"value": n_all * cfg.n_tokens / t_all, "unit": "tokens/s", "cores": cores,
            "kind": "oracle", "cpu_model": cpu_model(),
            "sample": f"{n_all} layer call(s) of {cfg.name} ({cfg.n_tokens} tokens each, "
                      f"instance 0), float64 NumPy, expert loop on {cores} threads, "
                      f"{t_all:.1f} s",
            "single_core": {"value": n_one * per_call_one / t_one, "unit": "tokens/s",
                            "cores": 1,
                            "sample": f"{n_one} {one_what}, one thread, {t_one:.1f} s"}}


def _counter_rows(path: str):
    """(kernel name, counter name, value) rows of every rocprofv3
    counter_collection.csv under `path`."""
    import csv
    for dirpath, _, files in os.walk(path):
        for fn in sorted(files):
            if fn.endswith("counter_collection.csv"):
                with open(os.path.join(dirpath, fn), newline="") as f:
                    for row in csv.DictReader(f):
                        yield row["Kernel_Name"], row["Counter_Name"], float(row["Counter_Value"])


def summarize_counters(fetch_dir: str, write_dir: str, workload: str, copy_bytes: int,
                       kernel: str) -> dict:
    """Scale the dominant kernel's FETCH_SIZE / WRITE_SIZE (KiB per dispatch)
    by the factors a plain copy of `copy_bytes` bytes reads on the same
    counters, and store the HBM bytes per launch for later bench runs."""
    def per_kernel(path, counter):
        acc = {}
        for name, cname, v in _counter_rows(path):
            if cname == counter:
                acc.setdefault(name, []).append(v)
        return acc

    out = {"kernel": kernel.split("<")[0], "dispatches": kernel, "workload": workload,
           "source_hash": source_hash(),
           "copy_bytes": copy_bytes}
    for counter, path in (("FETCH_SIZE", fetch_dir), ("WRITE_SIZE", write_dir)):
        acc = per_kernel(path, counter)
        prefix = f"void svr::{kernel}" if "<" in kernel else f"void svr::{kernel}<"
        dom = [v for n, vs in acc.items() if n.startswith(prefix) for v in vs]
        # The runtime's device-to-device copy kernel moving copy_bytes
        # (smaller copies of the same kernel are left out).
        cpy = [v for n, vs in acc.items() if "copybuffer" in n.lower()
               for v in vs if v * 1024 > copy_bytes / 4]
        if not dom or not cpy:
            raise SystemExit(f"{counter}: no dispatches of the dominant or copy kernel in {path}")
        scale = copy_bytes / (float(np.median(cpy)) * 1024.0)
        out[counter] = {"kib_per_launch": float(np.mean(dom)), "dispatches": len(dom),
                        "copy_kib": float(np.median(cpy)), "scale": scale,
                        "bytes_per_launch": float(np.mean(dom)) * 1024.0 * scale}
    out["bytes_per_launch"] = int(round(out["FETCH_SIZE"]["bytes_per_launch"]
                                        + out["WRITE_SIZE"]["bytes_per_launch"]))
    return out


def accept_bytes(rows: int, vocab: int, h_dim: int) -> int:
    """Algorithmic HBM bytes of one verify/accept call: the logits, the
    drafts, one verify row read and written as pending_h, the outputs."""
    return rows * vocab * 4 + (rows - 1) * 4 + 2 * h_dim * 4 + (2 * rows + 1) * 4


def cpu_baseline_accept(batch) -> dict:
    """The verify/accept oracle as it stands, repeated on one batch for about 10 s."""
    from oracle import accept_oracle as ao
    calls, t0 = 0, time.perf_counter()
    while True:
        ao.verify_accept(batch.logits, batch.drafts, batch.verify_h)
        calls += 1
        dt = time.perf_counter() - t0
        if dt >= 10.0:
            break
    M, V = batch.logits.shape
    return {"value": calls / dt, "unit": "batches/s", "cores": 1, "kind": "oracle",
            "cpu_model": cpu_model(),
            "sample": f"{calls} oracle calls on one verify batch ({M} rows x {V} logits, "
                      f"NumPy on one thread), {dt:.1f} s"}


def bench_accept(args) -> int:
    """Greedy verify/accept of a verify batch (moe_verify_accept): batches/s.

    Calls rotate over enough seeded batches (about 330 MB of logits) that no
    call finds its logits in the 256 MB Infinity Cache; every timed call is
    bracketed by HIP events on the launch stream."""
    import torch
    import speculative_verify_router_amd as svr
    import synth

    w = synth.ACCEPT_WORKLOADS[args.workload]
    M, V, Hd = w["rows"], w["vocab"], w["h_dim"]
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    per = M * V * 4
    R = max(args.instances, (330 << 20) // per + 1)
    batches, host0 = [], None
    for i in range(R):
        b = synth.draw_verify_batch(M, V, Hd, i % M, seed=i)
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        batches.append((up(b.logits), up(b.drafts), up(b.verify_h)))
        if i == 0:
            host0 = b
    print(f"# {R} verify batches resident", file=sys.stderr, flush=True)
    ws = svr.accept_workspace(M, V, dev)
    tok = torch.empty(M, dtype=torch.int32, device=dev)
    acc = torch.empty(M, dtype=torch.int32, device=dev)
    n = torch.empty(1, dtype=torch.int32, device=dev)
    pend = torch.empty(Hd, dtype=torch.float32, device=dev)
    stream = torch.cuda.current_stream()

    def call(i):
        lg, dr, vh = batches[i % R]
        svr.moe_verify_accept(lg, dr, tok, acc, n, vh, pend, ws=ws, stream=stream)

    for s in range(max(args.warmup, 1)):
        call(s)
    K = args.steps
    evs = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
           for _ in range(K)]
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for s in range(K):
        evs[s][0].record(stream)
        call(s)
        evs[s][1].record(stream)
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    ev_ms = float(np.mean([a.elapsed_time(b) for a, b in evs]))
    nbytes = accept_bytes(M, V, Hd)
    achieved = nbytes / (ev_ms * 1e-3) / 1e9
    out = {
        "metric": f"greedy MTP verify/accept batches/s (M={M} rows, {V}-column logits), 1 MI355X",
        "value": round(K / elapsed, 1),
        "unit": "batches/s",
        "n_gpus": 1,
        "steps": K,
        "warmup": args.warmup,
        "ms_per_step": round(elapsed * 1e3 / K, 5),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "f32",
        "data": "synthetic",
        "config": {"workload": args.workload, "rows": M, "vocab": V, "h_dim": Hd,
                   "batches_rotated": R},
        "roofline": {
            "kernel": "k_accept", "bound": "hbm", "achieved": round(achieved, 1),
            "peak": HBM_PEAK_GBS, "unit": "GB/s", "frac": round(achieved / HBM_PEAK_GBS, 4),
            "traffic": traffic_for("k_accept", args.workload), "bytes_per_launch": nbytes,
            "avg_launch_us": round(ev_ms * 1e3, 3), "timed_launches": K,
        },
    }
    if not args.no_cpu_baseline:
        out["cpu_baseline"] = cpu_baseline_accept(host0)
    print(json.dumps(out), flush=True)
    return 0


def bench_step(args) -> int:
    """A verify step's operators in the order of use: cache append, attention,
    the layer, verify/accept, log probabilities: steps/s.

    Steps rotate over layer and cache instances as the layer's own workload
    does; a graph of one step an instance is timed as well."""
    import torch
    import speculative_verify_router_amd as svr
    import synth

    w = synth.STEP_WORKLOADS[args.workload]
    cfg = synth.CONFIGS[w["layer"]]
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    M, D, P, V, top = cfg.n_tokens, w["dim"], w["page"], w["vocab"], w["top"]
    ld = svr.LayerDesc(cfg.hidden, cfg.n_experts, cfg.top_k, cfg.ffn, cfg.shared_ffn,
                       cfg.expert_type, cfg.shared_type, down_type=cfg.down_type)
    kd = svr.KvDesc(w["heads"], w["kv_heads"], D, P, rotary_dims=w["rotary"])
    i32, f32 = dict(dtype=torch.int32, device=dev), dict(dtype=torch.float32, device=dev)
    pages = -(-w["length"] // P)
    gen = torch.Generator(device=dev).manual_seed(0)
    steps = []
    for i in range(max(1, args.instances)):
        inp = synth.draw_layer(cfg, instance=i)
        x, _ = synth.draw_tokens(cfg, instance=i)
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        lw = svr.LayerWeights(up(inp.router), up(inp.gate), up(inp.up), up(inp.down))
        if cfg.shared_ffn:
            lw.shared_gate, lw.shared_up, lw.shared_down = (up(inp.shared_gate), up(inp.shared_up),
                                                            up(inp.shared_down))
        batch = svr.KvBatch(torch.tensor([0, M], **i32), torch.tensor([w["length"]], **i32),
                            torch.randperm(pages, generator=gen, device=dev).int()[None].contiguous(), M)
        cache = svr.kv_cache(kd, pages)
        cache.random_(0, 256, generator=gen)
        cache[..., P * D:] = 126  # scales of 1/2: codes of up to 3
        qkv = torch.randn((M, (w["heads"] + 2 * w["kv_heads"]) * D), generator=gen, device=dev).bfloat16()
        q, k, v = (t.unflatten(1, (-1, D)) for t in
                   qkv.split([w["heads"] * D, w["kv_heads"] * D, w["kv_heads"] * D], 1))
        b = synth.draw_verify_batch(M, V, 0, i % M, seed=i)
        steps.append((lw, up(x), batch, cache, q, k, v, up(b.logits), up(b.drafts)))
        print(f"# instance {i} resident", file=sys.stderr, flush=True)
    norm = torch.ones(D, **f32)
    inv_freq = 10000.0 ** (-torch.arange(0, w["rotary"], 2, **f32) / w["rotary"])
    qo = torch.empty((M, w["heads"], D), dtype=torch.bfloat16, device=dev)
    att, y = torch.empty_like(qo), torch.empty((M, cfg.hidden), **f32)
    tok, acc, n = torch.empty(M, **i32), torch.empty(M, **i32), torch.empty(1, **i32)
    lp, ent = torch.empty(M, **f32), torch.empty(M, **f32)
    ids, tlp = torch.empty((M, top), **i32), torch.empty((M, top), **f32)
    ws = (svr.kv_workspace(kd, steps[0][2], M), svr.workspace(ld, M), svr.accept_workspace(M, V),
          svr.logprobs_workspace(M, V, top))

    def call(i):
        lw, x, batch, cache, q, k, v, logits, drafts = steps[i % len(steps)]
        svr.moe_kv_append(kd, batch, q, k, v, cache, qo, q_norm=norm, k_norm=norm, inv_freq=inv_freq)
        svr.moe_kv_attention(kd, batch, qo, cache, att, ws=ws[0])
        svr.moe_layer_forward(ld, lw, x, y, None, None, ws=ws[1])
        svr.moe_verify_accept(logits, drafts, tok, acc, n, ws=ws[2])
        svr.moe_logprobs(logits, tok, lp, ent, ids, tlp, ws=ws[3])

    def timed(f, count):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for s in range(count):
            f(s)
        torch.cuda.synchronize()
        return (time.perf_counter() - t0) / count

    for s in range(max(args.warmup, len(steps))):
        call(s)
    eager = timed(call, args.steps)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        for s in range(len(steps)):
            call(s)
    g.replay()
    rounds = max(1, args.steps // len(steps))
    graph = timed(lambda s: g.replay(), rounds) / len(steps)
    print(json.dumps({
        "metric": f"verify steps/s (append, attention, layer, accept, log probabilities; M={M}), 1 MI355X",
        "value": round(1 / eager, 1), "unit": "steps/s", "n_gpus": 1, "steps": args.steps,
        "warmup": args.warmup, "ms_per_step": round(eager * 1e3, 5), "higher_is_better": True,
        "scaling": "weak", "vs_baseline": None, "dtype": "bf16", "data": "synthetic",
        "config": {"workload": args.workload, **w, "rows": M, "instances": len(steps)},
        "graph_ms_per_step": round(graph * 1e3, 5)}), flush=True)
    return 0


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--warmup", type=int, default=20)
    ap.add_argument("--instances", type=int, default=4, help="layer instances rotated over")
    ap.add_argument("--workload", default=DEFAULT_WORKLOAD)
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--events", choices=["dominant", "all"], default="dominant",
                    help="HIP events per step: around the dominant stage only, or every stage")
    ap.add_argument("--event-every", type=int, default=5, metavar="N",
                    help="record the stage events on every N-th timed step only (the markers "
                         "delay the next launch; the other steps run without them)")
    ap.add_argument("--graph", action="store_true",
                    help="also time the same steps replayed from a captured HIP graph")
    ap.add_argument("--copy-calibration", type=int, default=0, metavar="MIB",
                    help="after the timed steps, run five plain device copies of MIB MiB "
                         "(the reference kernel for the HBM byte counters)")
    ap.add_argument("--summarize-counters", nargs=3, metavar=("KERNEL", "FETCH_DIR", "WRITE_DIR"),
                    help="read rocprofv3 FETCH_SIZE / WRITE_SIZE runs of this script (taken "
                         "with --copy-calibration) and write KERNEL's HBM bytes per launch")
    args = ap.parse_args(argv)

    if args.summarize_counters:
        kern, fdir, wdir = args.summarize_counters
        t = summarize_counters(fdir, wdir, args.workload, (args.copy_calibration or 512) << 20,
                               kern)
        with open(traffic_file(kern, args.workload), "w") as f:
            json.dump(t, f, indent=1)
        print(json.dumps(t))
        return 0

    if args.gpus != 1 or int(os.environ.get("WORLD_SIZE", "1")) != 1:
        print("bench.py measures one GPU: the layer is built and timed on a single MI355X; "
              "runs on more than one GPU are not supported.", file=sys.stderr)
        return 2

    import torch
    import speculative_verify_router_amd as svr
    import synth

    if args.workload in synth.ACCEPT_WORKLOADS:
        return bench_accept(args)
    if args.workload in synth.STEP_WORKLOADS:
        return bench_step(args)
    cfg = synth.CONFIGS[args.workload]
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    desc = svr.LayerDesc(cfg.hidden, cfg.n_experts, cfg.top_k, cfg.ffn, cfg.shared_ffn,
                         cfg.expert_type, cfg.shared_type, down_type=cfg.down_type)
    M, k = cfg.n_tokens, cfg.top_k
    R = max(1, args.instances)

    t_gen = time.perf_counter()
    layers, xs, host0 = [], [], None
    for i in range(R):
        inp = synth.draw_layer(cfg, instance=i)
        x, _ = synth.draw_tokens(cfg, instance=i)
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        w = svr.LayerWeights(up(inp.router), up(inp.gate), up(inp.up), up(inp.down))
        if cfg.shared_ffn:
            w.shared_gate, w.shared_up, w.shared_down = (up(inp.shared_gate), up(inp.shared_up),
                                                         up(inp.shared_down))
        layers.append(w)
        xs.append(up(x))
        if i == 0:
            host0 = (inp, x)
        print(f"# instance {i} resident ({time.perf_counter() - t_gen:.1f} s)", file=sys.stderr,
              flush=True)
    ws = svr.workspace(desc, M, dev)
    y = torch.empty((M, cfg.hidden), dtype=torch.float32, device=dev)
    ids = [torch.empty((M, k), dtype=torch.int32, device=dev) for _ in range(R)]
    tw = [torch.empty((M, k), dtype=torch.float32, device=dev) for _ in range(R)]
    stream = torch.cuda.current_stream()

    calls = [svr.PreparedForward(desc, layers[i], xs[i], y, ids[i], tw[i], ws, stream)
             for i in range(R)]
    for s in range(args.warmup):
        calls[s % R]()
    torch.cuda.synchronize()
    if args.warmup < R:
        for i in range(R):
            calls[i]()
        torch.cuda.synchronize()
    distinct = [len(np.unique(t.cpu().numpy())) for t in ids]

    nst = svr.moe_stage_count(desc, M)
    names = [svr.moe_stage_name(desc, M, j) for j in range(nst)]
    DOMINANT = "gateup"
    batched = names[0] == "route"
    kernel = BATCHED_KERNEL if batched else KERNEL_OF_STAGE[DOMINANT]
    K = args.steps
    evs = [[torch.cuda.Event(enable_timing=True) for _ in range(nst + 1)] for _ in range(K)]
    for row in evs:  # create the underlying HIP events before the timed region
        for e in row:
            e.record(stream)
    import ctypes
    dom = names.index(DOMINANT)
    if args.events == "all":
        ev_arrays = [(ctypes.c_void_p * (nst + 1))(*[e.cuda_event for e in row]) for row in evs]
    else:
        # Only the dominant stage's boundaries carry real events; the others
        # are NULL entries, which the library skips.
        ev_arrays = [(ctypes.c_void_p * (nst + 1))(
            *[row[j].cuda_event if j in (dom, dom + 1) else None for j in range(nst + 1)])
            for row in evs]
    torch.cuda.synchronize()

    every = max(1, args.event_every)
    timed = [s for s in range(K) if s % every == 0]
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for s in range(K):
        calls[s % R](ev_arrays[s] if s % every == 0 else None)
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0

    stage_ms = np.zeros(nst)
    dom_ms, dom_bytes = 0.0, 0.0
    lay_bytes = 0.0
    for s in range(K):
        lay_bytes += layer_bytes(cfg, distinct[s % R])["total"]
    for s in timed:
        i = s % R
        if args.events == "all":
            stage_ms += [evs[s][j].elapsed_time(evs[s][j + 1]) for j in range(nst)]
        dom_ms += evs[s][dom].elapsed_time(evs[s][dom + 1])
        dom_bytes += layer_bytes(cfg, distinct[i], batched)[DOMINANT]

    graph_ms = None
    if args.graph:
        # One captured graph holds one call per instance; replays keep the
        # same rotation.  The workspace counters return to zero every call.
        g = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        gcalls = [svr.PreparedForward(desc, layers[i], xs[i], y, ids[i], tw[i], ws, side)
                  for i in range(R)]
        with torch.cuda.stream(side):
            for c in gcalls:
                c()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            for c in gcalls:
                c()
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        reps = max(1, K // R)
        t1 = time.perf_counter()
        for _ in range(reps):
            g.replay()
        torch.cuda.synchronize()
        graph_ms = (time.perf_counter() - t1) * 1e3 / (reps * R)

    # Per-call layer time: each call bracketed by two events on the launch
    # stream (a separate pass, so the whole-job timing above has no markers).
    call_ev = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
               for _ in range(K)]
    for a, b in call_ev:
        a.record(stream)
        b.record(stream)
    torch.cuda.synchronize()
    for s in range(K):
        call_ev[s][0].record(stream)
        calls[s % R]()
        call_ev[s][1].record(stream)
    torch.cuda.synchronize()
    per_call_us = np.array([a.elapsed_time(b) for a, b in call_ev]) * 1e3

    if args.copy_calibration:
        n = args.copy_calibration << 18  # floats
        src = torch.ones(n, dtype=torch.float32, device=dev)
        dst = torch.empty_like(src)
        for _ in range(5):
            dst.copy_(src)
        torch.cuda.synchronize()
        del src, dst

    ms_per_step = elapsed * 1e3 / K
    value = M * K / elapsed
    achieved = dom_bytes / (dom_ms * 1e-3) / 1e9
    traffic = traffic_for(kernel, cfg.name)

    metric = "MoE layer tokens/s + achieved HBM GB/s at verify batch M=4 (Q4_K), 1 MI355X"
    if cfg.name != DEFAULT_WORKLOAD:
        metric = f"MoE layer tokens/s + achieved HBM GB/s, {cfg.name} ({M} tokens), 1 MI355X"
    # Arithmetic of the expert products: integer quants times 16-bit integer
    # activations (int8 limbs, int32 sums, fp32 scales) up to 16 tokens; bf16
    # matrix-core products of exact integer quants and split activations above,
    # for every routed type and pairing of gate/up and down types.
    int_path = M <= 16
    dtype = "i8xi16->i32+f32" if int_path else "bf16x2->f32"
    out = {
        "metric": metric,
        "value": round(value, 1),
        "unit": "tokens/s",
        "n_gpus": 1,
        "steps": K,
        "warmup": args.warmup,
        "ms_per_step": round(ms_per_step, 5),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": dtype,
        "data": "synthetic",
        "config": {
            "workload": cfg.name, "tokens": M, "hidden": cfg.hidden, "experts": cfg.n_experts,
            "top_k": k, "ffn": cfg.ffn, "shared_ffn": cfg.shared_ffn,
            "routed": cfg.expert_type, "routed_down": cfg.routed_down_type,
            "shared": cfg.shared_type, "router": "f32",
            "instances_rotated": R, "distinct_experts": distinct,
        },
        "hbm_gbps": round(lay_bytes / K / (ms_per_step * 1e-3) / 1e9, 1),
        "layer_bytes": int(round(lay_bytes / K)),
        "events": args.events,
        "roofline": {
            "kernel": kernel, "stage": DOMINANT, "bound": "hbm", "achieved": round(achieved, 1),
            "peak": HBM_PEAK_GBS, "unit": "GB/s", "frac": round(achieved / HBM_PEAK_GBS, 4),
            "traffic": traffic, "bytes_per_launch": int(round(dom_bytes / len(timed))),
            "avg_launch_us": round(dom_ms * 1e3 / len(timed), 3), "timed_launches": len(timed),
        },
    }
    out["layer_us"] = {"median": round(float(np.median(per_call_us)), 2),
                       "p10": round(float(np.percentile(per_call_us, 10)), 2),
                       "p90": round(float(np.percentile(per_call_us, 90)), 2),
                       "calls": K, "how": "HIP events around each call, separate pass"}
    if batched:
        out["mfma"] = mfma_utilisation(cfg, [t.cpu().numpy() for t in ids],
                                       float(np.median(per_call_us)))
    if args.events == "all":
        out["stage_us"] = {n: round(v * 1e3 / len(timed), 2) for n, v in zip(names, stage_ms)}
    if graph_ms is not None:
        out["graph_replay"] = {"ms_per_step": round(graph_ms, 5),
                               "tokens_per_s": round(M / (graph_ms * 1e-3), 1)}
    if not args.no_cpu_baseline:
        out["cpu_baseline"] = cpu_baseline(cfg, *host0)
    print(json.dumps(out), flush=True)
    return 0


if __name__ == "__main__":
    sys.exit(main())
