"""Benchmark: DFlash speculative decode (block 8) on the E4B-shaped synthetic pair at 1k context.

One JSON line on stdout. A step is one speculative pass: draft block -> plant proposals -> batched
verify of 8 rows -> accept -> commit_verify_rows. `value` is decode tokens/s with every input resident
in HBM (weights, KV state, the planted-proposal table); `e2e` is the same loop through the host-buffer
calls (proposals copied in from host memory, proposals and target tokens copied out every step).
`roofline` reports the Q4_1 products (the dominant kernel) against the measured HBM copy bandwidth;
`cpu_baseline` times the oracle on a bounded sample of the same workload.

  python bench.py [--gpus N] [--steps K] [--warmup W] [--impl cuda|reference]
                  [--workload e4b|gemm|cut|27b|prefill|attn|long|draft]

`--workload 27b` runs the same step on the 27B-class pair (62 dense layers of width 5376, 16 GB of Q4_1
weights); `cut` is a 12-layer E4B cut for profiling captures; `gemm` the isolated product sweep;
`prefill` the tcgen05 product at many rows; `attn` a short attention profiling workload; `long` sampled
serving at long contexts over a pinned prefix (requests A, B, A); `draft` the draft on its own at contexts
of 30, 1024 and 4096 rows. Only the default prints the bench line.
"""
from __future__ import annotations

import argparse
import json
import os
import statistics
import subprocess
import sys
import threading
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

import numpy as np  # noqa: E402

import gen  # noqa: E402

PEAKS_FALLBACK = {"hbm_gbs": 6800.0, "bf16_tflops": 1900.0}
METRIC = "spec-decode tok/s (block 8, 1 GB300); Q4_1 verify-GEMM HBM GB/s vs 8 TB/s"


def peaks():
    p = os.path.join(ROOT, "MEASURED_PEAKS.json")
    if os.path.exists(p):
        d = json.load(open(p))
        return {"hbm_gbs": float(d["hbm_gbs"]), "bf16_tflops": float(d["bf16_tflops"]), "src": "measured"}
    return dict(PEAKS_FALLBACK, src="fallback")


class Clocks:
    """nvidia-smi samples (every 20 ms) with their host arrival times; stop() reports the samples that
    fell inside the timed window (and all of them when fewer than three did)."""

    def __init__(self, index=0):
        self.index, self.samples, self.proc = index, [], None
        self.t0 = self.t1 = None

    def start(self):
        q = ("index,clocks.sm,clocks.max.sm,power.draw,clocks_event_reasons.active,clocks_event_reasons.hw_slowdown,"
             "clocks_event_reasons.hw_thermal_slowdown,clocks_event_reasons.sw_thermal_slowdown,"
             "clocks_event_reasons.sw_power_cap")
        try:
            self.proc = subprocess.Popen(["nvidia-smi", f"--id={self.index}", f"--query-gpu={q}",
                                          "--format=csv,noheader,nounits", "-lms", "20"],
                                         stdout=subprocess.PIPE, stderr=subprocess.DEVNULL, text=True)
            self.thread = threading.Thread(target=self._read, daemon=True)
            self.thread.start()
            time.sleep(0.3)   # the first samples arrive before the timed region
        except OSError:
            self.proc = None

    def _read(self):
        for line in self.proc.stdout:
            parts = [x.strip() for x in line.split(",")]
            if len(parts) >= 9:
                self.samples.append((time.time(), parts))

    def window(self, t0, t1):
        self.t0, self.t1 = t0, t1

    def stop(self):
        time.sleep(0.1)
        if self.proc:
            self.proc.terminate()
            try:
                self.proc.wait(timeout=5)
            except subprocess.TimeoutExpired:
                self.proc.kill()
        inside = [p for t, p in self.samples if self.t0 is not None and self.t0 <= t <= self.t1 + 0.05]
        use = inside if len(inside) >= 3 else [p for _, p in self.samples]
        sm = [float(s[1]) for s in use if s[1].replace(".", "").isdigit()]
        mx = [float(s[2]) for s in use if s[2].replace(".", "").isdigit()]
        names = ["hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown", "sw_power_cap"]
        reasons = sorted({names[i] for s in use for i in range(4) if s[5 + i].lower() == "active"})
        return {"sm_mhz": statistics.median(sm) if sm else None, "sm_max_mhz": max(mx) if mx else None,
                "reasons": reasons, "samples": len(use), "samples_in_timed_region": len(inside),
                "period_ms": 20}


# ---------------------------------------------------------------------------------------------------
# workload
# ---------------------------------------------------------------------------------------------------
def cut_pair(max_ctx):
    """A 12-layer cut of the E4B-shaped target (layers 8-11 KV-shared, vocabulary 32768) with the full
    5-layer draft: the same kernels at the same per-layer shapes in about 2 GB (profiling captures)."""
    import dataclasses
    V = 32768
    t = gen.e4b_target(n_layers=12, first_shared=8, vocab=V)
    d = dataclasses.replace(gen.e4b_draft(vocab=V), taps=(1, 3, 5, 8, 11))
    return gen.PairConfig(t, d, max_ctx=max_ctx)


def e4b_workload(args):
    if args.workload == "27b":
        pc = gen.b27_pair(max_ctx=args.ctx + args.gen + 64)
        return pc, {"workload": f"27b-pair ctx {args.ctx} block 8 greedy, planted drafts p={args.p}, "
                                f"{args.gen}-token decodes", "target": "62 layers hidden 5376 ffn 21504 32/16x128 heads, "
                                "5 sliding (window 1024) : 1 full, vocab 262144, Q4_1",
                    "draft": "5 layers hidden 5376 ffn 10752 32/8x128, fc 5x5376", "context": args.ctx,
                    "generated_per_decode": args.gen, "corruption_p": args.p,
                    "note": "second workload (the 27B-class pair), not the benchmark configuration",
                    "l2": "weights streamed per step (about 17 GB) exceed the 129 MB L2"}
    if args.workload == "cut":
        pc = cut_pair(args.ctx + args.gen + 64)
        return pc, {"workload": f"e4b-cut (12 layers, vocab 32768) ctx {args.ctx} block 8 greedy, planted drafts "
                                f"p={args.p}, {args.gen}-token decodes", "context": args.ctx,
                    "note": "profiling workload, not the benchmark configuration"}
    pc = gen.e4b_pair(max_ctx=args.ctx + args.gen + 64)
    return pc, {"workload": f"e4b-pair ctx {args.ctx} block 8 greedy, planted drafts p={args.p}, "
                            f"{args.gen}-token decodes", "target": "42 layers hidden 2560 ffn 10240/20480 12x256 heads, "
                            "PLE 256, vocab 262144, Q4_1", "draft": "5 layers hidden 2560 ffn 5120 32/8x128, fc 5x2560",
                "context": args.ctx, "generated_per_decode": args.gen, "corruption_p": args.p,
                "l2": "weights streamed per step (6.4 GB) exceed the 129 MB L2"}


def load_engine(pc, keep=False, workers=None, prefill_rows=0, kv8=0):
    from dflash_speculative_decode_gb300 import Engine, config_from_pair
    eng = Engine(config_from_pair(pc, prefill_rows=prefill_rows, kv8=kv8))
    kept = {} if keep else None
    workers = workers or min(16, os.cpu_count() or 1)
    t0 = time.time()
    for name, arr in gen.iter_tensors(pc, workers=workers):
        eng.load_tensor(name, arr)
        if keep:
            kept[name] = arr
    return eng, kept, time.time() - t0


def planted_table(torch, eng, pc, first, n_gen, p):
    """Plain greedy decode on the GPU from the prefilled state (untimed) gives the target's own tokens G;
    the planted proposal for absolute position q is G[q] unless the position is corrupted
    (gen.corruption, keyed by q). Returns the prefix snapshot (taken before the decode)."""
    snap = eng.dfl_snapshot()
    P = eng.dfl_positions_held()
    toks = [first]
    while len(toks) < n_gen:
        tt, _ = eng.dfl_verify_block([toks[-1]])
        eng.dfl_commit_verify_rows(1)
        toks.append(int(tt[0]))
    L = pc.max_ctx + 32
    G = np.zeros(L, np.int32)
    G[P:P + len(toks)] = toks
    cor = gen.corruption(p, pc.target.vocab, L)
    table = cor.propose(G, np.arange(L))
    return snap, toks, torch.from_numpy(table).cuda()


def run_steps(eng, torch, table_dev, first_tok, snap, n0, steps, n_gen, host_rows=None, accepted=None):
    """`steps` speculative passes; a 512-token decode that runs out restarts from the prefix snapshot.
    Device mode: proposals planted from the device table. Host mode (host_rows = host table): proposals
    read back to host, planted there, and passed in host memory. `accepted`, when a list, receives each
    pass's accepted length."""
    from dflash_speculative_decode_gb300 import DFL_KEEP_ACCEPTED
    B = eng.cfg.block
    tokens = 0
    last = first_tok
    produced = 1
    for _ in range(steps):
        if produced >= n_gen:
            eng.dfl_restore(snap)
            last, produced = first_tok, 1
        if host_rows is None:
            eng.dfl_draft_block(last, want=False)
            eng.dfl_plant_proposals(table_dev)
            tt, a = eng.dfl_verify_block(None, k=B)
        else:
            n = eng.dfl_positions_held()
            eng.dfl_draft_block(last, want=True)
            rows = np.concatenate([[last], host_rows[n + 1:n + B]]).astype(np.int32)
            tt, a = eng.dfl_verify_block(rows)
        eng.dfl_commit_verify_rows(DFL_KEEP_ACCEPTED)
        last = int(tt[a])
        tokens += a + 1
        produced += a + 1
        if accepted is not None:
            accepted.append(a)
    return tokens


def acceptance(accepted, block):
    """Accepted proposals per pass, their histogram over 0..block-1, and the first proposal's hit rate."""
    n = max(len(accepted), 1)
    hist = [sum(1 for a in accepted if a == i) for i in range(block)]
    return {"accepted_per_pass": round(sum(accepted) / n, 4), "tokens_per_pass": round(1 + sum(accepted) / n, 4),
            "histogram": hist, "first_proposal_hit_rate": round(sum(1 for a in accepted if a >= 1) / n, 4),
            "passes": len(accepted)}


def combine_ranks(torch, ms: float, toks: float, device) -> tuple:
    """Replicas: the job's time is the slowest rank's, its tokens the sum over ranks."""
    t = torch.tensor([ms, toks], dtype=torch.float64, device=device)
    mx = t.clone()
    torch.distributed.all_reduce(mx, op=torch.distributed.ReduceOp.MAX)
    torch.distributed.all_reduce(t, op=torch.distributed.ReduceOp.SUM)
    return float(mx[0]), float(t[1])


# In-pass durations of the Q4_1 products (device clock, dfl_profile_read) are paired with the DRAM bytes
# ncu counted for one product launch of the same kernel source. The fraction dram/algorithmic of that
# capture scales to the average launch of the step; it is reported only while the product kernel's
# source still hashes to the value it had when the counters were taken.
TRAFFIC_CAPTURE = {"gemm_cu_sha16": "89c08baea2d03c0f", "dram_bytes": 16513536, "algorithmic_bytes": 16793600,
                   "profile": "profiles/k_gemm_q41_2560x10240_m8.md"}


def _gemm_source_hash():
    import hashlib
    src = os.path.join(ROOT, "dflash_speculative_decode_gb300", "csrc", "gemm.cu")
    return hashlib.sha256(open(src, "rb").read()).hexdigest()[:16]


def roofline(prof, steps, ms_step, pk):
    """The dominant kernel (the Q4_1 products) against measured HBM, from the in-pass stamps of a
    profiled rerun of the same steps."""
    names = ["q41_products", "bf16_products", "head", "attention", "qk_norm_rope_kv", "rows_embed_sample"]
    (q_n, q_ms, q_bytes), (f_n, f_ms, f_bytes), (h_n, h_ms, h_bytes) = prof[:3]
    total = sum(p[1] for p in prof)
    breakdown = {nm: {"launches_per_step": round(p[0] / steps, 1), "ms_per_step": round(p[1] / steps, 4),
                      "share_of_step": round(p[1] / steps / ms_step, 3) if ms_step else None}
                 for nm, p in zip(names, prof)}
    breakdown["untimed_rest_ms_per_step"] = round(max(ms_step - total / steps, 0.0), 4)
    breakdown["note"] = ("in-pass device durations (earliest CTA past its dependency wait to the latest CTA done) "
                         "of a profiled rerun of the same steps; programmatic-launch overlap kept")
    achieved = q_bytes / (q_ms / 1e3) / 1e9 if q_ms else 0.0
    per_launch = q_bytes / max(q_n, 1)
    traffic = None
    if TRAFFIC_CAPTURE and TRAFFIC_CAPTURE.get("gemm_cu_sha16") == _gemm_source_hash():
        traffic = round(per_launch * TRAFFIC_CAPTURE["dram_bytes"] / TRAFFIC_CAPTURE["algorithmic_bytes"])
    return {"bound": "hbm", "achieved": round(achieved, 1), "peak": pk["hbm_gbs"], "unit": "GB/s",
            "frac": round(achieved / pk["hbm_gbs"], 4), "traffic": traffic,
            "kernel": "k_gemm (the Q4_1 products of draft and verify)", "peak_source": pk["src"],
            "frac_vs_8TBs": round(achieved / 8000.0, 4), "launches": q_n,
            "avg_launch_us": round(q_ms * 1e3 / max(q_n, 1), 2), "bytes_per_launch": round(per_launch),
            "traffic_capture": (TRAFFIC_CAPTURE or {}).get("profile"),
            "head": {"achieved": round(h_bytes / (h_ms / 1e3) / 1e9, 1) if h_ms else None, "launches": h_n,
                     "avg_launch_us": round(h_ms * 1e3 / max(h_n, 1), 2),
                     "frac": round(h_bytes / (h_ms / 1e3) / 1e9 / pk["hbm_gbs"], 4) if h_ms else None},
            "breakdown": breakdown}


def bench_cuda(args):
    import torch
    from dflash_speculative_decode_gb300 import build
    from dflash_speculative_decode_gb300._abi import DFL_OPT_PROFILE
    build.build()
    rank = int(os.environ.get("RANK", "0"))
    world = int(os.environ.get("WORLD_SIZE", "1"))
    local = int(os.environ.get("LOCAL_RANK", "0"))
    if world > 1:
        torch.distributed.init_process_group("nccl" if torch.cuda.is_available() else "gloo")
    torch.cuda.set_device(local)
    pc, cfgdesc = e4b_workload(args)
    want_cpu = rank == 0 and world == 1 and not args.no_cpu_baseline and args.workload == "e4b"
    eng, W, t_load = load_engine(pc, keep=want_cpu, prefill_rows=args.prefill_rows)
    prompt = gen.prompt(pc.target.vocab, args.ctx)
    # the prompt ingest, timed on its second run (the first one sets up graphs and kernel attributes)
    snap_empty = eng.dfl_snapshot()
    eng.dfl_prefill(prompt)
    eng.dfl_restore(snap_empty)
    del snap_empty
    torch.cuda.synchronize()
    t0 = time.time()
    first = eng.dfl_prefill(prompt)
    torch.cuda.synchronize()
    t_prefill = time.time() - t0
    snap, plain, table = planted_table(torch, eng, pc, first, args.gen, args.p)
    eng.dfl_restore(snap)
    n0 = eng.dfl_positions_held()
    stream = torch.cuda.current_stream()

    # warm-up
    run_steps(eng, torch, table, first, snap, n0, args.warmup, args.gen)
    eng.dfl_restore(snap)
    sys.stderr.write(f"[bench] kernel launches before the timed region: {eng.dfl_launch_count()}\n")
    # timed: device-resident loop
    clk = Clocks(local)
    clk.start()
    if world > 1:
        torch.distributed.barrier()
    torch.cuda.synchronize()
    l0 = eng.dfl_launch_count()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t_wall0 = time.time()
    e0.record(stream)
    acc = []
    toks = run_steps(eng, torch, table, first, snap, n0, args.steps, args.gen, accepted=acc)
    e1.record(stream)
    torch.cuda.synchronize()
    clk.window(t_wall0, time.time())
    launches = eng.dfl_launch_count() - l0
    ms = e0.elapsed_time(e1)
    clocks = clk.stop()
    if world > 1:
        ms, toks_all = combine_ranks(torch, ms, toks, "cuda")
    else:
        toks_all = toks
    value = toks_all / (ms / 1e3)

    # e2e: host-buffer calls
    eng.dfl_restore(snap)
    host_table = table.cpu().numpy()
    torch.cuda.synchronize()
    t1 = time.perf_counter()
    toks_e2e = run_steps(eng, torch, table, first, snap, n0, args.steps, args.gen, host_rows=host_table)
    torch.cuda.synchronize()
    e2e_s = time.perf_counter() - t1

    # roofline: the same steps again with every pass's launches stamped on the device
    eng.dfl_restore(snap)
    eng.dfl_set_option(DFL_OPT_PROFILE, 1)
    run_steps(eng, torch, table, first, snap, n0, args.steps, args.gen)
    prof = [eng.dfl_profile_read(i) for i in range(6)]
    eng.dfl_set_option(DFL_OPT_PROFILE, 0)
    pk = peaks()
    roof = roofline(prof, args.steps, ms / args.steps, pk)

    out = {"metric": METRIC, "value": round(value, 2), "unit": "tokens/s", "n_gpus": world, "steps": args.steps,
           "warmup": args.warmup, "ms_per_step": round(ms / args.steps, 4), "higher_is_better": True,
           "scaling": "weak", "vs_baseline": None, "dtype": "fp32 activations, Q4_1/bf16 weights",
           "data": f"synthetic (seeded random-init weights of the {'27B-class' if args.workload == '27b' else 'E4B-shaped'}"
                   " pair, uniform prompt)",
           "config": dict(cfgdesc, parallelism=f"replicas x{world}" if world > 1 else "single GPU"),
           "tokens_per_step": round(toks_all / world / args.steps, 3),
           "acceptance": dict(acceptance(acc, pc.draft.block), planted_p=args.p,
                              expected_tokens_per_pass=round(1 + sum((1 - args.p) ** i for i in range(1, pc.draft.block)), 4)),
           "e2e": {"value": round(toks_e2e / e2e_s, 2), "unit": "tokens/s", "h2d_bytes_per_step": 4 * pc.draft.block,
                   "d2h_bytes_per_step": 4 * (pc.draft.block - 1) + 4 * pc.draft.block + 4},
           "gpu_launches": launches, "roofline": roof, "clocks": clocks,
           "setup_s": {"load": round(t_load, 1), "prefill": round(t_prefill, 3)},
           "prefill": {"tokens": args.ctx, "seconds": round(t_prefill, 4), "tokens_per_s": round(args.ctx / t_prefill, 1),
                       "prefill_rows": args.prefill_rows,
                       "note": "dfl_prefill wall time (second run); passes of up to prefill_rows rows with the "
                               "products on tcgen05, else passes of 16 rows"}}
    del eng
    torch.cuda.empty_cache()
    if rank == 0 and not args.no_sweep:
        out["product_sweep"] = product_sweep(torch, SWEEP_SHAPES_STEP, [1, 2, 4, 8, 16], buf_bytes=1.0e9, pk=pk)
    if want_cpu:
        out["cpu_baseline"] = cpu_baseline(pc, W, args, out["tokens_per_step"])
    if rank == 0:
        print(json.dumps(out), flush=True)
    if world > 1:
        torch.distributed.destroy_process_group()


def _attention_share(pc, ctx):
    """Multiply-adds of attention over a context of `ctx` keys as a fraction of one verify pass of 8 rows
    (target layers; the products dominate)."""
    t = pc.target
    macs_attn = 0
    for l in range(t.n_layers):
        keys = min(ctx, t.window) if t.layer_type[l] == gen.SLIDING else ctx
        macs_attn += 8 * t.n_heads * keys * t.head_dim * 2
    return macs_attn


def cpu_baseline(pc, W, args, tokens_per_step):
    """The oracle (C products, one row at a time, OpenMP over output columns) on a bounded sample of the
    same workload: one speculative pass (draft block + 8-row verify) of the E4B pair after a 4-token
    prefix (a 1024-token prefill costs the oracle about ten minutes); tokens/s = the GPU run's tokens per
    pass / the oracle's time per pass. At 1024 context the oracle's pass adds the attention over 1024
    keys, stated as `attention_share_1024`; its products are the same. Also the tiny pair's pass on one
    thread."""
    import oracle
    oracle.build()
    nthreads = oracle.threads()
    pair = oracle.Pair(pc, W)
    prompt = gen.prompt(pc.target.vocab, 4)
    first, _ = pair.prefill(prompt, oracle.Sampler())
    t0 = time.time()
    pair.sync_draft()
    dp, _ = pair.draft.block(first, W["emb"], W["head"])
    pair.verify([first] + [int(v) for v in dp], oracle.Sampler())
    dt = time.time() - t0
    t = pc.target
    weight_macs = 8 * sum(t.hidden * ((t.n_heads + (2 * t.kv_heads[l] if t.is_owner(l) else 0)) * t.head_dim)
                          + t.n_heads * t.head_dim * t.hidden + t.hidden * 3 * t.ffn[l] + 2 * t.hidden * t.ple_dim
                          for l in range(t.n_layers)) + 8 * t.hidden * t.vocab
    share = _attention_share(pc, args.ctx) / weight_macs
    # the tiny pair, one speculative pass on one thread
    tiny = gen.tiny_pair()
    Wt = gen.generate(tiny)
    oracle.set_threads(1)
    try:
        tp = oracle.Pair(tiny, Wt)
        f1, _ = tp.prefill(gen.prompt(tiny.target.vocab, 32), oracle.Sampler())
        t1 = time.time()
        tp.sync_draft()
        dp1, _ = tp.draft.block(f1, Wt["emb"], Wt["head"])
        tp.verify([f1] + [int(v) for v in dp1], oracle.Sampler())
        dt1 = time.time() - t1
    finally:
        oracle.set_threads(nthreads)
    return {"value": round(tokens_per_step / dt, 4), "unit": "tokens/s", "cores": nthreads,
            "threads": f"{nthreads} threads of {os.cpu_count()}", "kind": "oracle",
            "sample": "one speculative pass (draft block + 8-row verify) of the E4B pair at a 4-token context, "
                      "scaled by the GPU run's tokens per pass",
            "seconds_per_pass": round(dt, 2), "attention_share_1024": round(share, 4),
            "tiny_pair_one_thread": {"seconds_per_pass": round(dt1, 3), "threads": 1,
                                   "sample": "tiny pair, one speculative pass after a 32-token prompt"}}


REFERENCE_BUDGET_S = 120.0   # seconds of timed oracle passes in the reference arm


def bench_reference(args):
    """The oracle as the reference arm, on the machine's host cores: K timed speculative passes (draft block
    + 8-row verify + commit) of the E4B pair on a bounded sample of the workload (4-token context: a
    1024-token prefill alone costs the oracle about ten minutes; its passes at 1024 context add only the
    attention over 1024 keys, `attention_share_1024` of the products' multiply-adds).
    A pass costs the oracle the same whatever the proposals, so tokens/s = the planted stream's expected
    tokens per pass at corruption p, 1 + sum_{i=1..7} (1-p)^i, over the measured time per pass."""
    rank = int(os.environ.get("RANK", "0"))
    if rank != 0:
        return
    import oracle
    oracle.build()
    pc, cfgdesc = e4b_workload(args)
    W = gen.generate(pc, workers=min(16, os.cpu_count() or 1))
    pair = oracle.Pair(pc, W)
    sm = oracle.Sampler()
    first, _ = pair.prefill(gen.prompt(pc.target.vocab, 4), sm)
    last = first

    def one_pass():
        nonlocal last
        t0 = time.time()
        pair.sync_draft()
        dp, _ = pair.draft.block(last, W["emb"], W["head"])
        tt, _, _ = pair.verify([last] + [int(v) for v in dp], sm)
        a = oracle.accept_length([int(v) for v in dp], tt[:-1])
        pair.target.commit(a + 1)
        last = tt[a]
        return time.time() - t0

    # a pass costs the oracle seconds: at most two warm-up passes, and the timed passes stop at K or
    # once REFERENCE_BUDGET_S of them have run, so any --steps finishes within a few minutes
    warm = min(args.warmup, 2)
    for _ in range(warm):
        one_pass()
    timed, t_timed = 0, 0.0
    while timed < args.steps and (timed == 0 or t_timed < REFERENCE_BUDGET_S):
        t_timed += one_pass()
        timed += 1
    per_pass = 1.0 + sum((1.0 - args.p) ** i for i in range(1, pc.draft.block))
    value = per_pass * timed / t_timed
    nthreads = oracle.threads()
    out = {"impl": "reference", "metric": METRIC, "value": round(value, 4), "unit": "tokens/s", "n_gpus": 1,
           "steps": args.steps, "warmup": args.warmup, "steps_timed": timed, "warmup_run": warm,
           "ms_per_step": round(1e3 * t_timed / timed, 2),
           "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "fp64 arithmetic, fp32 storage",
           "data": "synthetic", "config": dict(cfgdesc, sample="4-token context"),
           "cpu_baseline": {"value": round(value, 4), "unit": "tokens/s", "cores": nthreads,
                            "threads": f"{nthreads} threads of {os.cpu_count()}", "kind": "oracle",
                            "sample": f"{timed} timed speculative passes (of {args.steps} requested; at most "
                                      f"{REFERENCE_BUDGET_S:.0f} s of passes) of the E4B pair at a 4-token context, "
                                      f"{per_pass:.3f} tokens per pass (planted p={args.p})"},
           "e2e": {"value": round(value, 4), "unit": "tokens/s", "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0}}
    print(json.dumps(out), flush=True)


# The isolated product sweep: K x N shapes of the step's Q4_1 products and the bf16 head.
SWEEP_SHAPES = [("q41", 2560, 10240), ("q41", 10240, 2560), ("q41", 2560, 4096), ("q41", 2560, 20480),
                ("q41", 20480, 2560), ("q41", 2560, 40960), ("q41", 3072, 2560), ("q41", 2560, 3584),
                ("bf16_head", 2560, 262144)]
SWEEP_SHAPES_STEP = [("q41", 2560, 10240), ("q41", 10240, 2560), ("q41", 2560, 4096), ("bf16_head", 2560, 262144)]


def product_sweep(torch, shapes, rows, buf_bytes, pk, reps=100):
    """Graph-timed back-to-back launches per (shape, M): weight images cycled so that every launch reads
    its weights from HBM (at least buf_bytes of images, or 2 images of the head); activations N(0,1)
    rounded to bf16, packed once (resident). GB/s = (weight bytes + M*K*4 + M*N*4) / time per launch."""
    import ctypes
    from dflash_speculative_decode_gb300 import _abi
    L = _abi.lib()
    dev = torch.device("cuda:0")
    st = torch.cuda.current_stream()
    vp = ctypes.c_void_p
    res = []
    for kind, K, N in shapes:
        q41 = kind == "q41"
        wb = K * N * (0.625 if q41 else 2.0)
        nbuf = max(2, min(100, int(buf_bytes // wb) + 1))
        spec = gen.TensorSpec("sweep", "q41" if q41 else "bf16", (N, K), 0.02)
        src = torch.from_numpy(gen.make_tensor(spec, seed=5).reshape(-1).view(np.uint8)).to(dev)
        imgs = []
        for _ in range(nbuf):
            if q41:
                img = torch.empty(L.dfl_q41_image_bytes(K, N), dtype=torch.uint8, device=dev)
                L.dfl_q41_pack(vp(src.data_ptr()), K, N, vp(img.data_ptr()), vp(st.cuda_stream))
            else:
                img = torch.empty(L.dfl_bf16_image_bytes(K, N), dtype=torch.uint8, device=dev)
                L.dfl_bf16_pack(vp(src.data_ptr()), K, N, vp(img.data_ptr()), vp(st.cuda_stream))
            imgs.append(img)
        del src
        for M in rows:
            xb = gen.activations(M, K, seed=M)
            x = torch.from_numpy((xb.astype(np.uint32) << 16).view(np.float32)).to(dev)   # bf16 values as fp32
            act = torch.empty(L.dfl_act_bytes(M, K), dtype=torch.uint8, device=dev)
            L.dfl_act_pack(vp(x.data_ptr()), M, K, vp(act.data_ptr()), vp(st.cuda_stream))
            if q41:
                y = torch.empty((M, N), dtype=torch.float32, device=dev)
                sb = L.dfl_q41_gemm_scratch_bytes(K, N, M)
            else:
                y = torch.empty(M, dtype=torch.int32, device=dev)
                sb = L.dfl_bf16_head_scratch_bytes(K, N, M)
            scratch = torch.zeros(max(sb, 256), dtype=torch.uint8, device=dev)

            def once(i, s):
                if q41:
                    L.dfl_q41_gemm(vp(imgs[i % nbuf].data_ptr()), K, N, vp(act.data_ptr()), M, vp(y.data_ptr()),
                                   vp(scratch.data_ptr()), sb, vp(s))
                else:
                    L.dfl_bf16_head_argmax(vp(imgs[i % nbuf].data_ptr()), K, N, vp(act.data_ptr()), M,
                                           vp(y.data_ptr()), None, vp(scratch.data_ptr()), sb, vp(s))
            for i in range(3):
                once(i, st.cuda_stream)
            n_rep = reps if q41 else 10
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                cs = torch.cuda.current_stream().cuda_stream
                for i in range(n_rep):
                    once(i, cs)
            g.replay()
            torch.cuda.synchronize()
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record(st)
            g.replay()
            e1.record(st)
            torch.cuda.synchronize()
            us = e0.elapsed_time(e1) * 1e3 / n_rep
            by = wb + M * K * 4 + M * N * 4 * (1 if q41 else 0)
            gbs = by / (us * 1e-6) / 1e9
            res.append({"kind": kind, "K": K, "N": N, "M": M, "us": round(us, 2), "GB/s": round(gbs, 1),
                        "frac_measured": round(gbs / pk["hbm_gbs"], 3), "frac_8TBs": round(gbs / 8000, 3)})
            del g
        del imgs
        torch.cuda.empty_cache()
    return res


# The Q4_1 product at many rows (prompt ingest) on the tcgen05 tensor cores: E4B and 27B-class shapes.
PREFILL_SHAPES = [(2560, 10240), (10240, 2560), (2560, 4096), (5376, 43008), (21504, 5376)]


def prefill_sweep(torch, shapes, rows, pk, reps=10):
    """dfl_q41_gemm_tc per (shape, M), event-timed over `reps` back-to-back calls after 3 warm-up calls.
    A call is three kernels: weight expansion to bf16 hi/lo, row split, the tcgen05 product. TFLOP/s
    counts the product's 2 M N K; the tensor cores run three bf16 products for it (hi*hi, hi*lo,
    lo*hi), reported against the measured dense bf16 peak as `tensor_frac`."""
    import ctypes
    from dflash_speculative_decode_gb300 import _abi
    L = _abi.lib()
    dev = torch.device("cuda:0")
    st = torch.cuda.current_stream()
    vp = ctypes.c_void_p
    res = []
    for K, N in shapes:
        spec = gen.TensorSpec("sweep", "q41", (N, K), 0.02)
        src = torch.from_numpy(gen.make_tensor(spec, seed=5).reshape(-1).view(np.uint8)).to(dev)
        img = torch.empty(L.dfl_q41_image_bytes(K, N), dtype=torch.uint8, device=dev)
        L.dfl_q41_pack(vp(src.data_ptr()), K, N, vp(img.data_ptr()), vp(st.cuda_stream))
        del src
        for M in rows:
            x = torch.randn((M, K), generator=torch.Generator(device=dev).manual_seed(M), device=dev)
            y = torch.empty((M, N), dtype=torch.float32, device=dev)
            sb = L.dfl_q41_gemm_tc_scratch_bytes(K, N, M)
            scratch = torch.zeros(sb + 1024, dtype=torch.uint8, device=dev)
            base = (scratch.data_ptr() + 1023) // 1024 * 1024

            def once():
                rc = L.dfl_q41_gemm_tc(vp(img.data_ptr()), K, N, vp(x.data_ptr()), M, vp(y.data_ptr()), vp(base),
                                       sb, vp(st.cuda_stream))
                assert rc == 0, rc
            for _ in range(3):
                once()
            torch.cuda.synchronize()
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record(st)
            for _ in range(reps):
                once()
            e1.record(st)
            torch.cuda.synchronize()
            assert L.dfl_q41_gemm_status(vp(base), vp(st.cuda_stream)) == 0
            us = e0.elapsed_time(e1) * 1e3 / reps
            tf = 2.0 * M * N * K / (us * 1e-6) / 1e12
            res.append({"K": K, "N": N, "M": M, "us": round(us, 1), "TFLOP/s": round(tf, 1),
                        "tensor_frac": round(3 * tf / pk["bf16_tflops"], 3),
                        })
            del scratch, x, y
        del img
        torch.cuda.empty_cache()
    return res


def bench_prefill(args):
    """The large-M product on its own (prompt-ingest shapes), one JSON line."""
    import torch
    from dflash_speculative_decode_gb300 import build
    build.build()
    pk = peaks()
    shapes = PREFILL_SHAPES
    if args.gemm_shape:
        shapes = [tuple(int(v) for v in args.gemm_shape.split("x"))]
    rows = [int(v) for v in args.sweep_rows.split(",")]
    res = prefill_sweep(torch, shapes, rows, pk)
    print(json.dumps({"workload": "Q4_1 product at many rows (tcgen05), prompt-ingest shapes",
                      "peak_bf16_tflops": pk["bf16_tflops"], "results": res}), flush=True)


def bench_attn(args):
    """Profiling workload for the attention kernel: a short E4B-shaped target (six layers, no KV sharing,
    vocab 32768) or two 27B-class layers, each with its full 5-layer draft, a prompt of --ctx tokens
    through long prefill passes, then two speculative steps. Prints one JSON line (not a bench line)
    with the attention launches per pass, so a profiler can skip the prompt's."""
    import dataclasses
    import torch
    from dflash_speculative_decode_gb300 import build
    build.build()
    if args.attn_pair == "27b":
        pc = gen.b27_cut(max_ctx=args.ctx + 64, n_layers=2, vocab=32768)
    else:
        t = gen.e4b_target(n_layers=6, first_shared=6, vocab=32768)
        d = dataclasses.replace(gen.e4b_draft(vocab=32768), taps=(1, 3, 5))
        pc = gen.PairConfig(t, d, max_ctx=args.ctx + 64)
    eng, _, _ = load_engine(pc, prefill_rows=1024)
    tok = eng.dfl_prefill(gen.prompt(pc.target.vocab, args.ctx))
    for _ in range(2):
        props = eng.dfl_draft_block(tok)
        tt, a = eng.dfl_verify_block([tok] + [int(v) for v in props])
        eng.dfl_commit_verify_rows(a + 1)
        tok = int(tt[a])
    torch.cuda.synchronize()
    long_passes = (args.ctx // 1024) + (1 if args.ctx % 1024 >= 128 else 0)
    print(json.dumps({"workload": f"attention profile, {args.attn_pair} layers, prompt {args.ctx}",
                      "positions": eng.dfl_positions_held(),
                      "prompt_attention_launches": long_passes * pc.target.n_layers,
                      "attention_launches_per_step": pc.target.n_layers + pc.draft.n_layers}), flush=True)


def _sampled_spec(eng, table, first, n_gen, temperature, seed):
    """Speculative decode from the current state until n_gen tokens: draft block, planted proposals from
    the device table, sampled verify of the block, commit of the accepted rows. Returns the tokens and
    the passes."""
    from dflash_speculative_decode_gb300 import DFL_KEEP_ACCEPTED
    B = eng.cfg.block
    out, last, passes = [first], first, 0
    while len(out) < n_gen:
        eng.dfl_draft_block(last, want=False)
        eng.dfl_plant_proposals(table)
        tt, a = eng.dfl_verify_block(None, k=B, temperature=temperature, seed=seed)
        eng.dfl_commit_verify_rows(DFL_KEEP_ACCEPTED)
        out += [int(v) for v in tt[:a + 1]]
        last = int(tt[a])
        passes += 1
    return out, passes


def bench_long(args):
    """Long-context sampled serving of the E4B pair, at each context of --long-ctx: a prefix of --prefix
    tokens is prefilled once and pinned as a device snapshot; requests A, B, A each restore the pin,
    prefill their own prompt up to the context, and decode --gen tokens speculatively at temperature
    --temperature with planted drafts (corruption p). Before each timed decode a plain sampled decode of
    the same request (untimed) gives the target's own tokens; they plant the drafts, and the speculative
    tokens must equal them exactly, since sampling is keyed by seed and absolute position and a row's
    logits do not depend on the rows verified beside it. A's two runs must give the same tokens
    (FastFlowLM PR #899 "gemma4e-dflash-flash", "Changes": the pinned prefix is restored, never
    overwritten). With --kv8 the full layers' planes are held in 8 bits and prompts are ingested in passes
    of 16 rows; a position's logits then depend on how its passes were cut, so the plain and the speculative
    tokens may part. Prints one JSON line (not the bench line)."""
    import torch
    from dflash_speculative_decode_gb300 import build
    build.build()
    T = args.temperature
    if args.kv8:
        args.prefill_rows = 0
    requests = [("A", 1, 11), ("B", 2, 12), ("A", 1, 11)]   # (name, prompt request id, sampling seed)
    clk = Clocks(0)
    clk.start()
    t_first = None
    results = []
    for ctx in [int(v) for v in args.long_ctx.split(",")]:
        if ctx <= args.prefix + 16:
            raise SystemExit(f"--long-ctx {ctx} must exceed --prefix {args.prefix} + 16")
        pc = gen.e4b_pair(max_ctx=ctx + args.gen + 64)
        eng, _, t_load = load_engine(pc, prefill_rows=args.prefill_rows, kv8=int(args.kv8))
        V, L = pc.target.vocab, pc.max_ctx + 32
        prefix = gen.prompt(V, args.prefix, request=100)
        empty = eng.dfl_snapshot()
        # warm-up: the prefix's passes, plain and speculative sampled passes (graphs, kernel attributes)
        t = eng.dfl_prefill(prefix, T, 1)
        eng.dfl_verify_block([t], temperature=T, seed=1)
        eng.dfl_commit_verify_rows(1)
        warm = torch.zeros(L, dtype=torch.int32, device="cuda")
        _sampled_spec(eng, warm, t, 12, T, 1)
        eng.dfl_restore(empty)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        eng.dfl_prefill(prefix, T, 1)
        torch.cuda.synchronize()
        t_prefix = time.perf_counter() - t0
        t0 = time.perf_counter()
        pin = eng.dfl_snapshot()
        torch.cuda.synchronize()
        t_snap = time.perf_counter() - t0
        reqs, tot_tok, tot_ms, tot_pass = [], 0, 0.0, 0
        for name, rid, seed in requests:
            torch.cuda.synchronize()
            t0 = time.perf_counter()
            eng.dfl_restore(pin)
            torch.cuda.synchronize()
            t_restore = time.perf_counter() - t0
            prompt = gen.prompt(V, ctx - args.prefix, request=rid)
            t0 = time.perf_counter()
            first = eng.dfl_prefill(prompt, T, seed)
            torch.cuda.synchronize()
            t_pf = time.perf_counter() - t0
            n0 = eng.dfl_positions_held()
            after_prompt = eng.dfl_snapshot()
            plain = [first]                                  # the target's own sampled tokens (untimed)
            while len(plain) < args.gen:
                tt, _ = eng.dfl_verify_block([plain[-1]], temperature=T, seed=seed)
                eng.dfl_commit_verify_rows(1)
                plain.append(int(tt[0]))
            G = np.zeros(L, np.int32)
            G[n0:n0 + len(plain)] = plain
            table = torch.from_numpy(gen.corruption(args.p, V, L, request=rid).propose(G, np.arange(L))).cuda()
            eng.dfl_restore(after_prompt)
            torch.cuda.synchronize()
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            tw = time.time()
            t_first = t_first or tw
            e0.record()
            out, passes = _sampled_spec(eng, table, first, args.gen, T, seed)
            e1.record()
            torch.cuda.synchronize()
            clk.window(t_first, time.time())
            ms = e0.elapsed_time(e1)
            emitted = len(out) - 1                            # the first token came from the prefill
            tot_tok, tot_ms, tot_pass = tot_tok + emitted, tot_ms + ms, tot_pass + passes
            reqs.append({"request": name, "seed": seed, "positions_before_decode": n0,
                         "prefill_s": round(t_pf, 4), "prefill_tokens_per_s": round((ctx - args.prefix) / t_pf, 1),
                         "restore_ms": round(t_restore * 1e3, 3), "decode_ms": round(ms, 3),
                         "tokens_per_s": round(emitted / (ms / 1e3), 2), "passes": passes,
                         "tokens_per_pass": round(emitted / passes, 3),
                         "spec_equals_plain": out[:args.gen] == plain[:args.gen], "tokens": out[:args.gen]})
        a_repeat = reqs[0]["tokens"] == reqs[2]["tokens"]
        for r in reqs:
            del r["tokens"]
        results.append({"context": ctx, "tokens_per_s": round(tot_tok / (tot_ms / 1e3), 2),
                        "ms_per_pass": round(tot_ms / tot_pass, 4), "tokens_per_pass": round(tot_tok / tot_pass, 3),
                        "prefix_prefill_s": round(t_prefix, 4), "snapshot_bytes": int(pin.numel()),
                        "snapshot_ms": round(t_snap * 1e3, 3), "load_s": round(t_load, 1),
                        "a_repeats_exactly": a_repeat,
                        "spec_equals_plain": all(r["spec_equals_plain"] for r in reqs), "requests": reqs})
        del eng, pin, empty, after_prompt, table, warm
        torch.cuda.empty_cache()
    clocks = clk.stop()
    print(json.dumps({"workload": "long-context sampled serving, e4b pair, pinned prefix, requests A, B, A",
                      "metric": "decode tokens/s (device-timed speculative passes, prefill excluded)",
                      "temperature": T, "prefix": args.prefix, "generated_per_request": args.gen,
                      "corruption_p": args.p, "block": 8, "prefill_rows": args.prefill_rows, "kv8": bool(args.kv8),
                      "dtype": "fp32 activations, Q4_1/bf16 weights",
                      "data": "synthetic (seeded random-init weights of the E4B-shaped pair, uniform prompts)",
                      "results": results, "clocks": clocks}), flush=True)


def draft_block_bytes(pc, ctx):
    """Algorithmic bytes of one draft block: the draft layers' Q4_1 images (0.625 bytes per weight), the
    shared bf16 head once, and the context keys and values the block's attention reads (fp32 planes,
    at most the draft's window of rows)."""
    d, H = pc.draft, pc.target.hidden
    per_layer = (H * (d.n_heads + 2 * d.n_kv_heads) * d.head_dim + d.n_heads * d.head_dim * H
                 + H * 2 * d.ffn + d.ffn * H)
    rows = min(ctx, d.window) if d.window > 0 else ctx
    kv = d.n_layers * rows * 2 * d.n_kv_heads * d.head_dim * 4
    return d.n_layers * per_layer * 0.625 + pc.target.vocab * H * 2 + kv


def bench_draft(args):
    """The E4B draft on its own: its context made of --draft-ctx rows of N(0, 1) taps (not timed), then
    --steps seeded blocks (8 rows: the last token and 7 mask tokens at the next positions; 5 layers;
    proposals from the shared head) timed back to back with device events. Each block reads the
    draft's weights and the 1.34 GB head once, so no L2 flush is needed. Prints one JSON line (not the
    bench line)."""
    import torch
    from dflash_speculative_decode_gb300 import build
    build.build()
    pk = peaks()
    ctxs = [int(v) for v in args.draft_ctx.split(",")]
    pc = gen.e4b_pair(max_ctx=max(ctxs) + 64)
    eng, _, t_load = load_engine(pc)
    taps = torch.from_numpy(gen.fc_taps(max(ctxs), len(pc.draft.taps) * pc.target.hidden)).cuda()
    toks = [int(v) for v in gen.prompt(pc.target.vocab, args.steps + args.warmup, request=7)]
    clk = Clocks(0)
    clk.start()
    t_first, have, res = None, 0, []
    for ctx in ctxs:
        eng.dfl_draft_append_taps(taps[have:ctx])
        have = ctx
        for t in toks[:args.warmup]:
            eng.dfl_draft_block(t, want=False)
        torch.cuda.synchronize()
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        tw = time.time()
        t_first = t_first or tw
        l0 = eng.dfl_launch_count()
        e0.record()
        for t in toks[args.warmup:]:
            eng.dfl_draft_block(t, want=False)
        e1.record()
        torch.cuda.synchronize()
        clk.window(t_first, time.time())
        us = e0.elapsed_time(e1) * 1e3 / args.steps
        by = draft_block_bytes(pc, ctx)
        res.append({"context": ctx, "us_per_block": round(us, 2), "blocks_per_s": round(1e6 / us, 1),
                    "launches_per_block": round((eng.dfl_launch_count() - l0) / args.steps, 1),
                    "algorithmic_bytes_per_block": int(by), "GB/s": round(by / us / 1e3, 1),
                    "frac_measured": round(by / us / 1e3 / pk["hbm_gbs"], 4), "frac_8TBs": round(by / us / 8e6, 4)})
    clocks = clk.stop()
    print(json.dumps({"workload": "E4B draft alone (5 layers, window 1024, shared head 2560 x 262144), "
                                  "context from N(0, 1) taps", "blocks_timed": args.steps, "warmup": args.warmup,
                      "peak_gbs": pk["hbm_gbs"], "peak_source": pk["src"], "load_s": round(t_load, 1),
                      "dtype": "fp32 activations, Q4_1/bf16 weights", "data": "synthetic",
                      "results": res, "clocks": clocks}), flush=True)


def bench_gemm(args):
    """The isolated product sweep on its own: every shape of SWEEP_SHAPES (or --gemm-shape), rows --gemm-rows."""
    import torch
    from dflash_speculative_decode_gb300 import build
    build.build()
    pk = peaks()
    shapes = SWEEP_SHAPES
    if args.gemm_shape:
        shapes = [("q41",) + tuple(int(v) for v in args.gemm_shape.split("x"))]
    rows = [int(v) for v in args.gemm_rows.split(",")]
    res = product_sweep(torch, shapes, rows, buf_bytes=args.gemm_bufs * 1e8, pk=pk)
    print(json.dumps({"workload": "isolated Q4_1 product sweep and the bf16 head", "peak_gbs": pk["hbm_gbs"],
                      "results": res}), flush=True)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=300)
    ap.add_argument("--warmup", type=int, default=10)
    ap.add_argument("--impl", default="cuda", choices=["cuda", "reference"])
    ap.add_argument("--workload", default="e4b", choices=["e4b", "gemm", "cut", "27b", "prefill", "attn", "long", "draft"])
    ap.add_argument("--attn-pair", default="e4b", choices=["e4b", "27b"], help="layers of --workload attn")
    ap.add_argument("--prefill-rows", type=int, default=1024,
                    help="rows per long prefill pass (tcgen05 products); 0 = passes of 16 rows")
    ap.add_argument("--sweep-rows", default="128,256,512,1024,2048", help="row counts of the prefill product sweep")
    ap.add_argument("--ctx", type=int, default=1024)
    ap.add_argument("--p", type=float, default=0.3)
    ap.add_argument("--gen", type=int, default=512, help="tokens per decode before restarting from the prefix")
    ap.add_argument("--gemm-bufs", type=int, default=40, help="sweep: cycle at least this many x 100 MB of images")
    ap.add_argument("--gemm-shape", default="", help="one KxN shape for the product sweep")
    ap.add_argument("--gemm-rows", default="1,2,4,8,16", help="row counts of the product sweep")
    ap.add_argument("--long-ctx", default="4096,16384", help="contexts of --workload long")
    ap.add_argument("--prefix", type=int, default=512, help="pinned prefix tokens of --workload long")
    ap.add_argument("--temperature", type=float, default=0.8, help="sampling temperature of --workload long")
    ap.add_argument("--kv8", action="store_true", help="--workload long with the full layers' planes in 8 bits")
    ap.add_argument("--draft-ctx", default="30,1024,4096", help="contexts of --workload draft")
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--no-sweep", action="store_true", help="leave the product sweep out of the bench line")
    args = ap.parse_args()
    if args.impl == "reference":
        return bench_reference(args)
    if args.workload == "gemm":
        return bench_gemm(args)
    if args.workload == "prefill":
        return bench_prefill(args)
    if args.workload == "attn":
        return bench_attn(args)
    if args.workload == "long":
        return bench_long(args)
    if args.workload == "draft":
        return bench_draft(args)
    return bench_cuda(args)


if __name__ == "__main__":
    main()
