#!/usr/bin/env python
"""Benchmark of exact attention on GB300: one step = the whole hot path
(forward: O and LSE; backward: dQ, dK, dV) over one batch of the largest
single-GPU workload, causal grouped-query attention B=1, Hq=32, Hkv=8,
Nq=Nk=16384, d=128, bf16, Q and K ~ N(0, 2^2), V and dO ~ N(0, 1), seeded
synthetic inputs resident in HBM.

Prints ONE JSON line on rank 0. `value` is TFLOP/s over all ranks (forward
4*B*Hq*N*N*d/2 plus backward 2.5x that, per step), timed on the device with
CUDA events over K steps with the L2 flushed (a 256 MB write) before every
step. Extra keys: `roofline` for the dominant kernel, `cpu_baseline` (the
fp64 oracle on bounded samples on the host cores, for this workload and for
every published one), `e2e` (the same metric through the public API with
pinned host buffers, copies included, beside the measured copy bandwidth),
`clocks` sampled during the timed region, `gpu_launches`, and `configs`
with kernel TFLOP/s of every published workload.

--impl reference times the fp64 CPU oracle on the same workload (a bounded
sample per step) and prints the same kind of line with "impl": "reference".
Multi-GPU (torchrun): every rank runs the same per-GPU workload (weak
scaling, no collective in the data path); the timing is the max over ranks.
"""
from __future__ import annotations

import argparse
import ctypes
import glob
import hashlib
import json
import math
import os
import statistics
import subprocess
import sys
import threading
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

import workloads  # noqa: E402

MAIN = workloads.BY_NAME["fwd_causal_gqa_b1_hq32_hkv8_n16384_d128"]
METRIC = "attention fwd/bwd TFLOP/s at 1 GB300 and fraction of dense BF16 tensor peak"
FLUSH_BYTES = 256 << 20
KERNEL_SOURCES = {"fa_fwd_kernel": ("fa_fwd.cu", "fa_fwd_pipeline.cuh"),
                  "bwd_main_kernel": ("fa_bwd.cu", "fa_bwd_layout.h"),
                  "fa_fwd8_kernel": ("fa_fwd8.cu", "fa_fwd_pipeline.cuh"),
                  "fa_fwd_pair_kernel": ("fa_fwd.cu", "fa_fwd_pipeline.cuh"),
                  "seq_fwd_kernel": ("fa_seq_fwd.cu", "fa_seq_plan.cuh", "fa_seq.cuh"),
                  "seq_bwd_kernel": ("fa_seq_bwd.cu", "fa_seq_plan.cuh", "fa_seq.cuh", "fa_bwd_layout.h")}
# profiling targets of the packed calls: causal sequences one behind the other
PACKED_CASES = {"packed_causal_b1_hq32_hkv8_n16384_d128": dict(lens=[16384], Hq=32, Hkv=8, d=128, seed=1050),
                "packed_causal_b1_hq32_hkv8_n16384_d64": dict(lens=[16384], Hq=32, Hkv=8, d=64, seed=1051),
                "packed_causal_b2_hq32_hkv8_n4096_d128": dict(lens=[4096, 4096], Hq=32, Hkv=8, d=128, seed=1052)}
PANEL = 1024  # query rows of one oracle sample


def step_flops(w) -> float:
    return w.fwd_flops() + w.bwd_flops()


def max_over_ranks(value: float) -> float:
    """Largest `value` over all ranks (the job is as slow as its slowest rank).
    Uses the process group's own device: CUDA for nccl, CPU for gloo."""
    import torch
    import torch.distributed as dist
    if not (dist.is_available() and dist.is_initialized()) or dist.get_world_size() == 1:
        return float(value)
    dev = "cuda" if dist.get_backend() == "nccl" else "cpu"
    t = torch.tensor([float(value)], dtype=torch.float64, device=dev)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    return float(t.item())


def job_tflops(world: int, steps: int, flops_per_step: float, total_ms: float) -> float:
    """Whole-job throughput: every rank runs `steps` steps of the same per-GPU
    workload (weak scaling), and the job takes `total_ms` (max over ranks)."""
    return world * steps * flops_per_step / (total_ms * 1e-3) / 1e12


def dist_env():
    rank = int(os.environ.get("RANK", "0"))
    world = int(os.environ.get("WORLD_SIZE", "1"))
    local = int(os.environ.get("LOCAL_RANK", "0"))
    return rank, world, local


def load_peaks():
    """(burst, sustained, source) dense bf16 peaks in TFLOP/s."""
    path = os.path.join(ROOT, "MEASURED_PEAKS.json")
    if os.path.exists(path):
        with open(path) as f:
            p = json.load(f)
        return (float(p["bf16_tflops"]), float(p.get("bf16_tflops_sustained", p["bf16_tflops"])),
                "measured (MEASURED_PEAKS.json: bf16_tflops burst, bf16_tflops_sustained)")
    return 1900.0, 1700.0, "fallback (1.9 PFLOP/s burst, 1.7 sustained, an earlier GB300 measurement)"


def source_sha(kernel: str) -> str:
    h = hashlib.sha256()
    for name in KERNEL_SOURCES[kernel]:
        with open(os.path.join(ROOT, "exact_attention_99_gb300", "csrc", name), "rb") as f:
            h.update(f.read())
    return h.hexdigest()[:16]


def profiled_traffic(kernel: str, workload: str):
    """dram bytes per launch from a committed ncu summary, if that summary was
    taken on the current source of the kernel; else None."""
    for path in glob.glob(os.path.join(ROOT, "profiles", "*.md")):
        fields = {}
        with open(path) as f:
            for line in f:
                if ":" in line and line.startswith("- "):
                    k, v = line[2:].split(":", 1)
                    fields[k.strip()] = v.strip().strip("`")
        if fields.get("kernel") == kernel and fields.get("workload") == workload:
            if fields.get("source_sha256") == source_sha(kernel) and "dram_bytes_per_launch" in fields:
                return int(float(fields["dram_bytes_per_launch"]))
    return None


class ClockSampler:
    """SM clock, power and clock-event reasons of one GPU, sampled every 5 ms
    through NVML (read-only queries) in a background thread; only the samples
    taken inside the timed window (mark_begin / mark_end) are summarised.
    Falls back to `nvidia-smi -lms 50` when NVML cannot be loaded."""
    REASONS = {0x8: "hw_slowdown", 0x40: "hw_thermal_slowdown", 0x20: "sw_thermal_slowdown", 0x4: "sw_power_cap",
               0x80: "hw_power_brake_slowdown"}

    def __init__(self, torch_device: int):
        self.torch_device = torch_device
        self.samples = []  # (time, sm_mhz, max_mhz, power_w, reasons bitmask)
        self.t_begin = self.t_end = None
        self.stop_flag = threading.Event()
        self.thread = None
        self.kind = None
        self.proc = None

    def _nvml_handle(self):
        import torch
        nv = ctypes.CDLL("libnvidia-ml.so.1")
        if nv.nvmlInit_v2() != 0:
            raise OSError("nvmlInit failed")
        h = ctypes.c_void_p()
        props = torch.cuda.get_device_properties(self.torch_device)
        bus = getattr(props, "pci_bus_id", None)
        if bus is not None:
            busid = f"{getattr(props, 'pci_domain_id', 0):08X}:{bus:02X}:{getattr(props, 'pci_device_id', 0):02X}.0"
            if nv.nvmlDeviceGetHandleByPciBusId_v2(busid.encode(), ctypes.byref(h)) == 0:
                return nv, h
        vis = os.environ.get("CUDA_VISIBLE_DEVICES", "")
        idx = int(vis.split(",")[self.torch_device]) if vis and vis.split(",")[0].isdigit() else self.torch_device
        if nv.nvmlDeviceGetHandleByIndex_v2(ctypes.c_uint(idx), ctypes.byref(h)) != 0:
            raise OSError("no NVML handle")
        return nv, h

    def start(self):
        try:
            nv, h = self._nvml_handle()
            reasons_fn = getattr(nv, "nvmlDeviceGetCurrentClocksEventReasons", None) or \
                nv.nvmlDeviceGetCurrentClocksThrottleReasons
            self.kind = "nvml, 5 ms"
            self.thread = threading.Thread(target=self._nvml_loop, args=(nv, h, reasons_fn), daemon=True)
            self.thread.start()
            return
        except (OSError, AttributeError):
            pass
        try:
            fields = ("timestamp,clocks.sm,clocks.max.sm,power.draw,clocks_event_reasons.hw_slowdown,"
                      "clocks_event_reasons.hw_thermal_slowdown,clocks_event_reasons.sw_thermal_slowdown,"
                      "clocks_event_reasons.sw_power_cap")
            self.proc = subprocess.Popen(["nvidia-smi", f"--query-gpu={fields}", "--format=csv,noheader,nounits",
                                          "-lms", "50", "-i", str(self.torch_device)], stdout=subprocess.PIPE,
                                         stderr=subprocess.DEVNULL, text=True)
            self.kind = "nvidia-smi, 50 ms"
            self.thread = threading.Thread(target=self._smi_loop, daemon=True)
            self.thread.start()
        except (OSError, FileNotFoundError):
            self.kind = None

    def _nvml_loop(self, nv, h, reasons_fn):
        clk, mx, pw, rs = ctypes.c_uint(), ctypes.c_uint(), ctypes.c_uint(), ctypes.c_ulonglong()
        while not self.stop_flag.is_set():
            t = time.time()
            if nv.nvmlDeviceGetClockInfo(h, 1, ctypes.byref(clk)) == 0 and \
                    nv.nvmlDeviceGetMaxClockInfo(h, 1, ctypes.byref(mx)) == 0:
                p = pw.value / 1000.0 if nv.nvmlDeviceGetPowerUsage(h, ctypes.byref(pw)) == 0 else float("nan")
                r = rs.value if reasons_fn(h, ctypes.byref(rs)) == 0 else 0
                self.samples.append((t, float(clk.value), float(mx.value), p, r))
            time.sleep(0.005)

    def _smi_loop(self):
        import datetime
        bits = [0x8, 0x40, 0x20, 0x4]
        for line in self.proc.stdout:
            parts = [x.strip() for x in line.split(",")]
            if len(parts) < 8:
                continue
            try:
                ts = datetime.datetime.strptime(parts[0], "%Y/%m/%d %H:%M:%S.%f").timestamp()
                r = sum(b for b, flag in zip(bits, parts[4:8]) if flag.lower().startswith("active"))
                self.samples.append((ts, float(parts[1]), float(parts[2]), float(parts[3]), r))
            except ValueError:
                continue

    def mark_begin(self):
        self.t_begin = time.time()

    def mark_end(self):
        self.t_end = time.time()

    def stop(self):
        if self.kind is None:
            return {"sm_mhz": None, "sm_max_mhz": None, "reasons": ["no clock source"], "samples": 0}
        time.sleep(0.1 if self.proc is None else 0.3)
        self.stop_flag.set()
        if self.proc is not None:
            self.proc.terminate()
            try:
                self.proc.wait(timeout=5)
            except subprocess.TimeoutExpired:
                self.proc.kill()
        if self.thread is not None:
            self.thread.join(timeout=5)
        inside = [s for s in list(self.samples) if self.t_begin <= s[0] <= self.t_end]
        if not inside:
            return {"sm_mhz": None, "sm_max_mhz": None, "reasons": ["no samples in the timed window"], "samples": 0,
                    "source": self.kind}
        reasons = sorted({name for s in inside for bit, name in self.REASONS.items() if s[4] & bit})
        power = [s[3] for s in inside if s[3] == s[3]]
        return {"sm_mhz": statistics.median(s[1] for s in inside), "sm_max_mhz": max(s[2] for s in inside),
                "sm_mhz_min": min(s[1] for s in inside), "reasons": reasons,
                "power_w_median": statistics.median(power) if power else None,
                "power_w_max": max(power) if power else None, "samples": len(inside),
                "window_s": round(self.t_end - self.t_begin, 3), "source": self.kind}


# ---------------------------------------------------------------- oracle legs
def visible_pairs(nq: int, nk: int, causal: bool, rows) -> int:
    """(query, key) pairs visible to the given query rows (bottom-right
    causal alignment: key j visible to row i iff j <= i + nk - nq)."""
    if not causal:
        return len(rows) * nk
    return int(sum(max(0, min(nk, i + nk - nq + 1)) for i in rows))


def oracle_panel(w, x, b: int, h: int, direction: str):
    """One bounded oracle sample of workload w: the last min(PANEL, Nq) query
    rows of (batch b, query head h) against all keys. With the bottom-right
    causal alignment, those rows as a problem of their own (Nq' rows, the
    same Nk keys) see exactly the keys they see in the whole problem, so the
    sample is that part of the workload. direction "fwd": the oracle's
    forward; "fwdbwd": forward and backward. Returns (credited flops,
    seconds): 4*d per visible pair forward, 2.5x that backward."""
    from oracle import attn_ref
    r = min(PANEL, w.Nq)
    kv = h // (w.Hq // w.Hkv)
    q = x["q"][b:b + 1, w.Nq - r:, h:h + 1].double().numpy()
    k = x["k"][b:b + 1, :, kv:kv + 1].double().numpy()
    v = x["v"][b:b + 1, :, kv:kv + 1].double().numpy()
    pairs = visible_pairs(w.Nq, w.Nk, w.causal, range(w.Nq - r, w.Nq))
    t0 = time.perf_counter()
    attn_ref.forward(q, k, v, w.scale, w.causal)
    flops = 4.0 * w.d * pairs
    if direction == "fwdbwd":
        do = x["do"][b:b + 1, w.Nq - r:, h:h + 1].double().numpy()
        attn_ref.backward(q, k, v, do, w.scale, w.causal)
        flops *= 3.5
    return flops, time.perf_counter() - t0


def oracle_sample(w, x, seconds: float, max_panels: int | None = None, first: int = 0, direction="fwdbwd"):
    """Oracle panels (oracle_panel) of successive (batch, head) slices,
    starting at slice `first`, until `seconds` have passed or `max_panels`
    are done. Returns (credited flops, seconds, panels)."""
    heads = [(b, h) for b in range(w.B) for h in range(w.Hq)]
    done, flops, el = 0, 0.0, 0.0
    i = first
    while True:
        b, h = heads[i % len(heads)]
        f, t = oracle_panel(w, x, b, h, direction)
        flops, el, done, i = flops + f, el + t, done + 1, i + 1
        if el >= seconds or (max_panels and done >= max_panels):
            break
    return flops, el, done


def cpu_model() -> str:
    try:
        out = subprocess.run(["lscpu"], capture_output=True, text=True, timeout=10).stdout
        for line in out.splitlines():
            if line.lower().startswith("model name"):
                return line.split(":", 1)[1].strip()
    except (OSError, subprocess.SubprocessError):
        pass
    return "unknown"


def blas_threads() -> int:
    for var in ("OPENBLAS_NUM_THREADS", "OMP_NUM_THREADS", "MKL_NUM_THREADS"):
        if os.environ.get(var):
            return int(os.environ[var])
    return os.cpu_count() or 1


def oracle_per_workload(seconds_each: float = 2.0):
    """The oracle on every published workload (bounded samples: oracle
    panels of successive heads for about `seconds_each`): forward for the
    forward workloads, forward + backward for the backward one."""
    out = {}
    for w in workloads.WORKLOADS:
        x = workloads.workload_inputs(w, with_dout=True)
        direction = "fwdbwd" if w.direction == "bwd" else "fwd"
        f, el, n = oracle_sample(w, x, seconds_each, direction=direction)
        out[w.name] = {"tflops": f / el / 1e12, "seconds": round(el, 2), "direction": direction,
                       "sample": f"{n} panel(s) of the last {min(PANEL, w.Nq)} query rows of one (batch, head)"}
    return out


def oracle_single_thread():
    """The oracle on one host thread (BLAS limited to 1 thread in a fresh
    interpreter) on the first two published workloads: forward panels for
    about 2 s each. Returns {workload: {tflops, seconds, panels}} or {} if
    the child fails."""
    env = dict(os.environ, OPENBLAS_NUM_THREADS="1", OMP_NUM_THREADS="1", MKL_NUM_THREADS="1")
    code = ("import json, bench, workloads\nout = {}\nfor w in workloads.WORKLOADS[:2]:\n"
            "    x = workloads.workload_inputs(w)\n"
            "    f, el, n = bench.oracle_sample(w, x, 2.0, direction='fwd')\n"
            "    out[w.name] = {'tflops': f / el / 1e12, 'seconds': round(el, 2), 'panels': n}\nprint(json.dumps(out))")
    try:
        r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=env, capture_output=True, text=True,
                           timeout=600)
        return json.loads(r.stdout.strip().splitlines()[-1])
    except (subprocess.SubprocessError, ValueError, IndexError):
        return {}


def run_reference(args):
    rank, world, _ = dist_env()
    if rank != 0:
        return
    w = MAIN
    x = workloads.workload_inputs(w, with_dout=True)
    for i in range(args.warmup):
        oracle_panel(w, x, 0, i % w.Hq, "fwdbwd")
    flops, times = 0.0, []
    for i in range(args.steps):
        f, el = oracle_panel(w, x, 0, (args.warmup + i) % w.Hq, "fwdbwd")
        flops += f
        times.append(el)
    total = sum(times)
    value = flops / total / 1e12
    sample = (f"per step: the last {min(PANEL, w.Nq)} query rows of one (batch, head) slice of {w.name} against "
              f"all {w.Nk} keys, fp64 forward + backward (credited flops: 4*d per visible pair, x3.5)")
    line = {
        "impl": "reference", "metric": METRIC, "value": value, "unit": "TFLOP/s", "n_gpus": world,
        "steps": args.steps, "warmup": args.warmup, "ms_per_step": 1e3 * total / args.steps,
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "f64", "data": "synthetic",
        "config": {"workload": w.name, "B": w.B, "Hq": w.Hq, "Hkv": w.Hkv, "Nq": w.Nq, "Nk": w.Nk, "d": w.d,
                   "causal": w.causal, "sigma_qk": w.sigma_qk, "step": "fwd+bwd of a bounded sample"},
        "cpu_baseline": {"value": value, "unit": "TFLOP/s", "cores": blas_threads(), "kind": "oracle",
                         "sample": sample, "cpu_model": cpu_model()},
        "e2e": {"value": value, "unit": "TFLOP/s", "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0},
    }
    print(json.dumps(line), flush=True)


# ------------------------------------------------------------------ GPU legs
def time_one(fn, flush, reps=20, warm=3, stats=None):
    """Median device time (ms) of `reps` calls after `warm` untimed ones, the
    L2 flushed before each; `stats` (a dict) also receives the minimum."""
    import torch
    for _ in range(warm):
        fn()
    ts = []
    for _ in range(reps):
        flush.zero_()
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        fn()
        e1.record()
        torch.cuda.synchronize()
        ts.append(e0.elapsed_time(e1))
    if stats is not None:
        stats["min"] = min(ts)
    return statistics.median(ts)


def per_config(fa, flush, peak):
    """Forward TFLOP/s of every workload; backward TFLOP/s (preprocess, main
    kernel and dQ convert) of the backward workload, the non-causal d = 128
    workload and the causal GQA workload (kernel-only, inputs resident, L2
    flushed)."""
    import torch
    out = {}
    for w in workloads.WORKLOADS:
        x = workloads.workload_inputs(w, with_dout=True)
        q, k, v, do = (x[n].cuda() for n in ("q", "k", "v", "do"))
        o = torch.empty_like(q)
        lse = torch.empty((w.B, w.Hq, w.Nq), device="cuda", dtype=torch.float32)
        fwd = lambda: fa.fa_fwd(q, k, v, o, lse, w.B, w.Hq, w.Hkv, w.Nq, w.Nk, w.d, w.scale, int(w.causal))
        st = {}
        ms = time_one(fwd, flush, stats=st)
        ent = {"fwd_ms": ms, "fwd_min_ms": st["min"], "fwd_tflops": w.fwd_flops() / ms / 1e9}
        ent["fwd_frac_of_peak"] = ent["fwd_tflops"] / peak
        if w.d == 128:  # the same forward on CTA pairs (cta_group::2)
            fa.fa_tune(fa.TUNE_CTA_PAIRS, 1)
            pms = time_one(fwd, flush, stats=st)
            fa.fa_tune(fa.TUNE_CTA_PAIRS, 0)
            ent.update({"fwd_pairs_ms": pms, "fwd_pairs_min_ms": st["min"],
                        "fwd_pairs_tflops": w.fwd_flops() / pms / 1e9})
        if w.direction == "bwd" or w.name == "fwd_b4_h16_n2048_d128" or w.Hkv < w.Hq:
            dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
            bwd = lambda: fa.fa_bwd(q, k, v, o, lse, do, dq, dk, dv, w.B, w.Hq, w.Hkv, w.Nq, w.Nk, w.d, w.scale,
                                    int(w.causal))
            ms = time_one(bwd, flush, stats=st)
            ent.update({"bwd_ms": ms, "bwd_min_ms": st["min"], "bwd_tflops": w.bwd_flops() / ms / 1e9})
            ent["bwd_frac_of_peak"] = ent["bwd_tflops"] / peak
        out[w.name] = {kk: (round(vv, 4) if isinstance(vv, float) else vv) for kk, vv in ent.items()}
        del q, k, v, do, o, lse
        torch.cuda.synchronize()
    assert fa.fa_get_status() == 0
    return out


WINDOW_CASE = dict(name="fwd_bwd_window1024_b2_h16_n8192_d128", B=2, H=16, N=8192, d=128, window=(1023, 0), seed=1042)


def window_pairs(nq: int, nk: int, wl: int, wr: int) -> int:
    """Visible (query, key) pairs of one head under a sliding window
    (bounds as fa_fwd_window; negative = no limit)."""
    import numpy as np
    i = np.arange(nq, dtype=np.int64)
    off = nk - nq
    lo = np.maximum(0, i + off - wl) if wl >= 0 else np.zeros_like(i)
    hi = np.minimum(nk - 1, i + off + wr) if wr >= 0 else np.full_like(i, nk - 1)
    return int(np.maximum(0, hi - lo + 1).sum())


def window_config(fa, flush, peak):
    """Forward and backward TFLOP/s of a causal local window (1024 keys) at
    B=2, H=16, N=8192, d=128, counting only the visible pairs: 4*d flops per
    pair forward, 2.5x that backward."""
    import torch
    c = WINDOW_CASE
    x = workloads.make_inputs(c["B"], c["H"], c["H"], c["N"], c["N"], c["d"], c["seed"], with_dout=True)
    q, k, v, do = (x[n].cuda() for n in ("q", "k", "v", "do"))
    o, dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    lse = torch.empty((c["B"], c["H"], c["N"]), device="cuda", dtype=torch.float32)
    a = (c["B"], c["H"], c["H"], c["N"], c["N"], c["d"], c["d"] ** -0.5, *c["window"])
    fwd_fl = 4.0 * c["d"] * c["B"] * c["H"] * window_pairs(c["N"], c["N"], *c["window"])
    fms = time_one(lambda: fa.fa_fwd_window(q, k, v, o, lse, *a), flush)
    bms = time_one(lambda: fa.fa_bwd_window(q, k, v, o, lse, do, dq, dk, dv, *a), flush)
    assert fa.fa_get_status() == 0
    return {"window": list(c["window"]), "fwd_ms": round(fms, 4), "fwd_tflops": round(fwd_fl / fms / 1e9, 4),
            "fwd_frac_of_peak": round(fwd_fl / fms / 1e9 / peak, 4), "bwd_ms": round(bms, 4),
            "bwd_tflops": round(2.5 * fwd_fl / bms / 1e9, 4), "bwd_frac_of_peak": round(2.5 * fwd_fl / bms / 1e9 / peak, 4)}


def fp8_peak(peak_bf16: float):
    """Dense e4m3 tensor throughput of this GPU, measured with the vendor
    library: torch._scaled_mm (cuBLASLt) on 8192^3 e4m3 operands with bf16
    output, best of 10 after warm-up (2 * 8192^3 flop per call). Returns
    (TFLOP/s, source); twice the bf16 peak (the nominal ratio) if the call
    is unavailable."""
    import torch
    try:
        n = 8192
        a = torch.randn(n, n, device="cuda").to(torch.float8_e4m3fn)
        b = torch.randn(n, n, device="cuda").to(torch.float8_e4m3fn).t()
        one = torch.ones((), device="cuda", dtype=torch.float32)
        mm = lambda: torch._scaled_mm(a, b, scale_a=one, scale_b=one, out_dtype=torch.bfloat16)
        for _ in range(3):
            mm()
        torch.cuda.synchronize()
        ts = []
        for _ in range(10):
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record()
            mm()
            e1.record()
            torch.cuda.synchronize()
            ts.append(e0.elapsed_time(e1))
        return 2.0 * n ** 3 / min(ts) / 1e9, "measured: torch._scaled_mm e4m3 8192^3 (cuBLASLt), best of 10"
    except (RuntimeError, AttributeError, TypeError) as exc:
        return 2.0 * peak_bf16, f"2 x measured bf16 (nominal ratio; _scaled_mm unavailable: {type(exc).__name__})"


def fp8_config(fa, flush, peak):
    """The e4m3 forward (incoherent transform on) of the three d = 128 forward
    workloads: whole call (quantisation included) and the attention kernel
    alone, against the measured dense e4m3 peak (fp8_peak), beside the bf16
    forward call on the same inputs."""
    import torch
    p8, p8_src = fp8_peak(peak)
    out = {"fp8_peak": {"tflops": round(p8, 1), "source": p8_src}}
    for w in (workloads.WORKLOADS[1], workloads.WORKLOADS[2], workloads.WORKLOADS[3]):
        x = workloads.workload_inputs(w)
        q, k, v = (x[n].cuda() for n in ("q", "k", "v"))
        o = torch.empty_like(q)
        lse = torch.empty((w.B, w.Hq, w.Nq), device="cuda", dtype=torch.float32)
        a = (w.B, w.Hq, w.Hkv, w.Nq, w.Nk, w.d, w.scale, int(w.causal), 1)
        ms = time_one(lambda: fa.fa_fwd_fp8(q, k, v, o, lse, *a), flush)
        ms16 = time_one(lambda: fa.fa_fwd(q, k, v, o, lse, *a[:-1]), flush)
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record(); e1.record()
        ks = []
        for _ in range(5):
            flush.zero_()
            fa.fa_profile_events(e0, e1)
            fa.fa_fwd_fp8(q, k, v, o, lse, *a)
            fa.fa_profile_events(None, None)
            torch.cuda.synchronize()
            ks.append(e0.elapsed_time(e1))
        kms = statistics.median(ks)
        fl = w.fwd_flops()
        out["fp8_" + w.name] = {"call_ms": round(ms, 4), "call_tflops": round(fl / ms / 1e9, 2),
                                "bf16_call_ms": round(ms16, 4), "call_vs_bf16": round(ms16 / ms, 4),
                                "kernel_ms": round(kms, 4), "kernel_tflops": round(fl / kms / 1e9, 2),
                                "kernel_frac_of_fp8_peak": round(fl / kms / 1e9 / p8, 4)}
        del q, k, v, o, lse
    assert fa.fa_get_status() == 0
    return out


def link_bandwidth(nbytes: int = 256 << 20, reps: int = 5):
    """Pinned host <-> device copy bandwidth (GB/s, best of `reps`), one
    cudaMemcpyAsync per copy (torch's copy_ between a pinned host tensor and
    a device tensor), each direction alone and both at once on two streams."""
    import torch
    h_in = torch.empty(nbytes, dtype=torch.uint8, pin_memory=True)
    h_out = torch.empty(nbytes, dtype=torch.uint8, pin_memory=True)
    d_a = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    d_b = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()

    def best(fn):
        ts = []
        for _ in range(reps):
            torch.cuda.synchronize()
            t0 = time.perf_counter()
            fn()
            torch.cuda.synchronize()
            ts.append(time.perf_counter() - t0)
        return min(ts)

    h2d = nbytes / best(lambda: d_a.copy_(h_in, non_blocking=True)) / 1e9
    d2h = nbytes / best(lambda: h_out.copy_(d_b, non_blocking=True)) / 1e9

    def both():
        with torch.cuda.stream(s1):
            d_a.copy_(h_in, non_blocking=True)
        with torch.cuda.stream(s2):
            h_out.copy_(d_b, non_blocking=True)
    duplex = 2 * nbytes / best(both) / 1e9
    return {"h2d_gbps": round(h2d, 1), "d2h_gbps": round(d2h, 1), "duplex_gbps": round(duplex, 1),
            "how": f"pinned {nbytes >> 20} MiB, one cudaMemcpyAsync per copy, best of {reps}"}


def run_ours(args):
    import torch
    import torch.distributed as dist

    rank, world, local = dist_env()
    if world > 1:
        dist.init_process_group("nccl")
    torch.cuda.set_device(local)
    import __graft_entry__
    __graft_entry__.build()
    import exact_attention_99_gb300 as fa
    fa.fa_debug_set(0, 0)

    w = MAIN
    peak, peak_sus, peak_src = load_peaks()
    x = workloads.workload_inputs(w, with_dout=True)
    q, k, v, do = (x[n].cuda() for n in ("q", "k", "v", "do"))
    o, dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    lse = torch.empty((w.B, w.Hq, w.Nq), device="cuda", dtype=torch.float32)
    flush = torch.empty(FLUSH_BYTES, dtype=torch.uint8, device="cuda")
    args_f = (w.B, w.Hq, w.Hkv, w.Nq, w.Nk, w.d, w.scale, int(w.causal))
    K = args.steps
    ev = lambda: torch.cuda.Event(enable_timing=True)
    e0, e1 = [ev() for _ in range(K)], [ev() for _ in range(K)]
    kf0, kf1, kb0, kb1 = ([ev() for _ in range(K)] for _ in range(4))
    for e in kf0 + kf1 + kb0 + kb1:  # torch creates the CUDA event on first record
        e.record()
    torch.cuda.synchronize()

    def step(i=None):
        if i is not None:
            fa.fa_profile_events(kf0[i], kf1[i])
        st = fa.fa_fwd(q, k, v, o, lse, *args_f)
        if i is not None:
            fa.fa_profile_events(kb0[i], kb1[i])
        st |= fa.fa_bwd(q, k, v, o, lse, do, dq, dk, dv, *args_f)
        if i is not None:
            fa.fa_profile_events(None, None)
        if st:
            raise RuntimeError(f"launch failed: {st}")

    for _ in range(args.warmup):
        flush.zero_()
        step()
    torch.cuda.synchronize()
    if world > 1:
        dist.barrier()
    sampler = ClockSampler(local)
    sampler.start()
    time.sleep(0.05)
    torch.cuda.synchronize()
    sampler.mark_begin()
    for i in range(K):
        flush.zero_()
        e0[i].record()
        step(i)
        e1[i].record()
    torch.cuda.synchronize()
    sampler.mark_end()
    if world > 1:
        dist.barrier()
    clocks = sampler.stop()
    status = fa.fa_get_status()
    if status != 0:
        raise RuntimeError(f"device status {fa.fa_status_string(status)}")
    step_ms = [a.elapsed_time(b) for a, b in zip(e0, e1)]
    total_ms = sum(step_ms)
    fwd_ms = statistics.mean(a.elapsed_time(b) for a, b in zip(kf0, kf1))
    bwd_ms = statistics.mean(a.elapsed_time(b) for a, b in zip(kb0, kb1))
    total_ms = max_over_ranks(total_ms)
    value = job_tflops(world, K, step_flops(w), total_ms)

    # end to end through the public API: pinned host inputs in, results out
    host_in = {n: x[n].pin_memory() for n in ("q", "k", "v", "do")}
    host_out = {n: torch.empty(t.shape, dtype=t.dtype, pin_memory=True) for n, t in
                (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv))}
    h2d = sum(t.numel() * t.element_size() for t in host_in.values())
    d2h = sum(t.numel() * t.element_size() for t in host_out.values())
    ke = K  # as many calls as the device loop has steps
    ee0, ee1 = ev(), ev()
    torch.cuda.synchronize()
    host_args = [host_in[n] for n in ("q", "k", "v", "do")] + [host_out[n] for n in ("o", "lse", "dq", "dk", "dv")]
    if fa.fa_step_host(*host_args, *args_f):  # untimed: creates the copy streams, grows the pool
        raise RuntimeError("fa_step_host failed")
    torch.cuda.synchronize()
    # no L2 flush between calls: the calls overlap (below), and each one
    # copies all its inputs in, more bytes than L2 holds
    ee0.record()
    for i in range(ke):
        # one call: inputs in, forward + backward, results out, pipelined over chunks of heads
        if fa.fa_step_host(*host_args, *args_f):
            raise RuntimeError("fa_step_host failed")
    ee1.record()
    torch.cuda.synchronize()
    if fa.fa_get_status() != 0:
        raise RuntimeError("device status not OK after fa_step_host")
    # consecutive calls overlap (a call's input copies run while the previous
    # one computes, and its kernels while the previous one's results go
    # out), so the step time is the whole loop's device time per call
    e2e_ms = ee0.elapsed_time(ee1) / ke
    e2e_value = world * step_flops(w) / (e2e_ms * 1e-3) / 1e12
    link = link_bandwidth()
    # the step cannot take less than its device time nor than its copies at
    # the measured link rate (each direction alone); e2e_frac compares it
    # with that bound
    copy_ms = max(h2d / link["h2d_gbps"], d2h / link["d2h_gbps"]) * 1e-6
    bound_ms = max(total_ms / K, copy_ms)

    if rank != 0:
        if world > 1:
            dist.barrier()
            dist.destroy_process_group()
        return

    # dominant kernel and its roofline
    if bwd_ms >= fwd_ms:
        kname, kflops, kms = "bwd_main_kernel", w.bwd_flops(), bwd_ms
    else:
        kname, kflops, kms = "fa_fwd_kernel", w.fwd_flops(), fwd_ms
    achieved = kflops / (kms * 1e-3) / 1e12
    roofline = {"bound": "tensor", "kernel": kname, "achieved": round(achieved, 2), "peak": peak,
                "peak_source": peak_src + "; burst used: each launch is timed alone with CUDA events",
                "unit": "TFLOP/s", "frac": round(achieved / peak, 4),
                "frac_of_sustained": round(achieved / peak_sus, 4), "peak_sustained": peak_sus,
                "traffic": profiled_traffic(kname, w.name), "avg_launch_ms": round(kms, 4),
                "flops_per_launch": kflops}

    per_workload = per_config(fa, flush, peak)
    per_workload.update({WINDOW_CASE["name"]: window_config(fa, flush, peak)})
    per_workload.update(fp8_config(fa, flush, peak))
    # a roofline entry per published d = 128 workload and pass: kernel-call
    # time (median of 20, L2 flushed) against the measured burst peak, and
    # the DRAM bytes per launch of the pass's main kernel from a committed ncu
    # summary taken on the current source (else null)
    rooflines = {}
    for wl in workloads.WORKLOADS:
        if wl.d != 128:
            continue
        ent = per_workload[wl.name]
        for pas, kern, fl in (("fwd", "fa_fwd_kernel", wl.fwd_flops()), ("bwd", "bwd_main_kernel", wl.bwd_flops())):
            if f"{pas}_ms" not in ent:
                continue
            ach = fl / ent[f"{pas}_ms"] / 1e9
            rooflines[f"{wl.name}:{pas}"] = {
                "bound": "tensor", "achieved": round(ach, 1), "peak": peak, "unit": "TFLOP/s",
                "frac": round(ach / peak, 4), "time": "whole call" + (" (preprocess, main, dQ convert)" if pas == "bwd" else ""),
                "traffic": profiled_traffic(kern, wl.name), "traffic_kernel": kern}
    line = {
        "metric": METRIC, "value": round(value, 2), "unit": "TFLOP/s", "n_gpus": world, "steps": K,
        "warmup": args.warmup, "ms_per_step": round(total_ms / K, 4), "higher_is_better": True, "scaling": "weak",
        "vs_baseline": None, "dtype": "bf16", "data": "synthetic",
        "config": {"workload": w.name, "B": w.B, "Hq": w.Hq, "Hkv": w.Hkv, "Nq": w.Nq, "Nk": w.Nk, "d": w.d,
                   "causal": w.causal, "sigma_qk": w.sigma_qk, "sigma_v": w.sigma_v, "sigma_do": 1.0,
                   "step": "fwd (O, LSE) + bwd (dQ, dK, dV)", "l2": "flushed before every step (256 MB write)",
                   "parallelism": f"replicas x{world}"},
        "fwd_kernel_ms": round(fwd_ms, 4), "bwd_main_kernel_ms": round(bwd_ms, 4),
        "fwd_tflops": round(w.fwd_flops() / fwd_ms / 1e9, 2), "fwd_frac_of_peak": round(w.fwd_flops() / fwd_ms / 1e9 / peak, 4),
        "bwd_main_tflops": round(w.bwd_flops() / bwd_ms / 1e9, 2),
        "roofline": roofline,
        "rooflines": rooflines,
        "clocks": clocks,
        "e2e": {"value": round(e2e_value, 2), "unit": "TFLOP/s", "h2d_bytes_per_step": h2d,
                "d2h_bytes_per_step": d2h, "ms_per_step": round(e2e_ms, 4), "calls": ke,
                "l2": f"not flushed: each call copies {h2d / 1e6:.0f} MB of inputs in (L2: 129 MB)", "link": link,
                "link_gbps": link["duplex_gbps"], "copy_ms_at_link": round(copy_ms, 4),
                "bound_ms": round(bound_ms, 4), "frac_of_bound": round(bound_ms / e2e_ms, 4),
                "copy_fraction_of_link": round((h2d + d2h) / (e2e_ms * 1e-3) / 1e9 / link["duplex_gbps"], 4)},
        # the forward and the backward's kernels (pre-pass, main, dQ
        # conversion, and the pass over the GQA tail pieces when there are any)
        "gpu_launches": (1 + fa.fa_bwd_launches(w.B, w.Hq, w.Hkv, w.Nq, w.Nk, w.d, int(w.causal))) * K,
        "configs": per_workload,
    }
    if world == 1:
        flops_done, el, panels = oracle_sample(w, x, args.cpu_seconds)
        line["cpu_baseline"] = {
            "value": flops_done / el / 1e12, "unit": "TFLOP/s", "cores": blas_threads(), "kind": "oracle",
            "cpu_model": cpu_model(), "host_cpus": os.cpu_count(),
            "sample": f"{panels} panel(s), each the last {min(PANEL, w.Nq)} query rows of one (batch, head) of "
                      f"{w.name} against all keys, fp64 forward + backward, {el:.1f} s",
            "per_workload": oracle_per_workload(args.cpu_seconds / 6),
            "single_thread": oracle_single_thread()}
    print(json.dumps(line), flush=True)
    if world > 1:
        dist.barrier()
        dist.destroy_process_group()


def run_profile_target(args):
    """Profiling target: runs only the forward (fwd), the e4m3 forward with
    the incoherent transform (fwd8, d = 128 workloads) or only the backward
    of one named workload, --warmup + --steps times, and prints nothing else.
    Used to capture one kernel of one workload under ncu; prints no bench
    line."""
    import torch
    import __graft_entry__
    __graft_entry__.build()
    import exact_attention_99_gb300 as fa
    fa.fa_debug_set(0, 0)
    if fa.fa_tune(fa.TUNE_EXP2_SPLIT, args.exp2_split) or fa.fa_tune(fa.TUNE_CTA_PAIRS, int(args.cta_pairs)):
        raise ValueError("bad --exp2-split")
    if args.profile_workload in PACKED_CASES:
        return run_packed_profile_target(fa, args, PACKED_CASES[args.profile_workload])
    if args.profile_workload == WINDOW_CASE["name"]:
        c = WINDOW_CASE
        x = workloads.make_inputs(c["B"], c["H"], c["H"], c["N"], c["N"], c["d"], c["seed"], with_dout=True)
        a = (c["B"], c["H"], c["H"], c["N"], c["N"], c["d"], c["d"] ** -0.5, *c["window"])
        fwd_call, bwd_call = fa.fa_fwd_window, fa.fa_bwd_window
        B, H, N = c["B"], c["H"], c["N"]
    else:
        w = workloads.BY_NAME[args.profile_workload]
        x = workloads.workload_inputs(w, with_dout=True)
        a = (w.B, w.Hq, w.Hkv, w.Nq, w.Nk, w.d, w.scale, int(w.causal))
        fwd_call, bwd_call = fa.fa_fwd, fa.fa_bwd
        B, H, N = w.B, w.Hq, w.Nq
    q, k, v, do = (x[n].cuda() for n in ("q", "k", "v", "do"))
    o, dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    lse = torch.empty((B, H, N), device="cuda", dtype=torch.float32)
    if fwd_call(q, k, v, o, lse, *a):
        raise RuntimeError("forward failed")
    if args.profile_pass == "fwd8":
        if fwd_call is not fa.fa_fwd:
            raise ValueError("fwd8 profiles the unmasked or causal forward only")
        fwd_call = lambda *xs: fa.fa_fwd_fp8(*xs, 1)
    for _ in range(args.warmup + args.steps):
        st = fwd_call(q, k, v, o, lse, *a) if args.profile_pass in ("fwd", "fwd8") else \
            bwd_call(q, k, v, o, lse, do, dq, dk, dv, *a)
        if st:
            raise RuntimeError(f"launch failed: {st}")
    torch.cuda.synchronize()
    if fa.fa_get_status() != 0:
        raise RuntimeError("device status not OK")


def run_packed_profile_target(fa, args, c):
    """run_profile_target for a case of the packed calls (fwd or bwd)."""
    import torch
    if args.profile_pass == "fwd8":
        raise ValueError("fwd8 profiles the dense calls only")
    x = workloads.make_inputs(1, c["Hq"], c["Hkv"], sum(c["lens"]), sum(c["lens"]), c["d"], c["seed"], with_dout=True)
    q, k, v, do = (x[n][0].cuda() for n in ("q", "k", "v", "do"))
    cu = torch.tensor([0] + c["lens"], device="cuda").cumsum(0).to(torch.int32)
    o, lse = fa.forward_varlen(q, k, v, cu, cu, causal=True)
    for _ in range(args.warmup + args.steps):
        if args.profile_pass == "fwd":
            fa.forward_varlen(q, k, v, cu, cu, causal=True, out=(o, lse))
        else:
            fa.backward_varlen(q, k, v, o, lse, do, cu, cu, causal=True)
    torch.cuda.synchronize()
    if fa.fa_get_status() != 0:
        raise RuntimeError("device status not OK")


def run_exp2_split_sweep(args):
    """The d = 128 forward workloads timed with each exp2 split (fa_tune
    FA_TUNE_EXP2_SPLIT = 0, 8, 4, 2, 1): median of 10 calls after 3 warm-ups,
    L2 flushed before each, inputs resident. Prints one JSON object; no
    bench line."""
    import torch
    import __graft_entry__
    __graft_entry__.build()
    import exact_attention_99_gb300 as fa
    fa.fa_debug_set(0, 0)
    flush = torch.empty(FLUSH_BYTES, dtype=torch.uint8, device="cuda")
    out = {}
    for w in workloads.WORKLOADS[1:4]:
        x = workloads.workload_inputs(w)
        q, k, v = (x[n].cuda() for n in ("q", "k", "v"))
        o = torch.empty_like(q)
        lse = torch.empty((w.B, w.Hq, w.Nq), device="cuda", dtype=torch.float32)
        a = (w.B, w.Hq, w.Hkv, w.Nq, w.Nk, w.d, w.scale, int(w.causal))
        r = {}
        for sp in (0, 8, 4, 2, 1):
            if fa.fa_tune(fa.TUNE_EXP2_SPLIT, sp):
                raise RuntimeError("fa_tune failed")
            ms = time_one(lambda: fa.fa_fwd(q, k, v, o, lse, *a), flush, reps=10)
            r[str(sp)] = {"ms": round(ms, 4), "tflops": round(w.fwd_flops() / ms / 1e9, 1)}
        fa.fa_tune(fa.TUNE_EXP2_SPLIT, 0)
        out[w.name] = r
        del q, k, v, o, lse
    if fa.fa_get_status() != 0:
        raise RuntimeError("device status not OK")
    print(json.dumps(out), flush=True)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=50)  # about 0.4 s timed
    ap.add_argument("--warmup", type=int, default=5)
    ap.add_argument("--impl", choices=["ours", "reference"], default="ours")
    ap.add_argument("--cpu-seconds", type=float, default=12.0)
    ap.add_argument("--profile-workload", default=None, help="profiling target: run one workload's pass only")
    ap.add_argument("--profile-pass", choices=["fwd", "fwd8", "bwd"], default="fwd")
    ap.add_argument("--exp2-split", type=int, default=0, help="profiling target: forward exp2 split (fa_tune)")
    ap.add_argument("--exp2-split-sweep", action="store_true", help="time the d = 128 forwards for each exp2 split")
    ap.add_argument("--cta-pairs", action="store_true", help="profiling target: the d = 128 forward on CTA pairs")
    args = ap.parse_args()
    args.warmup = max(3, args.warmup)  # at least 3 untimed warm-up steps
    if args.exp2_split_sweep:
        run_exp2_split_sweep(args)
    elif args.profile_workload:
        run_profile_target(args)
    elif args.impl == "reference":
        run_reference(args)
    else:
        run_ours(args)


if __name__ == "__main__":
    main()
