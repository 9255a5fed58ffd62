#!/usr/bin/env python3
"""Benchmark of the MI355X last-axis ArgMax: microseconds per call and achieved HBM GB/s.

Headline workload: ArgMax over fp32 [1, 202048] (vocabulary-sized sampler logits,
iid N(0, 4), seed 2), the shape the "[CUDA] Parallelize ArgMax/ArgMin over wide last axes"
page profiles; [4096, 4096] fp32 (iid U(-1,1) with planted inf/NaN rows, seed 4) is timed
as the second shape of the same metric, and `all_configs` holds the same figures for every
configuration of the workload set ([1,32000] fp32, [1,202048] fp32 ArgMax and ArgMin,
[32,202048] fp16 and bf16 ArgMax and ArgMin, [4096,4096] fp32 and fp64, [65536,1024] fp32
ArgMin, [65536,64] fp16), each at the same steps and warm-up. A step is one call of the
library (every kernel it enqueues), on inputs already resident in HBM.

Timing: ten trials of 200 calls (below), then W untimed warm-up calls, then exactly K calls
between two HIP events on the stream the library launches on, synchronised on both sides; the inputs rotate through copies that
together exceed the 256 MB Infinity Cache, so every call reads HBM ("hot" repeats one
buffer and is reported beside it). The timed region divided by K is the per-call time
(`value`); the roofline divides the algorithmic bytes by that per-call time. HIP events
recorded around the main kernel of single calls (the library's measurement hook) give
`kernel_event_us`, a cross-check that includes the events' own overhead. The ten trials give
the spread of the per-call figure (`trials_us_per_call`); `host_enqueue_us_per_call` is the host's
time to enqueue one call, which at these sizes is close to the GPU's time per call (the host
launch path, not only the kernel, sets the rate). The launch floor is an empty kernel
launched the same way; the read floor (`read_floor`, read-only workloads) is a plain
streaming-read kernel over the same rotated inputs and byte count, the practical read
roofline in the same harness. The CPU baseline is the oracle (a single-threaded sequential
scan) timed on this host: the headline workload on one pinned core (median and min of five
runs), and the [4096,4096] and [65536,1024] fp32 workloads on one pinned core and with their
rows split across the host's threads (at most 16), with the host's core count and CPU model.

`--pmc-pass` runs a fixed sequence for hardware-counter collection instead (a 256 MiB
device copy, whose known bytes calibrate FETCH_SIZE / WRITE_SIZE, then 100 calls of each
configuration and op, and of three more workloads) and prints nothing on stdout;
`--traffic-summary`, `--counter-summary` and `--trace-summary` turn rocprofv3's CSV output
of such runs into the committed summaries (no GPU). `--shape ROWS,COLS,DTYPE[,OP]`
(repeatable) times the last-axis reduction of any shape against its streaming-read floor
and prints one JSON line per shape instead of the bench line.

Prints ONE JSON line on stdout; progress goes to stderr.
"""
from __future__ import annotations

import argparse
import json
import math
import os
import sys
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

# Kernel arguments in host memory (a HIP runtime setting; read when HIP starts, so set
# before torch is imported; an explicit setting in the environment wins). With the
# library's kernels preloading their arguments, the GPU time per call is the same either
# way, while a launch costs the host about 1.7 us instead of 3.0-3.3 us: the us-scale
# calls then stay bound by the GPU on any host core.
os.environ.setdefault("HIP_FORCE_DEV_KERNARG", "0")

HBM_PEAK_GBPS = 8000.0  # MI355X HBM3E
TRAFFIC_FILE = os.path.join(ROOT, "profiles", "pmc_traffic.json")
KERNEL_SOURCES = ("argmin_reduction_wide_amd/csrc/argreduce_kernels.hip",
                  "argmin_reduction_wide_amd/csrc/argreduce_scan.hip",
                  "argmin_reduction_wide_amd/csrc/argreduce_launch.hpp",
                  "argmin_reduction_wide_amd/csrc/argreduce_device.hpp",
                  "argmin_reduction_wide_amd/csrc/argreduce_api.cpp",
                  "argmin_reduction_wide_amd/csrc/argreduce_internal.hpp",
                  "argmin_reduction_wide_amd/csrc/argreduce_logits.hip",
                  "argmin_reduction_wide_amd/csrc/argreduce_logits.hpp",
                  "argmin_reduction_wide_amd/csrc/argreduce_logits_api.cpp",
                  "include/argreduce.h")
ROTATE_BYTES = 1 << 29  # 512 MiB of rotated inputs, twice the Infinity Cache
PAGES_US_1x202048 = 6.4  # ArgMax fp32 [1,202048] per call on the pages' H200
# The pages' own before / after pairs for shapes and formats measured here (NVIDIA H200,
# per call: "[CUDA] Parallelize ArgMax/ArgMin over wide last axes", Description / Results;
# before = the serial thread-per-row kernel, after = the cooperative kernel): context only.
PAGES_BEFORE_AFTER_US = {("argmax_f32_1x32000", "max"): (695.6, 5.9),
                         ("argmax_argmin_f32_1x202048", "max"): (5056.5, 6.4)}


def log(msg: str) -> None:
    print(msg, file=sys.stderr, flush=True)


def algorithmic_bytes(w) -> int:
    """Bytes one call must move: the input read once and an int64 per output (and, for a
    cumulative scan, a value per element)."""
    if w.kind == "scan":
        return 2 * w.nbytes + w.rows * w.cols * 8
    if w.axis_shape is not None:
        outer, _, inner = w.axis_shape
        return w.nbytes + outer * inner * 8
    return w.nbytes + w.rows * 8


class Case:
    """One workload on the device: rotated input copies, output, scratch."""

    def __init__(self, w, op: str, rotate_bytes: int = ROTATE_BYTES):
        import numpy as np
        import torch

        import argmin_reduction_wide_amd.binding as B

        self.w, self.op, self.B = w, op, B
        self.rows, self.cols = w.rows, w.cols
        from argmin_reduction_wide_amd import workloads as W

        one = W.device_data(w)
        tdt = one.dtype
        self.n_rot = max(1, math.ceil(rotate_bytes / w.nbytes))
        if self.n_rot == 1:
            self.x = one.view(1, self.rows, self.cols)
        else:
            self.x = torch.empty((self.n_rot, self.rows, self.cols), dtype=tdt, device="cuda")
            for i in range(self.n_rot):
                self.x[i].copy_(one)
            del one
        self.ptrs = [self.x[i].data_ptr() for i in range(self.n_rot)]
        self.stream = torch.cuda.current_stream().cuda_stream
        self.dt = B.DTYPE_NAMES[w.dtype]
        self.opc = B.OP_NAMES[op]
        self.vals = None
        if w.kind == "scan":
            n_out = self.rows * self.cols
            self.shape = (self.rows, self.cols)
            self.need = B.argreduce_scan_scratch_bytes(self.rows, self.cols, w.dtype)
            self.fn = B.entry_point("argreduce_scan_lastaxis")
            self.plan = B.argreduce_scan_plan(self.rows, self.cols, w.dtype)
            self.vals = torch.empty((self.rows, self.cols), dtype=tdt, device="cuda")
        elif w.axis_shape is None:
            n_out = self.rows
            self.shape = (self.rows, self.cols)
            self.need = B.argreduce_scratch_bytes(self.rows, self.cols, w.dtype)
            self.fn = B.entry_point("argreduce_lastaxis")
            self.plan = B.argreduce_plan(self.rows, self.cols, w.dtype)
        else:
            outer, length, inner = w.axis_shape
            n_out = outer * inner
            self.shape = (outer, length, inner)
            self.need = B.argreduce_axis_scratch_bytes(outer, length, inner, w.dtype)
            self.fn = B.entry_point("argreduce_axis")
            self.plan = B.argreduce_axis_plan(outer, length, inner, w.dtype)
        self.out = torch.empty(n_out, dtype=torch.int64, device="cuda")
        self.scratch = torch.empty(max(self.need, 1), dtype=torch.uint8, device="cuda")
        self.binding = "cpython-fastcall" if B.fast() is not None else "ctypes"
        self._argv_cache = None
        self.bytes = algorithmic_bytes(w)

    def set_op(self, op: str) -> None:
        """Calls from now on compute ``op`` (same inputs, outputs and scratch: the plan and
        scratch size do not depend on the op)."""
        if op != self.op:
            self.op, self.opc, self._argv_cache = op, self.B.OP_NAMES[op], None

    def argv(self, k: int) -> tuple:
        """The C call's arguments for rotated copy k (built once per copy and stream)."""
        if self._argv_cache is None or self._argv_cache[0] != self.stream:
            tail = ((self.vals.data_ptr(),) if self.vals is not None else ()) + (
                self.out.data_ptr(), self.scratch.data_ptr(), self.need, self.stream)
            self._argv_cache = (self.stream, [(p, self.dt, *self.shape, self.opc, *tail)
                                              for p in self.ptrs])
        return self._argv_cache[1][k]

    def call(self, i: int) -> None:
        rc = self.fn(*self.argv(i % self.n_rot))
        if rc != 0:
            raise RuntimeError(f"argreduce call failed with status {rc}")

    def timed(self, steps: int, warmup: int, rotate: bool = True, start: int = 0) -> float:
        """Microseconds per call over exactly `steps` calls (rotating from copy `start`)."""
        import torch

        for i in range(warmup):
            self.call(start + i if rotate else 0)
        torch.cuda.synchronize()
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        t0 = time.perf_counter()
        for i in range(steps):
            self.call(start + warmup + i if rotate else 0)
        # host time to enqueue the calls: when it matches the GPU time per call, the host's
        # launch path, not the kernel, sets the rate
        self.host_us = (time.perf_counter() - t0) * 1e6 / steps
        e1.record()
        torch.cuda.synchronize()
        return e0.elapsed_time(e1) * 1000.0 / steps

    def graph_timed(self, calls: int, replays: int) -> float:
        """Microseconds per call when `calls` rotated calls are replayed from a HIP graph."""
        import torch

        calls = max(1, min(calls, self.n_rot * 4))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        saved = self.stream
        with torch.cuda.stream(s):
            self.stream = s.cuda_stream
            with torch.cuda.graph(g, stream=s):
                for i in range(calls):
                    self.call(i)
        self.stream = saved
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        for _ in range(replays):
            g.replay()
        e1.record()
        torch.cuda.synchronize()
        del g
        return e0.elapsed_time(e1) * 1000.0 / (calls * replays)

    def kernel_timed(self, steps: int) -> float:
        """Average duration (us) of the row-scanning kernel alone, from HIP events that the
        library records immediately around it on the launch stream."""
        import torch

        evs = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
               for _ in range(steps)]
        for a, b in evs:  # materialise the hipEvent_t handles on this stream
            a.record()
            b.record()
        torch.cuda.synchronize()
        try:
            for i, (a, b) in enumerate(evs):
                self.B.argreduce_debug_set_kernel_events(a.cuda_event, b.cuda_event)
                self.call(i)
        finally:
            self.B.argreduce_debug_set_kernel_events(0, 0)
        torch.cuda.synchronize()
        return sum(a.elapsed_time(b) for a, b in evs) * 1000.0 / steps

    def read_floor(self, steps: int, grids=(512, 1024, 2048, 4096)) -> dict:
        """The practical read roofline for this workload: a plain streaming-read kernel over
        the same rotated inputs and byte count (no reduction work), fastest of a few grids."""
        import torch

        nbytes = self.w.nbytes // 16 * 16
        sink = torch.empty(max(grids), dtype=torch.int32, device="cuda")
        best = None
        for grid in grids:
            read = self.B.entry_point("argreduce_debug_launch_read")
            sink_ptr = sink.data_ptr()

            def go(i):
                rc = read(self.ptrs[i % self.n_rot], nbytes, sink_ptr, grid, self.stream)
                if rc != 0:
                    raise RuntimeError(f"streaming read failed with status {rc}")
            for i in range(20):
                go(i)
            torch.cuda.synchronize()
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record()
            for i in range(steps):
                go(i)
            e1.record()
            torch.cuda.synchronize()
            us = e0.elapsed_time(e1) * 1000.0 / steps
            if best is None or us < best[0]:
                best = (us, grid)
        return {"us_per_call": round(best[0], 3), "grid": best[1], "bytes": nbytes,
                "gbps": round(nbytes / (best[0] * 1e-6) / 1e9, 1)}

    def result(self):
        import torch

        torch.cuda.synchronize()
        return self.out.cpu().numpy()


def launch_floor_us(steps: int, store: bool = False) -> float:
    """Per-call time of an empty kernel (no arguments), or, with `store`, of a kernel that
    takes one pointer argument and stores one int64: the floor of any call that returns a
    result. The difference is the host's launch path for a kernel with arguments: the host
    needs as long to enqueue such a launch as the GPU needs per call, and how long depends
    on the CPU core the launching thread runs on."""
    import torch

    import argmin_reduction_wide_amd.binding as B

    stream = torch.cuda.current_stream().cuda_stream
    if store:
        out = torch.zeros(1, dtype=torch.int64, device="cuda")
        out_ptr = out.data_ptr()
        g = B.entry_point("argreduce_debug_launch_store")
        f = lambda st: g(out_ptr, st)
    else:
        f = B.entry_point("argreduce_debug_launch_empty")
    for _ in range(50):
        f(stream)
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    for _ in range(steps):
        f(stream)
    e1.record()
    torch.cuda.synchronize()
    return e0.elapsed_time(e1) * 1000.0 / steps


def code_text(src: str) -> str:
    """Source text without comments and with whitespace collapsed: what the compiler sees
    (the sources hold no string literals with comment markers)."""
    import re

    src = re.sub(r"/\*.*?\*/", " ", src, flags=re.S)
    src = re.sub(r"//[^\n]*", " ", src)
    return " ".join(src.split())


def kernel_source_hash() -> str:
    """sha256 over the library sources' code (comments and layout excluded): counter figures
    are valid only for the library built from these sources."""
    import hashlib

    h = hashlib.sha256()
    for rel in KERNEL_SOURCES:
        with open(os.path.join(ROOT, rel), encoding="utf-8") as f:
            h.update(code_text(f.read()).encode())
    return h.hexdigest()[:16]


def measured_traffic(workload: str):
    """HBM bytes per launch of ``workload`` ("name:op") from the committed FETCH_SIZE /
    WRITE_SIZE summary (scaled by the copy-kernel calibration), or None when absent or taken
    on other kernel sources."""
    try:
        with open(TRAFFIC_FILE) as f:
            rec = json.load(f)
    except (OSError, ValueError):
        return None
    if rec.get("source_hash") != kernel_source_hash():
        return None
    k = rec.get("kernels", {}).get(workload)
    return None if k is None else int(round(k["traffic_bytes"]))


def roofline(bytes_per_call: int, kernel_us: float, workload: str = "") -> dict:
    achieved = bytes_per_call / (kernel_us * 1e-6) / 1e9
    return {"bound": "hbm", "achieved": round(achieved, 1), "peak": HBM_PEAK_GBPS,
            "unit": "GB/s", "frac": round(achieved / HBM_PEAK_GBPS, 4),
            "traffic": measured_traffic(workload)}


def cooperative_off(c) -> dict:
    """The same calls with the cooperative (split) path disabled: the pages compare their
    kernel with the serial thread-per-row kernel from the same binary and data ("[CUDA]
    Parallelize ArgMax/ArgMin over wide last axes", Verification log). Here the library's
    path override runs one lane per row (one 16-byte load in flight: milliseconds per call,
    so three timed calls) and one workgroup per row (200 calls), on the same rotated
    inputs; both must return the automatic path's indices."""
    B = c.B
    c.call(0)
    want = c.result().copy()
    rec = {"source": "this library with the split path overridden, same inputs and harness"}
    try:
        for name, path, steps, warm in (("thread_per_row", B.PATH_THREAD, 3, 1),
                                        ("block_per_row", B.PATH_BLOCK, 200, 20)):
            B.argreduce_debug_force_path(path)
            us = c.timed(steps, warm, rotate=True, start=4000)
            c.call(0)
            rec[name] = {"us_per_call": round(us, 3), "calls": steps,
                         "same_indices": bool((c.result() == want).all())}
            log(f"[bench]   split path off ({name}): {us:.3f} us per call")
    finally:
        B.argreduce_debug_force_path(B.PATH_AUTO)
    return rec


def measure(w, op: str, steps: int, warmup: int, graph: bool = True, case=None) -> dict:
    """One (workload, op) record; ``case`` reuses another op's rotated inputs of the same
    workload (a second 512 MiB allocation of the same data measured up to 0.35 us per call
    slower on [1,202048] than the first, op for op)."""
    c = case if case is not None else Case(w, op)
    c.set_op(op)
    log(f"[bench] {w.name} {op}: plan {c.plan}, {c.n_rot} rotated copies")
    # ten trials of 200 rotated calls, each continuing the rotation where the last one
    # stopped (no copy is read again while it can still sit in the Infinity Cache): the
    # spread of the per-call figure. They run first, so that the host's launch path is in
    # its steady state when the W warm-up and K timed calls follow (a host core that has
    # just been generating inputs enqueues the first few hundred calls up to twice as
    # slowly, which at these sizes the GPU would wait for).
    trials = sorted(c.timed(200, 0, rotate=True, start=200 * k) for k in range(10))
    us = c.timed(steps, warmup, rotate=True, start=2000)
    host_us = c.host_us
    hot = c.timed(steps, warmup // 4 + 1, rotate=False)
    kus = c.kernel_timed(min(steps, 1000))
    gus = c.graph_timed(min(steps, 200), max(1, steps // 200)) if graph else None
    # the read roofline in the same harness (read-only workloads: a scan also writes)
    rf = c.read_floor(min(steps, 500)) if c.vals is None else None
    rec = {
        "workload": w.name, "op": op, "dtype": w.dtype, "shape": list(c.shape),
        "us_per_call": round(us, 3), "host_enqueue_us_per_call": round(host_us, 3),
        "binding": c.binding,
        "hot_us_per_call": round(hot, 3),
        "trials_us_per_call": {"n": 10, "calls": 200, "min": round(trials[0], 3),
                               "median": round((trials[4] + trials[5]) / 2, 3),
                               "max": round(trials[-1], 3)},
        "graph_us_per_call": None if gus is None else round(gus, 3),
        "kernel_event_us": round(kus, 3),
        "gbps_per_call": round(c.bytes / (us * 1e-6) / 1e9, 1),
        "pct_hbm_peak_per_call": round(100 * c.bytes / (us * 1e-6) / 1e9 / HBM_PEAK_GBPS, 2),
        "algorithmic_bytes": c.bytes, "rotated_copies": c.n_rot, "plan": c.plan,
        "read_floor": rf,
        "pct_of_read_floor": None if rf is None else round(100 * rf["us_per_call"] / us, 1),
        # achieved bandwidth over the timed region: the HIP events around the K timed calls on
        # the launch stream, divided by K. In this GPU-bound loop that is the kernel's
        # average time per launch, which rocprofv3's kernel trace of the same command agrees
        # with; events recorded around each single launch (kernel_event_us) carry their own
        # overhead and serve as a cross-check only.
        "roofline": roofline(c.bytes, us, f"{w.name}:{op}"),
    }
    if c.plan["path"] == c.B.PATH_SPLIT:
        off = cooperative_off(c)
        for name in ("thread_per_row", "block_per_row"):
            off[name]["speedup_of_split"] = round(off[name]["us_per_call"] / us, 1)
        pages = PAGES_BEFORE_AFTER_US.get((w.name, op))
        if pages is not None:
            off["pages_h200"] = {"before_us": pages[0], "after_us": pages[1],
                                 "speedup": round(pages[0] / pages[1], 1)}
        rec["before"] = off
    log(f"[bench]   {json.dumps(rec)}")
    rec["_case"] = c
    return rec


COPY_BYTES = 256 << 20


def pmc_workloads() -> list:
    """(workload, op) of the counter pass, in launch order: every configuration of the
    metric's workload set, each op, then the [64,4096,256] fp32 and [4,16384,1001] fp16
    middle-axis ArgMax and the [4096,4096] and [1,2^24] fp32 cummax workloads."""
    from argmin_reduction_wide_amd import workloads as W

    out = []
    for name in W.CONFIG_NAMES:
        for w in W.config_workloads(name):
            out.extend((w, op) for op in w.ops)
    out += [(W.axis_many_outputs_f32(), "max"), (W.axis_element_loads_f16(), "max"),
            (W.scan_many_rows_f32(), "max"),
            (W.scan_long_row_f32(), "max")]
    return out


PMC_CALLS = 100


def pmc_pass() -> int:
    """Fixed kernel sequence for counter collection: a device-to-device copy of COPY_BYTES
    (the calibration: it reads and writes exactly that many bytes), then PMC_CALLS calls of
    each (workload, op) of pmc_workloads(), on rotated inputs."""
    import torch

    src = torch.empty(COPY_BYTES, dtype=torch.uint8, device="cuda")
    dst = torch.empty_like(src)
    src.fill_(1)
    torch.cuda.synchronize()
    dst.copy_(src)
    torch.cuda.synchronize()
    del src, dst
    torch.cuda.empty_cache()
    for w, op in pmc_workloads():
        c = Case(w, op)
        for i in range(PMC_CALLS):
            c.call(i)
        torch.cuda.synchronize()
        log(f"[pmc] {w.name} {op}: {PMC_CALLS} calls, {c.bytes} algorithmic bytes per call, "
            f"plan {c.plan}")
        del c
        torch.cuda.empty_cache()
    return 0


def _csv_rows(directory: str, suffix: str) -> list:
    import csv
    import glob

    paths = sorted(glob.glob(os.path.join(directory, "**", "*" + suffix), recursive=True))
    if not paths:
        raise FileNotFoundError(f"no *{suffix} under {directory}")
    rows = []
    for path in paths:
        with open(path, newline="") as f:
            rows.extend(csv.DictReader(f))
    return rows


def _short(name: str) -> str:
    """A kernel's name without its argument list (and the return type)."""
    anon = "(anonymous namespace)"
    name = name.replace(anon, "\0").split("(")[0].replace("\0", anon)
    return name[5:] if name.startswith("void ") else name


def _dispatch_values(directory: str, counter: str) -> list:
    """[(kernel name, value)] of one counter in dispatch order (rocprofv3 --pmc CSV)."""
    vals = {}
    for r in _csv_rows(directory, "counter_collection.csv"):
        if r["Counter_Name"] == counter:
            key = int(r["Dispatch_Id"])
            prev = vals.get(key)
            vals[key] = (r["Kernel_Name"], float(r["Counter_Value"]) + (prev[1] if prev else 0.0))
    if not vals:
        raise ValueError(f"no {counter} values under {directory}")
    return [vals[k] for k in sorted(vals)]


def _per_workload(disp: list):
    """Assigns the library's dispatches of a --pmc-pass run to pmc_workloads() in launch
    order (PMC_CALLS calls each; a split middle-axis call has a second, merge dispatch) and
    yields (workload, op, first kernel's name, that kernel's values)."""
    lib = [(n, v) for n, v in disp if "argreduce::" in n]
    pos = 0
    for w, op in pmc_workloads():
        first = lib[pos][0]
        per_call = 2 if pos + 1 < len(lib) and "merge" in lib[pos + 1][0] else 1
        vals = [v for n, v in lib[pos:pos + PMC_CALLS * per_call] if n == first]
        assert len(vals) == PMC_CALLS, (w.name, op, first, len(vals))
        pos += PMC_CALLS * per_call
        yield w, op, first, vals


def traffic_summary(fetch_dir: str, write_dir: str) -> int:
    """HBM bytes per dispatch from the rocprofv3 FETCH_SIZE and WRITE_SIZE passes over
    --pmc-pass: the calibration copy's readings give the scale factors, and the library's
    dispatches are assigned to pmc_workloads() in launch order. Writes the traffic file
    bench.py reads (keyed by workload and op, tagged with the source hash) and prints a
    markdown table."""
    fetch = _dispatch_values(fetch_dir, "FETCH_SIZE")
    write = _dispatch_values(write_dir, "WRITE_SIZE")
    assert [n for n, _ in fetch] == [n for n, _ in write], "the two passes launched different kernels"
    cal_f = next(v for n, v in fetch if "copyBuffer" in n)
    cal_w = next(v for n, v in write if "copyBuffer" in n)
    fetch_factor = COPY_BYTES / (cal_f * 1024.0)
    write_factor = COPY_BYTES / (cal_w * 1024.0)
    rec = {"source_hash": kernel_source_hash(), "fetch_factor": fetch_factor,
           "write_factor": write_factor,
           "calibration": f"device copy of {COPY_BYTES} bytes: FETCH_SIZE {cal_f} KiB, "
                          f"WRITE_SIZE {cal_w} KiB", "kernels": {}}
    lines = ["| kernel | workload | op | dispatches | FETCH_SIZE KiB | WRITE_SIZE KiB | traffic bytes "
             "| algorithmic bytes | traffic / algorithmic |",
             "|---|---|---|---:|---:|---:|---:|---:|---:|"]
    for (w, op, first, vf), (_, _, _, vw) in zip(_per_workload(fetch), _per_workload(write)):
        fk, wk = sum(vf) / len(vf), sum(vw) / len(vw)
        traffic = fk * 1024 * fetch_factor + wk * 1024 * write_factor
        c_bytes = algorithmic_bytes(w)
        rec["kernels"][f"{w.name}:{op}"] = {"kernel": first, "fetch_kib": fk, "write_kib": wk,
                                           "traffic_bytes": traffic, "algorithmic_bytes": c_bytes}
        lines.append(f"| `{_short(first)}` | {w.name} | {op} | {len(vf)} | {fk:.2f} | {wk:.2f} | "
                     f"{traffic:,.0f} | {c_bytes:,} | {traffic / c_bytes:.4f} |")
    with open(TRAFFIC_FILE, "w") as f:
        json.dump(rec, f, indent=1)
    print(f"Calibration: {rec['calibration']}; fetch factor {fetch_factor:.4f}, write factor "
          f"{write_factor:.4f}. Source hash {rec['source_hash']}.\n")
    print("\n".join(lines))
    return 0


def counter_summary(directories: list) -> int:
    """Per-workload averages of every counter found in rocprofv3 --pmc runs of --pmc-pass
    (one directory per run), as a markdown table."""
    import csv  # noqa: F401

    columns = []
    for d in directories:
        names = sorted({r["Counter_Name"] for r in _csv_rows(d, "counter_collection.csv")})
        columns += [(d, n) for n in names]
    tables = [list(_per_workload(_dispatch_values(d, n))) for d, n in columns]
    print("| kernel | workload | op | dispatches | " + " | ".join(n for _, n in columns) + " |")
    print("|---|---|---|---:|" + "---:|" * len(columns))
    for rows in zip(*tables):
        w, op, first, vals = rows[0]
        avgs = " | ".join(f"{sum(r[3]) / len(r[3]):.2f}" for r in rows)
        print(f"| `{_short(first)}` | {w.name} | {op} | {len(vals)} | {avgs} |")
    return 0


def trace_summary(directory: str) -> int:
    """A markdown table of rocprofv3's kernel statistics (--kernel-trace --stats), with the
    median duration per kernel when the per-dispatch trace is there too."""
    rows = _csv_rows(directory, "kernel_stats.csv")
    rows.sort(key=lambda r: -float(r["TotalDurationNs"]))
    medians = {}
    try:
        per = {}
        for r in _csv_rows(directory, "kernel_trace.csv"):
            per.setdefault(r["Kernel_Name"], []).append(
                int(r["End_Timestamp"]) - int(r["Start_Timestamp"]))
        for name, d in per.items():
            d.sort()
            medians[name] = d[len(d) // 2] / 1e3
    except FileNotFoundError:
        pass
    print("| kernel | calls | avg µs | median µs | min µs | max µs | % of GPU time |")
    print("|---|---:|---:|---:|---:|---:|---:|")
    for r in rows:
        med = medians.get(r["Name"])
        print(f"| `{_short(r['Name'])}` | {r['Calls']} | {float(r['AverageNs']) / 1e3:.3f} | "
              f"{'—' if med is None else f'{med:.3f}'} | {float(r['MinNs']) / 1e3:.3f} | "
              f"{float(r['MaxNs']) / 1e3:.3f} | {float(r['Percentage']):.2f} |")
    return 0


# Host threads of the all-cores oracle leg: at most the CPU share one GPU's job gets.
CPU_THREADS_MAX = 16


def host_info() -> dict:
    model = None
    try:
        with open("/proc/cpuinfo") as f:
            for line in f:
                if line.startswith("model name"):
                    model = line.split(":", 1)[1].strip()
                    break
    except OSError:
        pass
    return {"nproc": os.cpu_count(), "affinity_cpus": len(os.sched_getaffinity(0)),
            "cpu_model": model}


def oracle_leg(o, w, op: str, threads: int, runs: int = 5, min_run_s: float = 0.0) -> dict:
    """The oracle's time per call of ``arg{op}`` over the whole workload ``w``: one warm-up
    call, then ``runs`` timed runs (each of as many calls as fill ``min_run_s``, at least
    one); median and min of the per-call time over the runs. With ``threads`` == 1 the
    calling thread is pinned to one core for the runs; with more, the rows are split into
    ``threads`` contiguous slices, each scanned by the oracle on a thread of its own (the
    scan within a row stays sequential; the ctypes call releases the GIL)."""
    import threading

    data = w.data
    rows = data.shape[0]
    if threads == 1:
        def call():
            return o.argreduce_lastaxis(data, w.dtype, op)
    else:
        bounds = [rows * k // threads for k in range(threads + 1)]
        parts = [None] * threads

        def work(k):
            parts[k] = o.argreduce_lastaxis(data[bounds[k]:bounds[k + 1]], w.dtype, op)

        def call():
            ts = [threading.Thread(target=work, args=(k,)) for k in range(threads)]
            for t in ts:
                t.start()
            for t in ts:
                t.join()
            import numpy as np
            return np.concatenate(parts)

    saved = os.sched_getaffinity(0)
    core = min(saved)
    if threads == 1:
        os.sched_setaffinity(0, {core})
    try:
        res = call()  # warm-up
        per_call = []
        for _ in range(runs):
            n, t0 = 0, time.perf_counter()
            while True:
                call()
                n += 1
                el = time.perf_counter() - t0
                if el >= min_run_s:
                    break
            per_call.append(el / n)
    finally:
        os.sched_setaffinity(0, saved)
    per_call.sort()
    med = per_call[len(per_call) // 2]
    return {"workload": w.name, "op": op, "shape": [w.rows, w.cols], "dtype": w.dtype,
            "threads": threads, "pinned_core": core if threads == 1 else None, "runs": runs,
            "us_per_call_median": round(med * 1e6, 1),
            "us_per_call_min": round(per_call[0] * 1e6, 1),
            "gbps_median": round(w.nbytes / med / 1e9, 2), "_result": res}


def cpu_baseline(primary, multi: list, seconds: float) -> dict:
    """The oracle timed on this host: the headline workload on one pinned core (the
    reported value), and the multi-row workloads on one pinned core and on all host
    threads (rows split across them), each as the median and min of five runs."""
    import oracle

    o = oracle.load()
    host = host_info()
    threads = max(1, min(host["affinity_cpus"], CPU_THREADS_MAX))
    w, op = primary
    head = oracle_leg(o, w, op, 1, runs=5, min_run_s=seconds / 6)
    res = head.pop("_result")
    legs = [head]
    for mw, mop in multi:
        for t in (1, threads):
            leg = oracle_leg(o, mw, mop, t, runs=5)
            leg.pop("_result")
            legs.append(leg)
            log(f"[bench] oracle {mw.name} arg{mop} on {t} thread(s): "
                f"{leg['us_per_call_median']} us/call (median of 5)")
    return {"value": head["us_per_call_median"], "unit": "us/call", "cores": 1, "kind": "oracle",
            "min": head["us_per_call_min"],
            "sample": f"arg{op} {w.dtype} [{w.rows},{w.cols}] (the timed workload's input) by the "
                      f"single-threaded oracle pinned to core {head['pinned_core']}: median of 5 "
                      f"runs of about {seconds / 6:.1f} s each after one warm-up call; the legs "
                      f"add the multi-row workloads on 1 and on {threads} host threads",
            "host": host, "legs": legs, "_result": res}


def shape_lines(specs: list, steps: int, warmup: int) -> int:
    """--shape: per shape, the per-call time of the timed region (inputs rotated as for the
    workloads), the trials' median, and the streaming-read floor of the same bytes."""
    import numpy as np
    import torch

    import argmin_reduction_wide_amd.binding as B
    from argmin_reduction_wide_amd import workloads as W

    launch_floor_us(2000)  # brings the host's launch path up to speed first
    for spec in specs:
        parts = spec.split(",")
        if len(parts) not in (3, 4, 6):
            raise SystemExit(f"--shape {spec}: expected ROWS,COLS,DTYPE[,OP[,B,U]]")
        rows, cols, dtype = int(parts[0]), int(parts[1]), parts[2]
        op = parts[3] if len(parts) >= 4 else "max"
        forced = (int(parts[4]), int(parts[5])) if len(parts) == 6 else (0, 1)
        if B.argreduce_debug_force_split(*forced) != 0:
            raise SystemExit(f"--shape {spec}: invalid split B={forced[0]} U={forced[1]}")
        rng = np.random.default_rng(rows * 1000003 + cols)
        data = W.to_storage(rng.standard_normal((rows, cols)), dtype)
        w = W.Workload(name=f"arg{op}_{dtype}_{rows}x{cols}", dtype=dtype, ops=(op,), data=data,
                       seed=rows * 1000003 + cols, recipe="iid N(0,1)")
        c = Case(w, op)
        trials = sorted(c.timed(200, 10, start=1000 * k) for k in range(5))
        us = c.timed(steps, warmup)
        floor = c.read_floor(min(steps, 500)) if w.nbytes >= 16 else None
        print(json.dumps({
            "shape": [rows, cols], "dtype": dtype, "op": op, "us_per_call": round(us, 3),
            "trials_median_us": round(trials[2], 3),
            "gbps": round(algorithmic_bytes(w) / us / 1e3, 1),
            "read_floor_us": floor["us_per_call"] if floor else None,
            "pct_of_read_floor": round(100.0 * floor["us_per_call"] / us, 1) if floor else None,
            "plan": c.plan}), flush=True)
        del c
        B.argreduce_debug_force_split(0)
        torch.cuda.empty_cache()
    return 0


def main() -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=2000)
    ap.add_argument("--warmup", type=int, default=200)
    ap.add_argument("--cpu-seconds", type=float, default=10.0)
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--all", action="store_true",
                    help="also time the middle-axis, cumulative-scan and wide-row workloads")
    ap.add_argument("--pmc-pass", action="store_true",
                    help="run the counter-collection sequence (for rocprofv3 --pmc) and exit")
    ap.add_argument("--traffic-summary", nargs=2, metavar=("FETCH_DIR", "WRITE_DIR"),
                    help="summarise the rocprofv3 FETCH_SIZE / WRITE_SIZE passes over --pmc-pass "
                         "(writes the traffic file, prints a table; no GPU)")
    ap.add_argument("--counter-summary", nargs="+", metavar="DIR",
                    help="per-workload averages of the counters of rocprofv3 --pmc runs over "
                         "--pmc-pass (no GPU)")
    ap.add_argument("--trace-summary", metavar="DIR",
                    help="print rocprofv3's kernel statistics under DIR as a table (no GPU)")
    ap.add_argument("--shape", action="append", metavar="ROWS,COLS,DTYPE[,OP[,B,U]]",
                    help="time the last-axis reduction (OP: max, min, max_last, min_last; default "
                         "max) of one seeded N(0,1) [ROWS, COLS] tensor against its streaming-read "
                         "floor, one JSON line per shape instead of the bench line; B,U force a "
                         "split of B workgroups per row and U loads per lane; repeatable")
    args = ap.parse_args()
    if args.traffic_summary:
        return traffic_summary(*args.traffic_summary)
    if args.trace_summary:
        return trace_summary(args.trace_summary)
    if args.counter_summary:
        return counter_summary(args.counter_summary)
    if args.gpus != 1:
        print(f"bench.py measures one GPU; --gpus {args.gpus} is not supported: the library "
              "has no multi-GPU path (rows, or column slices of one wide row, would shard "
              "across GPUs, the slices with one all-gather of ~16-byte candidates).",
              file=sys.stderr)
        return 2

    import torch

    from argmin_reduction_wide_amd import workloads as W

    assert torch.cuda.is_available(), "bench.py needs a GPU"
    torch.cuda.set_device(0)
    props = torch.cuda.get_device_properties(0)
    log(f"[bench] device {props.name} {getattr(props, 'gcnArchName', '')} "
        f"CUs={props.multi_processor_count}")

    if args.pmc_pass:
        return pmc_pass()
    if args.shape:
        return shape_lines(args.shape, args.steps, args.warmup)

    # The launch floors first: they also bring the host's launch path up to speed (the first
    # thousands of launches of a process enqueue measurably slower), so the headline's timed
    # calls are not the process's first.
    floor = launch_floor_us(max(args.steps, 2000))
    store_floor = launch_floor_us(max(args.steps, 2000), store=True)
    log(f"[bench] launch floor (empty kernel) {floor:.3f} us; one-argument store kernel "
        f"{store_floor:.3f} us")
    primary_w = W.c2_row202048_f32()
    prim = measure(primary_w, "max", args.steps, args.warmup)
    parity_result = prim["_case"].result()
    # the headline's other op on the same rotated inputs
    done = {(primary_w.name, "max"): prim,
            (primary_w.name, "min"): measure(primary_w, "min", args.steps, args.warmup,
                                             graph=False, case=prim["_case"])}
    for r in done.values():
        r.pop("_case")
    torch.cuda.empty_cache()
    sec_w = W.c4_square_f32_f64("f32")
    sec = measure(sec_w, "max", args.steps, args.warmup)
    sec.pop("_case")
    done[(sec_w.name, "max")] = sec
    torch.cuda.empty_cache()

    # Every configuration of the metric's workload set (C1 .. C5b, each op), at the same
    # steps and warm-up, every op of a workload on one set of rotated inputs; the shapes
    # above are not timed twice.
    all_configs = []
    multi_rows = {}
    for name in W.CONFIG_NAMES:
        for w in W.config_workloads(name):
            case = None
            for op in w.ops:
                r = done.get((w.name, op))
                if r is None:
                    r = measure(w, op, args.steps, args.warmup, graph=False, case=case)
                    case = r.pop("_case")
                all_configs.append(dict(r, config=name))
            del case
            torch.cuda.empty_cache()
            if name in ("c4", "c5a") and w.dtype == "f32":
                multi_rows[name] = (w, w.ops[0])

    extra = []
    if args.all:
        for name in ("axis", "scan", "wide"):
            for w in W.config_workloads(name):
                for op in w.ops:
                    r = measure(w, op, max(200, args.steps // 4), args.warmup // 4 + 1, graph=False)
                    r.pop("_case")
                    extra.append(r)
                    torch.cuda.empty_cache()

    cpu = None
    parity = None
    if not args.no_cpu_baseline:
        cpu = cpu_baseline((primary_w, "max"), [multi_rows["c4"], multi_rows["c5a"]],
                           args.cpu_seconds)
        res = cpu.pop("_result")
        parity = bool((parity_result == res).all())
    rec = {
        "metric": "ArgMax µs/call and achieved HBM GB/s (% of peak) at [1,202048] and [4096,4096]",
        "value": prim["us_per_call"],
        "unit": "us/call",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(prim["us_per_call"] / 1000.0, 6),
        "higher_is_better": False,
        "scaling": "weak",
        # the pages' own figure for this workload and metric ("[CUDA] Parallelize
        # ArgMax/ArgMin over wide last axes", Description: the cooperative kernel on an
        # NVIDIA H200, per call including the launch): another machine's number, context
        # only; below 1 is faster (lower is better)
        "vs_baseline": round(prim["us_per_call"] / PAGES_US_1x202048, 3),
        "baseline": {"value": PAGES_US_1x202048, "unit": "us/call",
                     "source": "the pages' cooperative kernel on NVIDIA H200 (context)"},
        "dtype": "f32",
        "data": "synthetic",
        "config": {"workload": "ArgMax fp32 [1,202048], iid N(0,4) seed 2, inputs rotated over "
                               f"{prim['rotated_copies']} HBM-resident copies",
                   "rows": 1, "cols": 202048, "op": "max", "plan": prim["plan"]},
        "gbps_per_call": prim["gbps_per_call"],
        "pct_hbm_peak_per_call": prim["pct_hbm_peak_per_call"],
        "host_enqueue_us_per_call": prim["host_enqueue_us_per_call"],
        "binding": prim["binding"],
        "hip_kernel_args": "device memory" if os.environ.get("HIP_FORCE_DEV_KERNARG") == "1"
                           else "host memory",
        "hot_us_per_call": prim["hot_us_per_call"],
        # the same calls with the split path overridden (one lane per row: the pages'
        # "before" kernel; one workgroup per row), same library and inputs
        "before": prim.get("before"),
        "trials_us_per_call": prim["trials_us_per_call"],
        "graph_us_per_call": prim["graph_us_per_call"],
        "kernel_event_us": prim["kernel_event_us"],
        "launch_floor_us": round(floor, 3),
        "store_floor_us": round(store_floor, 3),
        "read_floor": prim["read_floor"],
        "pct_of_read_floor": prim["pct_of_read_floor"],
        "roofline": prim["roofline"],
        "cpu_baseline": cpu,
        "parity_vs_oracle": parity,
        "secondary": sec,
        "all_configs": all_configs,
        "device": props.name,
    }
    if extra:
        rec["extra_workloads"] = extra
    print(json.dumps(rec), flush=True)
    return 0


if __name__ == "__main__":
    sys.exit(main())
