#!/usr/bin/env python3
"""Cold-cache benchmark of the block-quantized skinny GEMV on GB300.

Headline workload: bf16 GEMV M=1, K=4096, N=12288 (100.7 MB of weights per
call), the decode shape of "The Shape That Actually Matters".  Protocol
(that page, "The instrument came first"): R distinct weight buffers so the
working set is >= 1 GiB (far past the 129 MB L2), a warm-up of >= 1 s on
the same rotation, then the timed launches split into repeats; a run whose
per-repeat spread is >= 5% of the mean is flagged.  Launches are captured
in a CUDA graph (one graph node per call, rotating through the buffers)
and timed with CUDA events on the launching stream.

One JSON line is printed (rank 0).  Extra "arms" report the other M=1
formats (q8_0, q4_0 x q8_1) and, with --suite full, every configuration.

    python bench.py [--gpus N] [--steps K] [--warmup W] [--impl ours|reference]
                    [--suite headline|full] [--pdl 0|1]
"""
from __future__ import annotations

import argparse
import ctypes
import hashlib
import json
import math
import os
import re
import statistics
import subprocess
import sys
import threading
import time

import numpy as np

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

K_HEAD, N_HEAD = 4096, 12288
GiB = 1 << 30


# ---------------------------------------------------------------------------
# helpers
# ---------------------------------------------------------------------------
def measured_peaks():
    p = os.path.join(ROOT, "MEASURED_PEAKS.json")
    if os.path.exists(p):
        d = json.load(open(p))
        return {"hbm_gbs": d["hbm_gbs"], "bf16_tflops": d["bf16_tflops"],
                "bf16_tflops_sustained": d.get("bf16_tflops_sustained"), "source": "measured"}
    return {"hbm_gbs": 6800.0, "bf16_tflops": 1900.0, "bf16_tflops_sustained": 1700.0, "source": "fallback"}


CSRC = os.path.join(ROOT, "block_quantized_gemv_gb300", "csrc")
# translation unit of a kernel key's kernels (the first prefix that fits)
KERNEL_SOURCE = (("gemm_", "bqg_gemm.cu"), ("decode_layer_", "bqg_layer.cu"), ("gemv_q4_0_q8_1_", "gemv_q4_0_q8_1.cu"),
                 ("gemv_q4_0_", "gemv_q4_0.cu"), ("gemv_q8_0_", "gemv_q8_0.cu"), ("gemv_bf16_", "gemv_bf16.cu"))


def source_hash(kernel_key, csrc=CSRC):
    """Hash of the sources that kernel_key's kernels are compiled from: their
    translation unit and the headers of csrc/ it includes, directly or not."""
    todo = [next(tu for prefix, tu in KERNEL_SOURCE if kernel_key.startswith(prefix))]
    texts = {}
    while todo:
        name = todo.pop()
        if name not in texts:
            texts[name] = open(os.path.join(csrc, name), "rb").read()
            todo += [n.decode() for n in re.findall(rb'^#include "([^"/]+)"', texts[name], re.M)]
    h = hashlib.sha256()
    for name in sorted(texts):
        h.update(texts[name])
    return h.hexdigest()[:16]


def profiled_traffic(kernel_key):
    """DRAM bytes per launch from the committed ncu summary, if the kernel's
    own sources have not changed since it was taken (else None)."""
    p = os.path.join(ROOT, "profiles", "traffic.json")
    if not os.path.exists(p):
        return None
    d = json.load(open(p))
    e = d.get(kernel_key)
    if not e or e.get("source_hash") != source_hash(kernel_key):
        return None
    return e.get("dram_bytes_per_launch")


def max_over_ranks(value, dist, device="cuda"):
    """The largest `value` over all ranks (every rank receives it); `value`
    itself on a single process.  The timed region of a replica run is the
    slowest rank's."""
    if dist is None:
        return value
    import torch
    t = torch.tensor([float(value)], dtype=torch.float64, device=device)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    return float(t.item())


def whole_job_gbs(bytes_per_call, calls_per_rank, world, seconds):
    """Whole-job throughput: every rank's bytes over the slowest rank's time."""
    return bytes_per_call * calls_per_rank * world / seconds / 1e9


# The instrument of "The Shape That Actually Matters", "The instrument came
# first": 200 timed launches per repeat, 10 repeats, and no number unless the
# spread of the repeat means is below 5 % of their mean.
REPEATS = 10
MIN_LAUNCHES_PER_REPEAT = 200
MAX_SPREAD = 0.05
ATTEMPTS = 3            # the measurement and at most two re-measurements


def protocol_launches(steps):
    """(repeats, launches per repeat) for a run asked for `steps` timed
    calls: always 10 repeats of at least 200 launches; more launches per
    repeat when `steps` asks for more."""
    return REPEATS, max(MIN_LAUNCHES_PER_REPEAT, -(-int(steps) // REPEATS))


class NvmlSampler:
    """Samples SM clock, temperature, power and clock-event reasons through
    NVML (read-only calls only)."""

    REASONS = {0x1: "gpu_idle", 0x2: "applications_clocks_setting", 0x4: "sw_power_cap",
               0x8: "hw_slowdown", 0x10: "sync_boost", 0x20: "sw_thermal_slowdown",
               0x40: "hw_thermal_slowdown", 0x80: "hw_power_brake_slowdown"}

    def __init__(self, uuid: str | None):
        self.ok = False
        self.samples = []
        self.max_mhz = None
        try:
            self.nv = ctypes.CDLL("libnvidia-ml.so.1")
            if self.nv.nvmlInit_v2() != 0:
                return
            self.h = ctypes.c_void_p()
            if uuid and self.nv.nvmlDeviceGetHandleByUUID(uuid.encode(), ctypes.byref(self.h)) == 0:
                pass
            elif self.nv.nvmlDeviceGetHandleByIndex_v2(0, ctypes.byref(self.h)) != 0:
                return
            mx = ctypes.c_uint(0)
            if self.nv.nvmlDeviceGetMaxClockInfo(self.h, 1, ctypes.byref(mx)) == 0:
                self.max_mhz = mx.value
            self.reason_fn = getattr(self.nv, "nvmlDeviceGetCurrentClocksEventReasons", None) or \
                getattr(self.nv, "nvmlDeviceGetCurrentClocksThrottleReasons")
            self.ok = True
        except (OSError, AttributeError):
            self.ok = False

    def _loop(self):
        clk, rs = ctypes.c_uint(0), ctypes.c_ulonglong(0)
        temp, mw = ctypes.c_uint(0), ctypes.c_uint(0)
        while not self._stop.is_set():
            if self.nv.nvmlDeviceGetClockInfo(self.h, 1, ctypes.byref(clk)) == 0 and \
                    self.reason_fn(self.h, ctypes.byref(rs)) == 0:
                t = temp.value if self.nv.nvmlDeviceGetTemperature(self.h, 0, ctypes.byref(temp)) == 0 else None
                w = mw.value / 1000.0 if self.nv.nvmlDeviceGetPowerUsage(self.h, ctypes.byref(mw)) == 0 else None
                self.samples.append((clk.value, rs.value, t, w))
            time.sleep(0.001)

    def start(self):
        """Start a fresh record (samples of an earlier region are dropped)."""
        if not self.ok:
            return
        self.samples = []
        self._stop = threading.Event()
        self._t = threading.Thread(target=self._loop, daemon=True)
        self._t.start()

    def stop(self):
        if not self.ok:
            return
        self._stop.set()
        self._t.join()

    def summary(self):
        if not self.samples:
            return {"sm_mhz": None, "sm_max_mhz": self.max_mhz, "reasons": [], "samples": 0,
                    "source": "nvml" if self.ok else "unavailable"}
        mhz = [c for c, _, _, _ in self.samples]
        temps = [t for _, _, t, _ in self.samples if t is not None]
        watts = [w for _, _, _, w in self.samples if w is not None]
        mask = 0
        for _, r, _, _ in self.samples:
            mask |= r
        reasons = [n for b, n in self.REASONS.items() if mask & b and n != "gpu_idle"]
        return {"sm_mhz": statistics.median(mhz), "sm_mhz_min": min(mhz), "sm_max_mhz": self.max_mhz,
                "temp_c_max": max(temps) if temps else None,
                "power_w_median": round(statistics.median(watts), 1) if watts else None,
                "power_w_max": round(max(watts), 1) if watts else None,
                "reasons": reasons, "samples": len(self.samples), "source": "nvml"}


# ---------------------------------------------------------------------------
# workloads ("arms")
# ---------------------------------------------------------------------------
_W_CACHE = {}


def cached_weights(N, K, seed):
    """synth.weights_f32(N, K, seed), remembered for the next arm of the same
    shape (the sweep's formats share their fp32 weights); one entry."""
    from block_quantized_gemv_gb300 import synth
    key = (N, K, seed)
    if key not in _W_CACHE:
        _W_CACHE.clear()
        _W_CACHE[key] = synth.weights_f32(N, K, seed)
    return _W_CACHE[key]


class Arm:
    """One call = one pass over one weight set; `sets` rotate."""
    name = ""
    launches_per_call = 1
    kernel_key = ""

    def __init__(self):
        self.sets = []

    @staticmethod
    def rotation(bytes_per_call):
        return max(10, math.ceil(GiB / bytes_per_call))


class GemvArm(Arm):
    def __init__(self, fmt, xfmt, M, N, K, seed=1, sets=None):
        import torch
        import block_quantized_gemv_gb300 as bqg
        from block_quantized_gemv_gb300 import synth
        super().__init__()
        self.bqg, self.torch = bqg, torch
        self.fmt, self.xfmt, self.M, self.N, self.K = fmt, xfmt, M, N, K
        names = {bqg.BF16: "bf16", bqg.Q8_0: "q8_0", bqg.Q4_0: "q4_0"}
        xs = "q8_1" if xfmt == bqg.Q8_1 else "bf16"
        self.name = f"{names[fmt]} x {xs} GEMV M={M} K={K} N={N}"
        self.kernel_key = f"gemv_{names[fmt]}_{xs}_M{M}_K{K}_N{N}"
        # weights: fp32 N(0, 0.02) -> (GPU encoder) -> canonical -> (GPU repack)
        Wf = torch.from_numpy(cached_weights(N, K, seed)).cuda()
        if fmt == bqg.BF16:
            canon = Wf.to(torch.bfloat16).view(torch.uint8).reshape(-1)
        else:
            canon = bqg.quantize_weights(fmt, Wf)
        Wp = bqg.repack_weights(fmt, canon, N, K)
        del Wf, canon
        x = torch.from_numpy(synth.activations_f32(M, K, seed + 1)).cuda().to(torch.bfloat16)
        X = bqg.quantize_q8_1(x) if xfmt == bqg.Q8_1 else x
        self.w_bytes = Wp.numel()
        self.x_bytes = X.numel() * X.element_size()
        self.y_bytes = M * N * 4
        self.bytes_per_call = self.w_bytes + self.x_bytes + self.y_bytes
        self.R = sets or self.rotation(self.bytes_per_call)
        self.fn = {bqg.BF16: bqg.gemv_bf16, bqg.Q8_0: bqg.gemv_q8_0, bqg.Q4_0: bqg.gemv_q4_0}[fmt]
        if xfmt == bqg.Q8_1:
            self.fn = bqg.gemv_q4_0_q8_1
        op = {"bf16": bqg.OP_GEMV_BF16, "q8_0": bqg.OP_GEMV_Q8_0, "q4_0": bqg.OP_GEMV_Q4_0}[names[fmt]]
        if xfmt == bqg.Q8_1:
            op = bqg.OP_GEMV_Q4_0_Q8_1
        self.route = bqg.ROUTE_NAMES[bqg.gemv_route(op, M, N, K)]
        for r in range(self.R):
            self.sets.append({"W": Wp if r == 0 else Wp.clone(), "X": X.clone(),
                              "Y": torch.empty((M, N), dtype=torch.float32, device="cuda"),
                              "ws": bqg.workspace(op, M, N, K)})
        self.X_host = torch.empty_like(X, device="cpu").pin_memory()
        self.X_host.copy_(X)
        self.Y_host = torch.empty((M, N), dtype=torch.float32).pin_memory()

    def call(self, i):
        s = self.sets[i % self.R]
        self.fn(s["W"], s["X"], self.N, self.K, out=s["Y"], ws=s["ws"])

    def call_e2e(self, i):
        """One step from pinned host memory to pinned host memory: the SMs
        pull x over the CPU-GPU link into this set's device buffer
        (bqg_copy_sm), and the GEMV writes y straight into the pinned host
        buffer (its host alias)."""
        s = self.sets[i % self.R]
        self.bqg.copy_sm(s["X"], self.X_host)
        self.fn(s["W"], s["X"], self.N, self.K, out=self.Y_host, ws=s["ws"])

    def call_e2e_copy_engine(self, i):
        """The same step with copy-engine transfers (torch copies) on both sides."""
        s = self.sets[i % self.R]
        s["X"].copy_(self.X_host, non_blocking=True)
        self.fn(s["W"], s["X"], self.N, self.K, out=s["Y"], ws=s["ws"])
        self.Y_host.copy_(s["Y"], non_blocking=True)

    def flops_per_call(self):
        return 2 * self.M * self.N * self.K


class VendorGemvArm(Arm):
    """Context arm, not this library: torch.matmul (cuBLAS) bf16 y = x W^T at the
    same shape, rotation and timing as the bf16 GEMV arm (bf16 output, as the
    library call returns).  Its launches are not counted as ours."""
    vendor = True
    launches_per_call = 0

    def __init__(self, M=1, N=12288, K=4096, seed=1):
        import torch
        from block_quantized_gemv_gb300 import synth
        super().__init__()
        self.M, self.N, self.K = M, N, K
        self.name = f"vendor arm: torch.matmul (cuBLAS) bf16 GEMV M={M} K={K} N={N}"
        self.kernel_key = ""
        W = torch.from_numpy(cached_weights(N, K, seed)).cuda().to(torch.bfloat16)
        x = torch.from_numpy(synth.activations_f32(M, K, seed + 1)).cuda().to(torch.bfloat16)
        self.bytes_per_call = N * K * 2 + M * K * 2 + M * N * 2
        self.R = self.rotation(self.bytes_per_call)
        for r in range(self.R):
            self.sets.append({"W": W if r == 0 else W.clone(), "x": x.clone(),
                              "y": torch.empty((M, N), dtype=torch.bfloat16, device="cuda")})

    def call(self, i):
        import torch
        s = self.sets[i % self.R]
        torch.matmul(s["x"], s["W"].t(), out=s["y"])


class GemmArm(Arm):
    """Prefill GEMM M=512 (bf16 activations) x q4_0 (or q8_0) weights."""

    def __init__(self, M=512, N=14336, K=4096, seed=9, sets=None, fmt=None):
        import torch
        import block_quantized_gemv_gb300 as bqg
        from block_quantized_gemv_gb300 import synth
        super().__init__()
        self.bqg, self.M, self.N, self.K = bqg, M, N, K
        fmt = bqg.Q4_0 if fmt is None else fmt
        fname = "q8_0" if fmt == bqg.Q8_0 else "q4_0"
        self.fn = bqg.gemm_q8_0_bf16 if fmt == bqg.Q8_0 else bqg.gemm_q4_0_bf16
        self.name = f"{fname} x bf16 prefill GEMM M={M} K={K} N={N}"
        self.kernel_key = f"gemm_{fname}_bf16_M{M}_K{K}_N{N}"
        Wf = torch.from_numpy(cached_weights(N, K, seed)).cuda()
        Wp = bqg.repack_weights(fmt, bqg.quantize_weights(fmt, Wf), N, K)
        del Wf
        X = torch.from_numpy(synth.activations_f32(M, K, seed + 1)).cuda().to(torch.bfloat16)
        self.bytes_per_call = Wp.numel() + X.numel() * 2 + M * N * 4
        self.flops = 2.0 * M * N * K
        self.R = sets or self.rotation(self.bytes_per_call)
        for r in range(self.R):
            self.sets.append({"W": Wp if r == 0 else Wp.clone(), "X": X.clone(),
                              "Y": torch.empty((M, N), dtype=torch.float32, device="cuda")})
        self.X_host = X.cpu().pin_memory()
        self.Y_host = torch.empty((M, N), dtype=torch.float32).pin_memory()

    def call(self, i):
        s = self.sets[i % self.R]
        self.fn(s["W"], s["X"], self.N, self.K, out=s["Y"])

    def call_e2e(self, i):
        s = self.sets[i % self.R]
        s["X"].copy_(self.X_host, non_blocking=True)
        self.call(i)
        self.Y_host.copy_(s["Y"], non_blocking=True)


class DecodeLayerArm(Arm):
    """q4_0 x q8_1 decode layer: quantize(x), QKV, gate+up+SwiGLU, quantize(h), down.
    With fused_norm the layer starts from the raw activation row: its first
    step is the fused RMSNorm -> q8_1 encoder, and the gate+up epilogue writes
    h as q8_1 for the down projection (four launches instead of five).  With
    persistent the whole layer (q8_1 of x, QKV, gate+up+SwiGLU->q8_1, down) is
    one cooperative launch with a grid barrier before the down projection."""

    def __init__(self, seed=5, K=4096, Nq=4096, Nff=11008, fused_norm=False, persistent=False):
        import torch
        import block_quantized_gemv_gb300 as bqg
        from block_quantized_gemv_gb300 import synth
        super().__init__()
        self.bqg, self.torch = bqg, torch
        self.fused_norm, self.persistent = fused_norm, persistent
        self.name = (f"q4_0 x q8_1 decode layer M=1 (QKV 3x{Nq}x{K}, gate+up 2x{Nff}x{K}, down {K}x{Nff})"
                     + (", fused RMSNorm->q8_1 and SwiGLU->q8_1" if fused_norm else "")
                     + (", one persistent launch" if persistent else ""))
        self.kernel_key = ("decode_layer_q4_0_q8_1" + ("_fused_norm" if fused_norm else "")
                           + ("_persistent" if persistent else ""))
        self.launches_per_call = 1 if persistent else 4 if fused_norm else 5
        self.K, self.Nq, self.Nff = K, Nq, Nff

        def mk(N, KK, sd):
            Wf = torch.from_numpy(cached_weights(N, KK, sd)).cuda()
            return bqg.repack_weights(bqg.Q4_0, bqg.quantize_weights(bqg.Q4_0, Wf), N, KK)

        base = {"Wq": mk(Nq, K, seed), "Wk": mk(Nq, K, seed + 1), "Wv": mk(Nq, K, seed + 2),
                "Wg": mk(Nff, K, seed + 3), "Wu": mk(Nff, K, seed + 4), "Wd": mk(K, Nff, seed + 5)}
        w_bytes = sum(v.numel() for v in base.values())
        x = torch.from_numpy(synth.activations_f32(1, K, seed + 6) if fused_norm else
                             synth.rms_normalised_f32(1, K, seed + 6)).cuda().to(torch.bfloat16)
        self.bytes_per_call = (w_bytes + K * 2 + (K // 32) * 36 * 2 + 3 * Nq * 4 + Nff * 4 * 2 +
                               (Nff // 32) * 36 * 2 + K * 4)
        self.R = self.rotation(self.bytes_per_call)
        for r in range(self.R):
            s = {k: (v if r == 0 else v.clone()) for k, v in base.items()}
            s.update({"x": x.clone(), "xq": torch.empty((1, (K // 32) * 36), dtype=torch.uint8, device="cuda"),
                      "q": torch.empty((1, Nq), device="cuda"), "k": torch.empty((1, Nq), device="cuda"),
                      "v": torch.empty((1, Nq), device="cuda"), "h": torch.empty((1, Nff), device="cuda"),
                      "hq": torch.empty((1, (Nff // 32) * 36), dtype=torch.uint8, device="cuda"),
                      "y": torch.empty((1, K), device="cuda"),
                      "ws_qkv": bqg.workspace(bqg.OP_QKV_Q4_0_Q8_1, 1, 3 * Nq, K),
                      "ws_gu": bqg.workspace(bqg.OP_GATE_UP_Q8_1_Q4_0_Q8_1 if fused_norm else
                                             bqg.OP_GATE_UP_Q4_0_Q8_1, 1, Nff, K),
                      "ws_d": bqg.workspace(bqg.OP_GEMV_Q4_0_Q8_1, 1, K, Nff),
                      "ws_layer": bqg.workspace(bqg.OP_DECODE_LAYER_Q4_0_Q8_1, 1, Nff, K) if persistent else None})
            self.sets.append(s)
        self.x_host = x.cpu().pin_memory()
        self.y_host = torch.empty((1, K), dtype=torch.float32).pin_memory()

    def call(self, i):
        b, s = self.bqg, self.sets[i % self.R]
        if self.persistent:
            b.decode_layer_q4_0_q8_1(s["x"], s["x"], s["Wq"], s["Wk"], s["Wv"], s["Wg"], s["Wu"], s["Wd"], self.Nq,
                                     self.Nq, self.Nff, self.K, out=(s["q"], s["k"], s["v"], s["y"]),
                                     ws=s["ws_layer"])
            return
        if self.fused_norm:
            b.rmsnorm_quantize_q8_1(s["x"], None, 1e-5, out=s["xq"])
        else:
            b.quantize_q8_1(s["x"], out=s["xq"])
        b.gemv_q4_0_q8_1_qkv(s["Wq"], s["Wk"], s["Wv"], s["xq"], self.Nq, self.Nq, self.K,
                             out=(s["q"], s["k"], s["v"]), ws=s["ws_qkv"])
        if self.fused_norm:
            b.gemv_q4_0_q8_1_gate_up_swiglu_q8_1(s["Wg"], s["Wu"], s["xq"], self.Nff, self.K, out=s["hq"],
                                                 ws=s["ws_gu"])
        else:
            b.gemv_q4_0_q8_1_gate_up_swiglu(s["Wg"], s["Wu"], s["xq"], self.Nff, self.K, out=s["h"], ws=s["ws_gu"])
            b.quantize_q8_1(s["h"], out=s["hq"])
        b.gemv_q4_0_q8_1(s["Wd"], s["hq"], self.K, self.Nff, out=s["y"], ws=s["ws_d"])

    def call_e2e(self, i):
        s = self.sets[i % self.R]
        s["x"].copy_(self.x_host, non_blocking=True)
        self.call(i)
        self.y_host.copy_(s["y"], non_blocking=True)


# ---------------------------------------------------------------------------
# timing
# ---------------------------------------------------------------------------
def time_arm(arm, steps, warmup, use_graph=True, min_warm_s=1.0, sampler=None, dist=None):
    """One measurement of `arm` under the protocol: 10 repeats of L >= 200
    launches (one CUDA graph of L calls rotating through the buffer sets, so
    every call streams its inputs from HBM), warm-up of at least `warmup`
    calls and `min_warm_s` seconds on the same rotation, CUDA events on the
    launching stream around each repeat, NVML sampled over the timed region."""
    import torch
    repeats, L = protocol_launches(steps)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for i in range(min(arm.R, 4)):           # populate plan caches eagerly
            arm.call(i)
    torch.cuda.synchronize()
    graph = None
    if use_graph:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            for i in range(L):
                arm.call(i)
        torch.cuda.synchronize()

    def run_once():
        if graph is not None:
            graph.replay()
        else:
            for i in range(L):
                arm.call(i)

    with torch.cuda.stream(stream):
        t0 = time.perf_counter()
        done = 0
        while done < warmup or time.perf_counter() - t0 < min_warm_s:
            run_once()
            done += L
            if done % (50 * L) == 0:
                stream.synchronize()
        stream.synchronize()
    times = []
    if dist is not None:
        dist.barrier()
    torch.cuda.synchronize()
    if sampler:
        sampler.start()
    ev = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)) for _ in range(repeats)]
    with torch.cuda.stream(stream):
        for a, b in ev:
            a.record(stream)
            run_once()
            b.record(stream)
    stream.synchronize()
    torch.cuda.synchronize()
    if sampler:
        sampler.stop()
    times = [a.elapsed_time(b) / 1e3 for a, b in ev]     # seconds per repeat
    total = max_over_ranks(sum(times), dist)
    mean = statistics.mean(times)
    spread = (max(times) - min(times)) / mean if mean > 0 else 0.0
    spread = max_over_ranks(spread, dist)
    del graph
    return {"seconds": total, "per_repeat_s": times, "repeats": repeats, "launches_per_repeat": L,
            "timed_calls": repeats * L, "spread": spread, "spread_ok": spread < MAX_SPREAD,
            "graph": use_graph, "clocks": sampler.summary() if sampler else None}


def measure(arm, steps, warmup, **kw):
    """time_arm under the rejection rule: re-measured while the repeat spread
    is >= 5 %, at most ATTEMPTS times in all; the last attempt is returned
    with `rejected` set when its spread still fails."""
    spreads = []
    for _ in range(ATTEMPTS):
        t = time_arm(arm, steps, warmup, **kw)
        spreads.append(round(t["spread"], 4))
        if t["spread_ok"]:
            break
    t["attempt_spreads"] = spreads
    t["rejected"] = not t["spread_ok"]
    return t


def time_e2e(arm, steps, step_fn=None):
    """Device time of `steps` end-to-end steps enqueued back to back (CUDA
    events on the launching stream)."""
    import torch
    step = step_fn or arm.call_e2e
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for i in range(3):
            step(i)
        stream.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record(stream)
        for i in range(steps):
            step(i)
        b.record(stream)
        stream.synchronize()
    return a.elapsed_time(b) / 1e3


def time_e2e_host(arm, steps, step_fn=None):
    """Host-clock time per step of a decode loop: every step is the binding
    call(s) from pinned x to pinned y followed by a stream synchronize, timed
    with time.perf_counter (the latency an autoregressive host loop sees,
    host launch cost included).  Returns the median and mean seconds per step."""
    import torch
    step = step_fn or arm.call_e2e
    stream = torch.cuda.Stream()
    per = []
    with torch.cuda.stream(stream):
        for i in range(5):
            step(i)
            stream.synchronize()
        for i in range(steps):
            t0 = time.perf_counter()
            step(i)
            stream.synchronize()
            per.append(time.perf_counter() - t0)
    return statistics.median(per), statistics.mean(per)


def gb_s(bytes_, seconds):
    return bytes_ / seconds / 1e9


def arm_record(arm, t, peaks):
    """The arm's record.  A rejected measurement (repeat spread still >= 5 %
    after the re-measurements) carries no rate: only its spreads."""
    calls = t["repeats"] * t["launches_per_repeat"]
    rec = {"workload": arm.name, "bytes_per_call": arm.bytes_per_call,
           "rotating_sets": arm.R, "working_set_bytes": arm.R * arm.bytes_per_call,
           "repeats": t["repeats"], "launches_per_repeat": t["launches_per_repeat"], "timed_calls": calls,
           "spread": round(t["spread"], 4), "spread_ok": t["spread_ok"],
           "attempt_spreads": t.get("attempt_spreads"), "rejected": t.get("rejected", not t["spread_ok"]),
           "launches": calls * arm.launches_per_call, "clocks": t.get("clocks")}
    if getattr(arm, "vendor", False):
        rec["vendor"] = "library GEMV for context (cuBLAS through torch.matmul), not this repository's kernels"
    if getattr(arm, "route", None):
        rec["route"] = arm.route
    if rec["rejected"]:
        return rec
    us = t["seconds"] / calls * 1e6
    gbs = gb_s(arm.bytes_per_call * calls, t["seconds"])
    rec.update({"us_per_call": round(us, 3), "GB_per_s": round(gbs, 1), "frac_of_peak": round(gbs / peaks["hbm_gbs"], 4)})
    if getattr(arm, "flops", None):
        tf = arm.flops * calls / t["seconds"] / 1e12
        rec.update({"bound": "tensor", "TFLOP_per_s": round(tf, 1),
                    "frac_of_tensor_peak": round(tf / peaks["bf16_tflops"], 4),
                    "peak_note": "dense bf16 burst peak, MEASURED_PEAKS.json bf16_tflops"})
        del rec["frac_of_peak"]
    return rec


# ---------------------------------------------------------------------------
# the CPU oracle (baseline and reference arm)
# ---------------------------------------------------------------------------
def _oracle_headline_inputs():
    from block_quantized_gemv_gb300 import synth
    W = synth.bf16_bits(synth.weights_f32(N_HEAD, K_HEAD, 1))
    X = synth.bf16_bits(synth.activations_f32(1, K_HEAD, 2))
    return W, X


def oracle_gemv_sample(rows_per_step, steps, budget_s=None):
    """Time the fp64 oracle on the headline workload, `rows_per_step` rows per
    step (a different slice every step), OpenMP over rows on every core."""
    import oracle
    ora = oracle.default()
    W, X = _oracle_headline_inputs()
    threads = max(1, os.cpu_count() or 1)
    rng = np.random.default_rng(0)
    starts = rng.integers(0, N_HEAD - rows_per_step + 1, size=max(1, steps))
    ora.gemv(oracle.BF16, W, oracle.BF16, X, 1, N_HEAD, K_HEAD, rows=np.arange(min(64, N_HEAD)), nthreads=threads)
    t0 = time.perf_counter()
    done = 0
    for i in range(steps):
        rows = np.arange(starts[i], starts[i] + rows_per_step)
        ora.gemv(oracle.BF16, W, oracle.BF16, X, 1, N_HEAD, K_HEAD, rows=rows, nthreads=threads)
        done += 1
        if budget_s is not None and time.perf_counter() - t0 > budget_s:
            break
    dt = time.perf_counter() - t0
    bytes_per_row = K_HEAD * 2 + 4
    total = done * rows_per_step * bytes_per_row + done * K_HEAD * 2
    return {"value": round(gb_s(total, dt), 4), "unit": "GB/s", "cores": ora.openmp_threads() if threads > 1 else 1,
            "threads_used": threads, "seconds": dt, "steps": done, "rows_per_step": rows_per_step}


def oracle_baseline(runs=5, run_s=1.0):
    """The oracle as it stands, timed on the host's cores in both of its
    modes: one thread, and OpenMP over output rows on every core (each row's
    fp64 sum keeps its order, so both give the same results).  A run is as
    many whole headline GEMVs (12288 x 4096 bf16) as fit in about `run_s`
    seconds (at least one); each mode reports the median of `runs` runs."""
    import oracle
    ora = oracle.default()
    W, X = _oracle_headline_inputs()
    bytes_per_call = N_HEAD * K_HEAD * 2 + K_HEAD * 2 + N_HEAD * 4
    cores = os.cpu_count() or 1
    modes = {}
    for name, threads in (("single_thread", 1), ("openmp", cores)):
        rates, calls_per_run = [], []
        for _ in range(runs):
            t0 = time.perf_counter()
            n = 0
            while n == 0 or time.perf_counter() - t0 < run_s:
                ora.gemv(oracle.BF16, W, oracle.BF16, X, 1, N_HEAD, K_HEAD, nthreads=threads)
                n += 1
            dt = time.perf_counter() - t0
            rates.append(gb_s(bytes_per_call * n, dt))
            calls_per_run.append(n)
        med = statistics.median(rates)
        modes[name] = {"value": round(med, 4), "unit": "GB/s", "threads": threads,
                       "us_per_call": round(bytes_per_call / (med * 1e9) * 1e6, 1),
                       "runs": [round(r, 4) for r in rates], "calls_per_run": calls_per_run}
    return {"value": modes["openmp"]["value"], "unit": "GB/s", "cores": cores, "kind": "oracle",
            "sample": f"whole headline GEMVs (12288 x 4096 bf16 weights) of the fp64 C oracle, runs of about "
                      f"{run_s:g} s, median of {runs} runs per mode; value = the OpenMP mode on all "
                      f"{cores} host cores (os.cpu_count())",
            "modes": modes}


# ---------------------------------------------------------------------------
# main
# ---------------------------------------------------------------------------
def headline_config():
    """The workload both arms (this library and the oracle) report."""
    return {"workload": f"bf16 GEMV M=1 K={K_HEAD} N={N_HEAD}", "M": 1, "K": K_HEAD, "N": N_HEAD,
            "weights": "bf16 N(0,0.02), activation bf16 N(0,1), fp32 output"}


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=2000)
    ap.add_argument("--warmup", type=int, default=200)
    ap.add_argument("--impl", choices=["ours", "reference"], default="ours")
    ap.add_argument("--suite", choices=["headline", "full"], default="full",
                    help="full (default): every configuration; headline: the M=1 K=4096 N=12288 arms, "
                         "the prefill GEMM and the vendor arm")
    ap.add_argument("--pdl", type=int, default=1)
    ap.add_argument("--no-graph", action="store_true")
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--json-out", default=None)
    ap.add_argument("--min-warm-s", type=float, default=1.0, help="minimum warm-up time per arm")
    ap.add_argument("--profile", default=None,
                    help="profiling case, 2 weight sets, eager calls: gemm, or a GEMV arm bf16 | q8_0 | "
                         "q4_0 | q4_0_q8_1 (M=1 K=4096 N=12288), optionally ':<N>x<M>' (K=4096)")
    args = ap.parse_args()

    world = int(os.environ.get("WORLD_SIZE", "1"))
    rank = int(os.environ.get("RANK", "0"))
    local = int(os.environ.get("LOCAL_RANK", "0"))

    headline_metric = "cold-cache HBM GB/s (% of peak) and µs/call, GEMV M=1 K=4096 N=12288"

    if args.impl == "reference":
        if rank != 0:
            return 0
        r = oracle_gemv_sample(N_HEAD, args.steps + args.warmup)
        out = {"impl": "reference", "metric": headline_metric, "value": r["value"], "unit": "GB/s",
               "n_gpus": args.gpus, "steps": args.steps, "warmup": args.warmup,
               "ms_per_step": round(r["seconds"] / max(1, r["steps"]) * 1e3, 4),
               "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "f64",
               "data": "synthetic", "config": headline_config(),
               "reference": "the CPU oracle (fp64, plain C, OpenMP over rows), the only implementation of the "
                            "pages' definition: the pages publish no code",
               "cpu_baseline": {"kind": "oracle", "value": r["value"], "unit": "GB/s", "cores": r["threads_used"],
                                "sample": f"{r['steps']} whole GEMVs (12288 x 4096 bf16 weights), one per step, "
                                          f"warm-up included in the count ({args.warmup} + {args.steps})"},
               "e2e": {"value": r["value"], "unit": "GB/s", "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0}}
        print(json.dumps(out))
        return 0

    import torch
    dist = None
    if world > 1:
        import torch.distributed as tdist
        torch.cuda.set_device(local)
        tdist.init_process_group("nccl", device_id=torch.device("cuda", local))
        dist = tdist
    torch.cuda.set_device(local)
    from block_quantized_gemv_gb300 import build as bqg_build
    import block_quantized_gemv_gb300 as bqg
    bqg_build.build()
    bqg.load()
    bqg.set_pdl(bool(args.pdl))
    peaks = measured_peaks()
    props = torch.cuda.get_device_properties(local)
    uuid = None
    try:
        u = str(props.uuid)
        uuid = u if u.startswith("GPU-") else "GPU-" + u
    except Exception:
        pass
    sampler = NvmlSampler(uuid)

    if args.profile == "gemm":
        arm = GemmArm(sets=2)
        for i in range(args.warmup + args.steps):
            arm.call(i)
        torch.cuda.synchronize()
        print(json.dumps({"profile": arm.name, "calls": args.warmup + args.steps}))
        return 0
    if args.profile:
        # a small case for ncu: two weight sets (cache state is ncu's to control);
        # "<fmt>" is the headline shape, "<fmt>:<N>x<M>" another (K = 4096)
        name, shape = (args.profile.split(":") + [f"{N_HEAD}x1"])[:2]
        n_rows, m_rows = map(int, shape.split("x"))
        fmt = {"bf16": bqg.BF16, "q8_0": bqg.Q8_0, "q4_0": bqg.Q4_0, "q4_0_q8_1": bqg.Q4_0}[name]
        xf = bqg.Q8_1 if name == "q4_0_q8_1" else bqg.BF16
        arm = GemvArm(fmt, xf, m_rows, n_rows, K_HEAD, sets=2)
        for i in range(args.warmup + args.steps):
            arm.call(i)
        torch.cuda.synchronize()
        print(json.dumps({"profile": arm.name, "calls": args.warmup + args.steps}))
        return 0

    head = GemvArm(bqg.BF16, bqg.BF16, 1, N_HEAD, K_HEAD)
    kw = dict(use_graph=not args.no_graph, sampler=sampler, dist=dist)
    t = measure(head, args.steps, args.warmup, min_warm_s=args.min_warm_s, **kw)
    rec = arm_record(head, t, peaks)
    calls = t["timed_calls"]
    rejected = t["rejected"]
    value = None if rejected else whole_job_gbs(head.bytes_per_call, calls, world, t["seconds"])

    e2e_steps = max(args.steps, MIN_LAUNCHES_PER_REPEAT)
    e2e_s = time_e2e(head, e2e_steps)
    ce_s = time_e2e(head, e2e_steps, head.call_e2e_copy_engine)
    host_med, host_mean = time_e2e_host(head, e2e_steps)
    host_ce_med, _ = time_e2e_host(head, e2e_steps, head.call_e2e_copy_engine)
    e2e = {"value": round(gb_s(head.bytes_per_call * e2e_steps, e2e_s), 1), "unit": "GB/s",
           "h2d_bytes_per_step": head.x_bytes, "d2h_bytes_per_step": head.y_bytes,
           "steps": e2e_steps, "us_per_step": round(e2e_s / e2e_steps * 1e6, 3),
           "timing": "CUDA events around the steps enqueued back to back on one stream",
           "host_us_per_step": round(host_med * 1e6, 3), "host_us_per_step_mean": round(host_mean * 1e6, 3),
           "host_value": round(gb_s(head.bytes_per_call, host_med), 1),
           "host_timing": "time.perf_counter around each step (binding calls, then stream.synchronize): "
                          "the per-token latency a host decode loop sees, median over the steps",
           "path": "through the Python binding, every step: x from pinned host memory into device memory by "
                   "bqg_copy_sm (SM loads over the CPU-GPU link), bqg_gemv_bf16 writing y straight into pinned "
                   "host memory (bqg_host_alias); the host reads y there after the final synchronize",
           "copy_engine": {"value": round(gb_s(head.bytes_per_call * e2e_steps, ce_s), 1), "unit": "GB/s",
                           "us_per_step": round(ce_s / e2e_steps * 1e6, 3),
                           "host_us_per_step": round(host_ce_med * 1e6, 3),
                           "path": "the same step with torch copies (copy-engine transfers) of x in and y out"}}

    arms = [rec]
    specs = [lambda: GemvArm(bqg.Q8_0, bqg.BF16, 1, N_HEAD, K_HEAD),
             lambda: GemvArm(bqg.Q4_0, bqg.Q8_1, 1, N_HEAD, K_HEAD),
             lambda: GemmArm(), lambda: VendorGemvArm(1, N_HEAD, K_HEAD)]
    if args.suite == "full":
        specs += [lambda: GemmArm(fmt=bqg.Q8_0), lambda: GemvArm(bqg.Q8_0, bqg.BF16, 1, 4096, 4096),
                  lambda: DecodeLayerArm(), lambda: DecodeLayerArm(fused_norm=True),
                  lambda: DecodeLayerArm(persistent=True)]
        for M in (1, 2, 4, 8):
            for f in (bqg.BF16, bqg.Q8_0, bqg.Q4_0):
                specs.append(lambda M=M, f=f: GemvArm(f, bqg.BF16, M, 14336, 4096))
            specs.append(lambda M=M: GemvArm(bqg.Q4_0, bqg.Q8_1, M, 14336, 4096))
    launches_all = calls * head.launches_per_call
    for mk in specs:
        a = mk()
        ta = measure(a, args.steps, max(3, args.warmup // 4), min_warm_s=min(0.3, args.min_warm_s), **kw)
        r = arm_record(a, ta, peaks)
        arms.append(r)
        launches_all += r["launches"]
        del a
        torch.cuda.empty_cache()

    cpu = None
    if rank == 0 and world == 1 and not args.no_cpu_baseline:
        cpu = oracle_baseline()

    traffic = profiled_traffic(head.kernel_key)
    knobs = {k: v for k, v in sorted(os.environ.items()) if k.startswith("BQG_")}
    out = {
        "metric": headline_metric,
        "value": None if value is None else round(value, 1),
        "unit": "GB/s",
        "n_gpus": world,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": None if rejected else round(t["seconds"] / calls * 1e3, 6),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "bf16",
        "data": "synthetic",
        "rejected": rejected,
        "timed_launches": calls,
        "config": headline_config(),
        "protocol": {"step": "one GEMV call (one pass of the path over one activation row)",
                     "repeats": t["repeats"], "launches_per_repeat": t["launches_per_repeat"],
                     "timed_calls": calls, "spread": round(t["spread"], 4), "spread_ok": t["spread_ok"],
                     "attempt_spreads": t["attempt_spreads"], "max_spread": MAX_SPREAD,
                     "rotating_weight_sets": head.R, "working_set_bytes": head.R * head.bytes_per_call,
                     "l2_bytes": props.L2_cache_size,
                     "cold_cache": "inputs larger than L2: rotating buffer sets, >= 1 GiB working set",
                     "timing": "CUDA graph of the launches of a repeat, CUDA events on the launching stream",
                     "us_per_call": rec.get("us_per_call"),
                     "parallelism": "replicas" if world > 1 else "single GPU"},
        "library": {"pdl": bool(args.pdl), "env_knobs": knobs, "version": bqg.version()},
        "roofline": None if rejected else {
            "bound": "hbm", "achieved": rec["GB_per_s"], "peak": peaks["hbm_gbs"], "unit": "GB/s",
            "frac": round(rec["GB_per_s"] / peaks["hbm_gbs"], 4), "traffic": traffic,
            "peak_source": peaks["source"] + " (MEASURED_PEAKS.json hbm_gbs, copy bandwidth)",
            "algorithmic_bytes_per_launch": head.bytes_per_call},
        "cpu_baseline": cpu,
        "e2e": e2e,
        "gpu_launches": calls * head.launches_per_call,
        "gpu_launches_all_arms": launches_all,
        "clocks": t["clocks"],
        "arms": arms,
    }
    if rank == 0:
        line = json.dumps(out)
        print(line)
        if args.json_out:
            with open(args.json_out, "w") as f:
                f.write(line + "\n")
    if dist is not None:
        dist.barrier()
        dist.destroy_process_group()
    return 0


if __name__ == "__main__":
    sys.exit(main())
