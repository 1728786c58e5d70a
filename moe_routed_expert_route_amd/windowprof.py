"""Profiles of the calls on windows: a program to run under rocprofv3, and the table of its trace.

    rocprofv3 --kernel-trace --output-format csv -d DIR -o run -- python3 -m moe_routed_expert_route_amd.windowprof run
    rocprofv3 --pmc FETCH_SIZE --kernel-trace --output-format csv -d DIR1 -o run -- \\
        python3 -m moe_routed_expert_route_amd.windowprof run --counters
    python -m moe_routed_expert_route_amd.windowprof table --trace DIR/run_kernel_trace.csv \\
        --counters DIR1/run_counter_collection.csv ... --command "..."

`run` makes PASSES passes of each case that perf/more_operators.py lists and of those in MORE, on two inputs in
turn; first as they come (small inputs are in a cache then), then each after 1 GiB was read, which leaves none of
them there. A streaming read stands before each pass and marks where it begins. `table` writes
profiles/kernels_window.md: the library's launches alone, medians, registers and scratch as the trace has them, and the
counters per launch (--counters: one pass of the cases in COUNTED, after a copy of known size).
"""
from __future__ import annotations

import argparse
import csv
import hashlib
import os
import re
import statistics
from collections import defaultdict

from . import profsum

SOURCES = ("moe_routed_expert_route_amd/csrc/moe_window.hip", "moe_routed_expert_route_amd/csrc/moe_rows.hpp",
           "moe_routed_expert_route_amd/csrc/moe_device.hpp", "moe_routed_expert_route_amd/build.py", "perf/more_operators.py")
PASSES = 10
CALIB_BYTES = 256 << 20
MARK = "moe::k_stream_read"
# (a listed case, what differs): what the listed ones leave out
MORE = [("append 8x1024 bf16", dict(cache="i8"), "append 8x1024 bf16 into i8"),
        ("append 8x1024 bf16", dict(seqs=1, T=1000), "append 1x1000 bf16"),
        ("append 1x1 bf16", dict(seqs=1000), "append 1000x1 bf16"),
        ("append 1x1 bf16", dict(seqs=4096, lo=100, hi=100), "append 4096x1 bf16"),
        ("attend 1x1 4096 bf16", dict(lo=131071, hi=131071), "attend 1x1 131072 bf16"),
        ("attend 1x1 4096 bf16", dict(seqs=1024, lo=16, hi=900, kv=8), "attend 1024x1 900 bf16"),
        ("attend 1x1 4096 bf16", dict(seqs=4096, lo=16, hi=200, kv=8), "attend 4096x1 200 bf16"),
        ("attend 64x4 8192 i8", dict(cache="bf16"), "attend 64x4 8192 bf16"),
        ("attend 64x4 8192 i8", dict(T=8), "attend 64x8 8192 i8"),
        ("attend 64x4 8192 i8", dict(d=256, seqs=32), "attend 32x4 8192 i8 of 256"),
        ("attend 1x4 131072 bf16", dict(d=256), "attend 1x4 131072 bf16 of 256"),
        ("attend 8x64 8192 f16", dict(type="bf16", cache="bf16"), "attend 8x64 8192 bf16"),
        ("attend 8x64 8192 f16", dict(type="bf16", cache="i8"), "attend 8x64 8192 bf16 over i8"),
        ("attend 8x64 8192 f16", dict(cache="i8"), "attend 8x64 8192 f16 over i8"),
        ("attend 8x64 8192 f16", dict(d=256), "attend 8x64 8192 f16 of 256"),
        ("logprobs 257x50021 f32 masked", dict(n=131072, extra=0), "logprobs 257x131072 f32 masked"),
        ("logprobs 1024x131072 bf16", dict(k=0), "logprobs 1024x131072 bf16, none best")]
COUNTED = ("append 8x1024 bf16", "attend 1x4 131072 bf16", "attend 64x4 8192 i8", "attend 8x64 8192 f16", "logprobs 1024x131072 bf16")


def cases():
    from perf import more_operators
    listed = more_operators.listed()
    by = {c["name"]: c for c in listed}
    return listed + [dict(by[name], **change, name=new) for name, change, new in MORE]


def source_digest() -> str:
    h = hashlib.sha256()
    for p in SOURCES:
        with open(os.path.join(profsum.ROOT, p), "rb") as f:
            h.update(f.read())
    return h.hexdigest()


def run(counters):
    import torch

    from perf import more_operators

    from . import binding as B
    more_operators.own = True
    if counters:
        src = torch.zeros(CALIB_BYTES, dtype=torch.uint8, device="cuda")
        torch.empty_like(src).copy_(src)
    other = torch.zeros(16 if counters else 1 << 30, dtype=torch.uint8, device="cuda")
    sums = torch.empty(1024, dtype=torch.int32, device="cuda")
    for case in cases():
        if counters and case["name"] not in COUNTED:
            continue
        states = [more_operators.prepare(case, seed) for seed in range(1 if counters else 2)]
        for cold in (False,) if counters else (False, True):
            for i in range(1 if counters else PASSES):
                B.moe_stream_read(other if cold else other[:16], sums, 1024 if cold else 1)   # a fill would leave lines to write back
                more_operators.run(states[i % len(states)])
        torch.cuda.synchronize()
        del states
        print(case["name"], flush=True)


def _name(kernel):
    return re.sub(r"moe::|^void |\(.*", "", kernel)


def passes(trace_csv):
    """The library's launches of each pass in order: lists of (kernel, workgroups, threads, start ns, end ns, scratch bytes)."""
    with open(trace_csv, newline="") as f:
        rows = [r for r in csv.DictReader(f) if "moe::k_" in r["Kernel_Name"]]
    rows.sort(key=lambda r: int(r["Start_Timestamp"]))
    out = []
    for r in rows:
        if MARK in r["Kernel_Name"]:
            out.append([])
        elif out:
            groups = 1
            for axis in "XYZ":
                groups *= int(r["Grid_Size_" + axis]) // int(r["Workgroup_Size_" + axis])
            out[-1].append((_name(r["Kernel_Name"]), groups, int(r["Workgroup_Size_X"]), int(r["Start_Timestamp"]),
                            int(r["End_Timestamp"]), int(r["Scratch_Size"])))
    return out


def counted(path):
    """counter -> per case in order: [(kernel, value) of each launch] (values of one dispatch summed over its rows)."""
    with open(path, newline="") as f:
        rows = list(csv.DictReader(f))
    out = {}
    for name in sorted({r["Counter_Name"] for r in rows}):
        per, kernel = defaultdict(float), {}
        for r in rows:
            if r["Counter_Name"] == name:
                per[int(r["Dispatch_Id"])] += float(r["Counter_Value"])
                kernel[int(r["Dispatch_Id"])] = r["Kernel_Name"]
        out[name] = []
        for d in sorted(per):
            if MARK in kernel[d]:
                out[name].append([])
            elif "moe::k_" in kernel[d] and out[name]:
                out[name][-1].append((_name(kernel[d]), per[d]))
    return out


def table(trace_csv, counter_csvs, command):
    from perf import more_operators
    mine, every = passes(trace_csv), cases()
    if len(mine) != 2 * PASSES * len(every):
        raise ValueError(f"{len(mine)} passes, not {2 * PASSES} of each of {len(every)} cases")
    lines = ["# Windows over a paged cache and log probabilities: the launches' own time", "", "Commands (repo root, one MI355X):", "",
             f"    {command}", "",
             f"The library's launches alone, medians of the last {PASSES - 2} of {PASSES} passes in µs: each kernel, and the sum of a pass; as "
             "they come (small inputs are in a cache), and cold, each after 1 GiB was read. GB/s and TFLOP/s go by the cold sum and by the bytes "
             "and operations that the case cannot do without.", "",
             "| case | kernels: workgroups × threads, µs (cold µs), scratch | µs | cold µs | GB/s | TFLOP/s |", "|---|---|---|---|---|---|"]
    for i, case in enumerate(every):
        part = mine[2 * PASSES * i:2 * PASSES * (i + 1)]
        if not part[0] or len({tuple(x[:3] for x in p) for p in part}) != 1:
            raise ValueError(f"{case['name']}: passes of different launches")
        warm, cold = ([[(x[4] - x[3]) / 1e3 for x in p] for p in half[2:]] for half in (part[:PASSES], part[PASSES:]))
        cells = []
        for j, (kernel, groups, threads, _, _, scratch) in enumerate(part[0]):
            cells.append(f"`{kernel}` {groups} × {threads}, {statistics.median(p[j] for p in warm):.2f} "
                         f"({statistics.median(p[j] for p in cold):.2f})" + (f", {scratch} bytes a lane" if scratch else ""))
        us, w = statistics.median(sum(p) for p in cold), more_operators.work(case)
        lines.append(f"| {case['name']} | {'; '.join(cells)} | {statistics.median(sum(p) for p in warm):.2f} | {us:.2f} | "
                     f"{w['bytes'] / us / 1e3:.0f} | {w['flops'] / us / 1e6:.1f} |")
    if counter_csvs:
        lines += ["", "Counters per launch (inputs not in a cache; FETCH_SIZE and WRITE_SIZE are in KiB as counted; the copy moves 256 MiB):", "",
                  "| case | launch | counter | value |", "|---|---|---|---|"]
    for path in counter_csvs:
        for name, per in counted(path).items():
            if name in ("FETCH_SIZE", "WRITE_SIZE"):
                lines.append(f"| | the copy | {name} | {max(profsum.dispatch_values(path, name, profsum.CALIB)):.0f} |")
            if len(per) != len(COUNTED):
                raise ValueError(f"{path}: {len(per)} passes of {len(COUNTED)} cases")
            for case, runs in zip((c["name"] for c in every if c["name"] in COUNTED), per):
                lines += [f"| {case} | `{kernel}` | {name} | {value:.0f} |" for kernel, value in runs]
    lines += ["", f"Sources SHA-256 ({', '.join(SOURCES)}): `{source_digest()}`", ""]
    with open(os.path.join(profsum.PROFILES, "kernels_window.md"), "w") as f:
        f.write("\n".join(lines))


def main():
    ap = argparse.ArgumentParser()
    sub = ap.add_subparsers(dest="what", required=True)
    r = sub.add_parser("run")
    r.add_argument("--counters", action="store_true")
    t = sub.add_parser("table")
    t.add_argument("--trace", required=True)
    t.add_argument("--counters", nargs="*", default=[])
    t.add_argument("--command", required=True)
    a = ap.parse_args()
    if a.what == "run":
        run(a.counters)
    else:
        table(a.trace, a.counters, a.command)


if __name__ == "__main__":
    main()
