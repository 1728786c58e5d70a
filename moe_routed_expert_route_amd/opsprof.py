"""Profiles of the operators around the layer: a program to run under rocprofv3, and the table of its trace.

    rocprofv3 --kernel-trace --output-format csv -d DIR -o run -- python3 -m moe_routed_expert_route_amd.opsprof run
    rocprofv3 --pmc FETCH_SIZE --kernel-trace --output-format csv -d DIR1 -o run -- \\
        python3 -m moe_routed_expert_route_amd.opsprof run --counters
    python -m moe_routed_expert_route_amd.opsprof table --trace DIR/run_kernel_trace.csv \\
        --counters DIR1/run_counter_collection.csv ... --command "..."

`run` makes PASSES passes of each case that perf/operators.py lists and of the products in MORE, on two
inputs in turn; first as they come (small inputs are in a cache then), then each after 1 GiB was read, which leaves
none of them there. `table` writes profiles/kernels_ops.md: the library's launches alone, medians, and the
counters per launch (--counters: one pass of the cases in COUNTED, after a copy of known size).
"""
from __future__ import annotations

import argparse
import csv
import hashlib
import os
import re
import statistics

from . import profsum

SOURCES = ("moe_routed_expert_route_amd/csrc/moe_ops.hip", "moe_routed_expert_route_amd/csrc/moe_device.hpp",
           "moe_routed_expert_route_amd/build.py", "perf/operators.py")
PASSES = 10
COUNTED = ("norm 8192x4096 bf16", "swiglu 4096x5461 bf16", "matmul 8192x8192x4096")
# a prompt of 512 tokens through the shared expert: gate and up stacked, and down added into the layer's Y
MORE = [dict(name="matmul 512x1536x2560", op="matmul", M=512, N=1536, K=2560, out="bf16"),
        dict(name="matmul 512x2560x768 added to f32", op="matmul", M=512, N=2560, K=768, out="f32", accumulate=True),
        dict(name="matmul 512x2560x768 added to bf16", op="matmul", M=512, N=2560, K=768, out="bf16", accumulate=True)]
CALIB_BYTES = 256 << 20


def cases():
    from perf import operators
    return operators.listed() + MORE


def work(case):
    from perf import operators
    w = operators.work(case)
    if case.get("accumulate"):   # C is read too
        w["bytes"] += case["M"] * case["N"] * operators.SIZE[case["out"]]
    return w


def source_digest() -> str:
    h = hashlib.sha256()
    for p in SOURCES:
        with open(os.path.join(profsum.ROOT, p), "rb") as f:
            h.update(f.read())
    return h.hexdigest()


def run(counters):
    import torch

    from perf import operators

    from . import binding as B
    operators.own = True

    def one(case, state):
        if not case.get("accumulate"):
            return operators.run(state)
        if "c" not in state:
            state["c"] = torch.zeros((case["M"], case["N"]), dtype=operators.DTYPES[case["out"]], device="cuda")
        return B.moe_matmul_i8(state["a"], state["sa"], state["b"], state["sb"], c=state["c"], accumulate=True)

    if counters:
        src = torch.zeros(CALIB_BYTES, dtype=torch.uint8, device="cuda")
        torch.empty_like(src).copy_(src)
    other = torch.zeros(16 if counters else 1 << 30, dtype=torch.uint8, device="cuda")
    sums = torch.empty(1024, dtype=torch.int32, device="cuda")
    for case in cases():
        if counters and case["name"] not in COUNTED:
            continue
        states = [operators.prepare(case, seed) for seed in range(2)]
        for cold in (False,) if counters else (False, True):
            for i in range(1 if counters else PASSES):
                if cold:
                    B.moe_stream_read(other, sums, 1024)   # a fill would leave lines to write back
                one(case, states[i % 2])
        torch.cuda.synchronize()
        print(case["name"], flush=True)


def launches(trace_csv):
    """The operators' launches of a kernel trace in order: (kernel, workgroups, threads, us)."""
    with open(trace_csv, newline="") as f:
        rows = [r for r in csv.DictReader(f) if "moe::k_" in r["Kernel_Name"] and "k_stream_read" not in r["Kernel_Name"]]
    rows.sort(key=lambda r: int(r["Start_Timestamp"]))
    return [(re.sub(r"moe::|^void |\(.*", "", r["Kernel_Name"]), int(r["Grid_Size_X"]) // int(r["Workgroup_Size_X"]),
             int(r["Workgroup_Size_X"]), (int(r["End_Timestamp"]) - int(r["Start_Timestamp"])) / 1e3) for r in rows]


def table(trace_csv, counter_csvs, command):
    runs = launches(trace_csv)
    if len(runs) != 2 * PASSES * len(cases()):
        raise ValueError(f"{len(runs)} launches, not {2 * PASSES} of each of {len(cases())} cases")
    lines = ["# Kernel trace of the operators around the layer", "", "Commands (repo root, one MI355X):", "", f"    {command}", "",
             f"The library's launches alone, median and least of the last {PASSES - 2} of {PASSES}: as they come (small inputs are in a "
             "cache), and cold, each after 1 GiB was read. GB/s and T(FL)OP/s go by the cold median and by the bytes and operations that the "
             "case cannot do without.", "",
             "| case | kernel | workgroups × threads | median µs | least µs | cold µs | GB/s | T(FL)OP/s |", "|---|---|---|---|---|---|---|---|"]
    for i, case in enumerate(cases()):
        mine = runs[2 * PASSES * i:2 * PASSES * (i + 1)]
        if len({m[:3] for m in mine}) != 1:
            raise ValueError(f"{case['name']}: several kernels")
        warm, cold = ([m[3] for m in part[2:]] for part in (mine[:PASSES], mine[PASSES:]))
        us, w = statistics.median(cold), work(case)
        lines.append(f"| {case['name']} | `{mine[0][0]}` | {mine[0][1]} × {mine[0][2]} | {statistics.median(warm):.2f} | {min(warm):.2f} | "
                     f"{us:.2f} | {w['bytes'] / us / 1e3:.0f} | {w['flops'] / us / 1e6:.1f} |")
    if counter_csvs:
        lines += ["", "Counters per launch (inputs not in a cache; the copy moves 256 MiB, and FETCH_SIZE and WRITE_SIZE are in KiB as counted):", "",
                  "| counter | launch | value |", "|---|---|---|"]
    for path in counter_csvs:
        with open(path, newline="") as f:
            names = sorted({r["Counter_Name"] for r in csv.DictReader(f)})
        for name in names:
            per = profsum.counter_per_dispatch(path, name)
            if name in ("FETCH_SIZE", "WRITE_SIZE"):
                lines.append(f"| {name} | the copy | {max(profsum.dispatch_values(path, name, profsum.CALIB)):.0f} |")
            for kernel, (value, _) in per.items():
                if "moe::k_" in kernel:
                    lines.append(f"| {name} | `{re.sub(r'moe::|^void |[(].*', '', kernel)}` | {value:.0f} |")
    lines += ["", f"Sources SHA-256 ({', '.join(SOURCES)}): `{source_digest()}`", ""]
    with open(os.path.join(profsum.PROFILES, "kernels_ops.md"), "w") as f:
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
