"""The table of a trace of the calls on windows, from a made-up trace."""
import csv

import pytest

from moe_routed_expert_route_amd import profsum, windowprof


def _write(path, header, rows):
    with open(path, "w", newline="") as f:
        w = csv.writer(f)
        w.writerow(header)
        w.writerows(rows)


def test_table(tmp_path, monkeypatch):
    cases, rows, at = windowprof.cases(), [], 1000
    assert len({c["name"] for c in cases}) == len(cases) and {c["name"] for c in cases} >= set(windowprof.COUNTED)
    for i in range(len(cases)):
        for p in range(2 * windowprof.PASSES):
            dur = 4000 + 100 * i if p < windowprof.PASSES else 8000 + 100 * i
            if p in (0, 1, windowprof.PASSES):          # the first two of each kind do not count
                dur = 90000
            rows += [["moe::k_stream_read(x)", at - 500, at - 400, 256, 1, 1, 2560, 1, 1, 0],
                     ["at::fill(x)", at - 300, at - 200, 256, 1, 1, 256, 1, 1, 0],
                     [f"void moe::k_case{i}<moe::bf16_t, 4>(moe::Args)", at, at + dur, 128, 1, 1, 128 * (i + 1), 3, 1, 16 if i == 2 else 0],
                     ["moe::k_join(moe::Args)", at + dur + 1000, at + dur + 3000, 64, 1, 1, 640, 1, 1, 0]]
            at += 100000
    hdr = ["Kernel_Name", "Start_Timestamp", "End_Timestamp", "Workgroup_Size_X", "Workgroup_Size_Y", "Workgroup_Size_Z", "Grid_Size_X",
           "Grid_Size_Y", "Grid_Size_Z", "Scratch_Size"]
    _write(tmp_path / "t.csv", hdr, reversed(rows))
    n = len(windowprof.COUNTED)
    _write(tmp_path / "c.csv", ["Dispatch_Id", "Kernel_Name", "Counter_Name", "Counter_Value"],
           [[1, "__amd_rocclr_copyBuffer", "FETCH_SIZE", 131072]] +
           [row for i in range(n) for row in ([10 + 3 * i, "moe::k_stream_read(x)", "FETCH_SIZE", 9],
                                              [11 + 3 * i, "void moe::k_a<4>(x)", "FETCH_SIZE", 70 + i], [11 + 3 * i, "void moe::k_a<4>(x)", "FETCH_SIZE", 1],
                                              [12 + 3 * i, "moe::k_b(x)", "FETCH_SIZE", 5])])
    monkeypatch.setattr(profsum, "PROFILES", str(tmp_path))
    windowprof.table(str(tmp_path / "t.csv"), [str(tmp_path / "c.csv")], "cmd")
    text = open(tmp_path / "kernels_window.md").read()
    from perf import more_operators
    w = more_operators.work(cases[2])
    assert (f"| {cases[2]['name']} | `k_case2<bf16_t, 4>` 9 × 128, 4.20 (8.20), 16 bytes a lane; `k_join` 10 × 64, 2.00 (2.00) | 6.20 | 10.20 | "
            f"{w['bytes'] / 10.2 / 1e3:.0f} |") in text
    assert "| | the copy | FETCH_SIZE | 131072 |" in text
    names = [c["name"] for c in cases if c["name"] in windowprof.COUNTED]
    assert f"| {names[1]} | `k_a<4>` | FETCH_SIZE | 72 |" in text and f"| {names[n - 1]} | `k_b` | FETCH_SIZE | 5 |" in text
    assert windowprof.source_digest() in text
    _write(tmp_path / "t.csv", hdr, rows[:-4])
    with pytest.raises(ValueError, match="passes"):
        windowprof.table(str(tmp_path / "t.csv"), [], "cmd")
    rows[1 + 2][0] = "moe::k_other(x)"
    _write(tmp_path / "t.csv", hdr, rows)
    with pytest.raises(ValueError, match="different launches"):
        windowprof.table(str(tmp_path / "t.csv"), [], "cmd")
