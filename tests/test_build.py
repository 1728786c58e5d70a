"""The build step, with a stand-in for the compiler: builds side by side and builds that fail."""
import os
import threading

import pytest

from moe_routed_expert_route_amd import build

# Joins its inputs into -o's file; refuses a source that says so; the second to link waits for `first_done`.
COMPILER = """#!/bin/sh
inputs=
link=yes
while [ $# -gt 0 ]; do
  case "$1" in
    -o) out=$2; shift;;
    -c) link=;;
    *.hip|*.o) inputs="$inputs $1";;
  esac
  shift
done
grep -q refuse $inputs && { sleep 0.2; exit 1; }
if [ -n "$link" ] && ! mkdir "$STUB/linked" 2>/dev/null; then
  i=0
  while [ ! -e "$STUB/first_done" ] && [ $i -lt 100 ]; do sleep 0.05; i=$((i + 1)); done
fi
cat $inputs > "$out"
"""


@pytest.fixture
def stub(tmp_path, monkeypatch):
    src = tmp_path / "src"
    src.mkdir()
    (tmp_path / "hipcc").write_text(COMPILER)
    (tmp_path / "hipcc").chmod(0o755)
    for name in "ab":
        (src / f"{name}.hip").write_text(name)
    monkeypatch.setenv("HIPCC", str(tmp_path / "hipcc"))
    monkeypatch.setenv("STUB", str(tmp_path))
    monkeypatch.setattr(build, "SRCS", [str(src / "a.hip"), str(src / "b.hip")])
    monkeypatch.setattr(build, "LIB", str(src / "lib.so"))
    return tmp_path


def test_two_builds_at_once(stub):
    failed = []

    def one():
        try:
            build.build()
        except Exception as e:
            failed.append(e)
        (stub / "first_done").touch()

    threads = [threading.Thread(target=one) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    assert (stub / "src" / "lib.so").read_text() == "ab"
    assert sorted(os.listdir(stub / "src")) == ["a.hip", "b.hip", "lib.so"]


def test_a_failed_build_leaves_nothing_and_keeps_the_library(stub):
    (stub / "src" / "lib.so").write_text("before")
    (stub / "src" / "b.hip").write_text("refuse")
    with pytest.raises(RuntimeError, match="hipcc failed"):
        build.build()
    assert sorted(os.listdir(stub / "src")) == ["a.hip", "b.hip", "lib.so"]
    assert (stub / "src" / "lib.so").read_text() == "before"
