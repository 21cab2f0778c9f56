"""The splits of a context: the planner's page arithmetic, compiled as plain C++, against whole
numbers of any size, up to the longest contexts that 32 bits hold (no GPU)."""
import os
import random
import shutil
import subprocess

import pytest

from paged_kv_attention_18_gb300 import build as B

MAX_PAGES = (2 ** 31 - 1024 - 1 + 15) // 16  # of the longest context that is served
MAX_SPLITS = 32
PROGRAM = """
#include <cstdio>
#include "ps_split.h"
int main() {
  int first, end, ns;
  while (std::scanf("%d %d %d", &first, &end, &ns) == 3) {
    for (int k = 0; k <= ns; ++k) std::printf("%d ", ps::split_start(first, end, ns, k));
    std::printf("\\n");
  }
}
"""


def stepped(first, end, ns):
    """The starts as the planner's count of partial results steps them, by a running remainder."""
    q, r = divmod(end - first, ns)
    at, rem, starts = first, 0, []
    for _ in range(ns + 1):
        starts.append(at)
        at, rem = at + q, rem + r
        if rem >= ns:
            at, rem = at + 1, rem - ns
    return starts


def cases():
    spans = [1, 2, 31, 32, 33, 1000, 2 ** 20 + 7]
    for near in (2 ** 26 // MAX_SPLITS * 32, 2 ** 26, 2 ** 27 // 3, MAX_PAGES):
        spans += [near + d for d in range(-40, 41) if 0 < near + d <= MAX_PAGES]
    r = random.Random(1)
    spans += [r.randint(1, MAX_PAGES) for _ in range(200)]
    for span in spans:
        for ns in {1, 2, 3, 7, 31, MAX_SPLITS, r.randint(1, MAX_SPLITS)}:
            if ns <= span:
                yield r.choice([0, MAX_PAGES - span, r.randint(0, MAX_PAGES - span)]), span, ns
        # a stream's pages, the sinks' counted ahead of the window's first
        yield -min(5, span), span, min(MAX_SPLITS, span)


def test_starts_of_splits(tmp_path):
    cxx = shutil.which(os.environ.get("CXX", "g++"))
    if cxx is None:
        pytest.skip("no host compiler")
    (tmp_path / "starts.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "starts")
    subprocess.run([cxx, "-std=c++17", "-O2", f"-I{B.CSRC}", str(tmp_path / "starts.cpp"), "-o",
                    exe], check=True)
    todo = [(first, first + span, ns) for first, span, ns in cases()]
    got = subprocess.run([exe], input="".join("%d %d %d\n" % t for t in todo), text=True,
                         capture_output=True)
    assert got.returncode == 0, got.stderr
    lines = got.stdout.splitlines()
    assert len(lines) == len(todo)
    for (first, end, ns), line in zip(todo, lines):
        want = [first + k * (end - first) // ns for k in range(ns + 1)]
        assert stepped(first, end, ns) == want
        assert [int(x) for x in line.split()] == want, (first, end, ns)
