"""The record of an item that the join of shared prefixes follows, run on the host: whatever an unwritten one holds, nothing
outside the pass' parts is named."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "online_kv_cache_02_gb300", "csrc")

MODEL = r"""
#include "tq_kv8_parts.h"

#include <climits>
#include <cstdio>
#include <random>

int main() {
  std::mt19937 rng(2);
  const int edges[] = {INT_MIN, INT_MIN + 1, -2, -1, 0, 1, 2, 150, 151, 152, 153, 455, 456, INT_MAX - 1, INT_MAX};
  long long records = 0;
  for (int i = 0; i < 2000000; ++i) {
    const int ctas = 1 + rng() % 608;
    const int a = i % 3 ? edges[rng() % 15] : static_cast<int>(rng()), b = i % 2 ? edges[rng() % 15] : static_cast<int>(rng() % 700);
    if (a < 0) continue;             // a whole item
    const int n = tq::kv8_item_parts(a, b, ctas);
    const bool record = a <= b && b < ctas;
    if (record ? n != b - a + 1 : n != 0) return std::printf("%d %d of %d: %d\n", a, b, ctas, n), 1;
    records += record;
  }
  return records < 10000;
}
"""


def test_no_record_names_parts_that_are_not_there(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "parts.cpp", tmp_path / "parts"
    src.write_text(MODEL)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stdout
