"""The count of blocks ahead of the list of attention over packed prompts, run on the host: whatever the offsets are, what is
listed fits the list, no sum passes 31 bits, and offsets that ascend are listed whole."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "online_kv_cache_02_gb300", "csrc")

MODEL = r"""
#include "tq_prompt_list.h"

#include <algorithm>
#include <climits>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

using namespace tq;

struct Count {
  bool lists;                        // by the sizes alone, as the host decides
  int taken, blocks;                 // sequences and blocks that the device lists
  long long all;                     // blocks of all pairs that are sequences
};

#define NEED(x)                                                                            \
  if (!(x)) {                                                                              \
    std::printf("line %d: %s (S %d, total %d, G %d, rows %d)\n", __LINE__, #x, S, total, G, rows); \
    std::exit(1);                                                                          \
  }

// As the host and then each block of the kernels count.
Count count(const std::vector<int>& cu, int total, int max_q, int G, int rows, long long units = 100) {
  const int S = static_cast<int>(cu.size()) - 1;
  Count c{};
  max_q = std::min(max_q, total);
  const long long bound = prompt_most_blocks(S, max_q, total, G, rows);
  const int most = prompt_list_room(units);
  c.lists = S <= kPromptList && bound <= most;
  if (!c.lists) return c;
  std::vector<int> firsts(S), exact(S);
  long long sum = 0;
  bool ascends = true;
  for (int s = 0; s < S; ++s) {
    const bool ok = prompt_pair(cu[s], cu[s + 1], total, max_q);
    ascends = ascends && ok;
    exact[s] = ok ? prompt_blocks(cu[s + 1] - cu[s], G, rows) : 0;
    c.all += exact[s];
    NEED(sum <= INT_MAX);
    firsts[s] = static_cast<int>(sum);
    sum += prompt_counted(exact[s], most);
  }
  NEED(sum <= INT_MAX);
  c.taken = prompt_taken(firsts.data(), S, static_cast<int>(sum), most);
  NEED(c.taken >= 0 && c.taken <= S);
  c.blocks = c.taken < S ? firsts[c.taken] : static_cast<int>(sum);
  NEED(c.blocks <= kPromptList && c.blocks * units <= INT_MAX);         // places in the list, and their units
  long long listed = 0;
  for (int s = 0; s < c.taken; ++s) {
    NEED(firsts[s] == listed);                                          // as they are without the limit
    listed += exact[s];
  }
  NEED(listed == c.blocks);
  if (c.taken < S) NEED(c.blocks + exact[c.taken] > most || exact[c.taken] == 0);
  if (ascends) NEED(c.taken == S && c.blocks == c.all);
  return c;
}

int main() {
  // the same rows again and again
  for (int pairs : {1, 2, 3, 60, 1000}) {
    std::vector<int> cu;
    const int n = 100000;
    for (int i = 0; i <= pairs; ++i) cu.push_back(0), cu.push_back(n);
    const Count c = count(cu, n, n, 4, 256);
    if (!c.lists && pairs < 400) return std::printf("not listed: %d pairs\n", pairs), 1;
    if (c.lists && c.all <= (pairs >= 1 ? kPromptList : 0)) return std::printf("the model's offsets do not pass the list\n"), 1;
  }
  {
    std::vector<int> cu;             // more than 31 bits of blocks
    const int n = 1 << 15;
    for (int i = 0; i < 1000; ++i) cu.push_back(0), cu.push_back(n);
    (void)count(cu, n, n, 1, 32);
    (void)count(cu, n, n, 1, 16);
  }
  std::mt19937 rng(1);
  int listed = 0, cut = 0;
  for (int i = 0; i < 20000; ++i) {
    const int S = 1 + static_cast<int>(rng() % (i % 10 ? 30 : 2048)), G = 1 + rng() % 9, rows_of[] = {16, 64, 128, 256, 2 * (128 / G) * G};
    const int rows = rows_of[rng() % 5], total = 1 + static_cast<int>(rng() % (rng() % 2 ? 300000 : 3000));
    const int max_q = rng() % 3 ? total : 1 + static_cast<int>(rng() % total);
    std::vector<int> cu(S + 1);
    for (int& x : cu) x = static_cast<int>(rng() % (total + 1));
    const int kind = rng() % 4;
    if (kind == 0) std::sort(cu.begin(), cu.end());
    if (kind == 1)                   // ascending, a few out of place
      std::sort(cu.begin(), cu.end()), cu[rng() % (S + 1)] = static_cast<int>(rng()), cu[rng() % (S + 1)] = 0;
    if (kind == 2)
      for (int& x : cu)
        if (rng() % 8 == 0) x = static_cast<int>(rng());
    const Count c = count(cu, total, max_q, G, rows, 5 + rng() % (1 << rng() % 24));
    listed += c.lists;
    cut += c.lists && c.taken < S;
  }
  if (listed < 2000 || cut < 200) return std::printf("too few cases: %d listed, %d cut\n", listed, cut), 1;
  return 0;
}
"""


def test_offsets_of_any_kind_fit_the_list(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "list.cpp", tmp_path / "list"
    src.write_text(MODEL)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout + run.stderr
