"""The ring of pages of the 8-bit decode kernel, run on the host against a model of its copies and barriers.

The model keeps each stage's barrier (one arrival and one copy a phase) and says what the hardware would not: a second
arrival while a phase's copy is under way, a copy into a stage that another copy still fills, and copies under way when
the run has ended.  Copies are late and waits give up at chosen places."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "online_kv_cache_02_gb300", "csrc")

MODEL = r"""
#include "tq_kv8_ring.h"

#include <cstdio>
#include <cstdlib>
#include <vector>

struct Model {                       // stages' barriers and copies
  int st;
  std::vector<int> phase, page;      // phases ended; the page on its way or in place
  std::vector<bool> flying;
  int faults = 0, waits = 0, give_up_at = -1;
  explicit Model(int n) : st(n), phase(n, 0), page(n, -1), flying(n, false) {}
  void send(int p, unsigned s) {
    if (flying[s]) ++faults;         // an arrival and a copy on top of the one before
    flying[s] = true;
    page[s] = p;
  }
  bool wait(unsigned s, unsigned parity) {
    if (waits++ == give_up_at) return false;
    if (flying[s]) {                 // the copy comes: its phase ends
      flying[s] = false;
      ++phase[s];
    }
    return ((phase[s] - 1) & 1) == static_cast<int>(parity) && phase[s] > 0;
  }
  bool any_flying() const {
    for (bool f : flying)
      if (f) return true;
    return false;
  }
};

// What the kernel does with the ring: runs of `n` pages; returns the faults, or -1 for a wrong page.
template <int ST>
int through_ring(const std::vector<int>& runs, int give_up_at) {
  tq::PageRing<ST> ring;
  Model m(ST);
  m.give_up_at = give_up_at;
  bool gave_up = false;
  for (int n : runs) {
    auto send = [&](int ahead, unsigned s) { m.send(ring.k + ahead, s); };
    auto wait = [&](unsigned s, unsigned p) { return m.wait(s, p); };
    ring.start(n, send);
    while (ring.k < ring.n) {
      const int k = ring.k;
      const unsigned s = ring.stage();
      if (!ring.land(wait)) {
        gave_up = true;
        break;
      }
      if (m.page[s] != k) return -1;
      ring.pass(send);
    }
    if (!gave_up && ring.k != n) return -1;
    if (m.any_flying()) ++m.faults;  // lands in memory that has another use
  }
  if (gave_up != ring.failed || (give_up_at < 0 && gave_up)) return -1;
  return m.faults;
}

// The order that goes wrong: after a wait that gave up every further page is still asked for, and what is waited for
// at the end are the stages by a count that no longer matches their phases.
template <int ST>
int asking_on(int n, int give_up_at) {
  Model m(ST);
  m.give_up_at = give_up_at;
  bool failed = false;
  unsigned used = 0;
  auto issue = [&](int k) {
    if (k < n) m.send(k, k % ST);
  };
  for (int i = 0; i < ST; ++i) issue(i);
  for (int k = 0; k < n; ++k, ++used) {
    if (!failed && !m.wait(used % ST, (used / ST) & 1)) failed = true;
    issue(k + ST);
  }
  for (int i = 0; i < ST && failed; ++i) (void)m.wait((used + i) % ST, ((used + i) / ST) & 1);
  return m.faults + (m.any_flying() ? 1 : 0);
}

template <int ST>
void all() {
  for (int n = 0; n < 40; ++n)
    for (int at = -1; at < n; ++at) {
      const int a = through_ring<ST>({n}, at), b = through_ring<ST>({n, 7, 0, 33}, at);
      if (a || b) {
        std::printf("stages %d pages %d wait %d: %d %d\n", ST, n, at, a, b);
        std::exit(1);
      }
    }
  if (asking_on<ST>(30, -1) != 0 || asking_on<ST>(30, 9) == 0) {
    std::printf("stages %d: the model does not tell the wrong order\n", ST);
    std::exit(1);
  }
}

int main() {
  all<2>();
  all<3>();
  all<4>();
  return 0;
}
"""


def test_ring_asks_for_nothing_after_a_wait_that_gave_up(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(MODEL)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stdout
