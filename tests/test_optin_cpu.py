"""The record of shared-memory opt-ins (csrc/dyt_optin.h), compiled with the host
compiler and called from two threads with a stand-in for the CUDA call: a smaller
request that is under way when a larger one arrives never lowers the limit, and
what the record calls ready is in force."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "elementwise_reduction_b200", "csrc")

PROGRAM = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>

#include "dyt_optin.h"

using Clock = std::chrono::steady_clock;

// Waits until c holds, half a second at most: the threads below meet in the order given if nothing keeps
// them apart, and go on by themselves if a lock does.
template <typename C>
static void until(C c) {
  const auto end = Clock::now() + std::chrono::milliseconds(500);
  while (!c() && Clock::now() < end) std::this_thread::yield();
}

int main() {
  const int small = 12288, large = 98304;
  for (int order = 0; order < 2; ++order) {
    dyt::host::SmemOptIn opt;
    std::atomic<int> limit{0}, calls{0};
    std::atomic<bool> small_in{false}, large_set{false}, large_done{false};
    std::thread a([&] {
      opt.raise(7, small, [&](int b) {
        small_in = true;
        until([&] { return order ? large_set.load() : large_done.load(); });  // the larger request overtakes
        limit = b;
        ++calls;
        return 0;
      });
    });
    until([&] { return small_in.load(); });
    opt.raise(7, large, [&](int b) {
      limit = b;
      ++calls;
      large_set = true;
      if (order) std::this_thread::sleep_for(std::chrono::milliseconds(200));  // recorded after the smaller one
      return 0;
    });
    large_done = true;
    a.join();
    // a later call for the large size: either the limit holds already, or the record knows that it does not
    opt.raise(7, large, [&](int b) {
      limit = b;
      ++calls;
      return 0;
    });
    std::printf("order %d limit %d calls %d\n", order, limit.load(), calls.load());
    if (limit != large || calls != 2) return 1;
  }
  dyt::host::SmemOptIn opt;
  int n = 0;
  if (opt.raise(1, 100, [&](int) { return ++n, 5; }) != 5) return 2;     // a failure is returned and not recorded
  if (opt.raise(1, 100, [&](int) { return ++n, 0; }) != 0 || n != 2) return 3;
  if (opt.raise(1, 40, [&](int) { return ++n, 0; }) != 0 || n != 2) return 4;   // covered
  if (opt.raise(2, 40, [&](int) { return ++n, 0; }) != 0 || n != 3) return 5;   // another key
  return 0;
}
"""


def test_opt_ins_from_two_threads_only_raise_the_limit(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "optin.cpp", tmp_path / "optin"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stdout)
