"""The record of how many clusters run at once (csrc/dyt_capacity.h), compiled with the host compiler and called with a
stand-in for the CUDA call: launches that differ in anything the answer depends on do not share one,
whichever came first."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "elementwise_reduction_b200", "csrc")

PROGRAM = r"""
#include <cstdio>

#include "dyt_capacity.h"

int main() {
  const char kernels[2] = {};
  // clusters of 4 of 480 threads, with a row of 480 lanes or three of 160 side by side
  struct Launch { int dev, kernel; unsigned threads; size_t smem; int ctas, fit; };
  const Launch all[] = {{0, 0, 480, 50000, 4, 33}, {0, 0, 480, 53760, 4, 31}, {0, 0, 480, 50000, 2, 74},
                        {0, 0, 512, 50000, 4, 30}, {0, 1, 480, 50000, 4, 29}, {1, 0, 480, 50000, 4, 28}};
  constexpr int kAll = sizeof(all) / sizeof(all[0]);
  for (int order = 0; order < 2; ++order) {
    dyt::host::Capacities c;
    int asked = 0;
    for (int round = 0; round < 2; ++round)
      for (int i = 0; i < kAll; ++i) {
        const Launch &l = all[order ? kAll - 1 - i : i];
        int n = 0;
        if (c.get(l.dev, kernels + l.kernel, l.threads, l.smem, l.ctas, &n, [&](int *out) {
              ++asked;
              *out = l.fit;
              return 0;
            }) != 0)
          return 1;
        if (n != l.fit) {
          std::printf("order %d launch %d: %d, not %d\n", order, i, n, l.fit);
          return 2;
        }
      }
    if (asked != kAll) return 3;  // each is asked for once
  }
  dyt::host::Capacities c;
  int n = 7, asked = 0;
  auto fail = [&](int *) { return ++asked, 5; };
  auto none = [&](int *out) { return ++asked, *out = 0; };
  if (c.get(0, kernels, 32, 0, 2, &n, fail) != 5 || c.get(0, kernels, 32, 0, 2, &n, fail) != 5 || asked != 2) return 4;
  if (c.get(0, kernels, 32, 0, 2, &n, none) != 0 || n != 1 || asked != 3) return 5;  // a launch of one cluster
  return 0;
}
"""


def test_an_answer_is_for_one_kind_of_launch(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "capacity.cpp", tmp_path / "capacity"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stdout)
