"""The waits with a limit (csrc/dyt_cluster.cuh, csrc/dyt_steal.cuh) in a small kernel of their own, where they run out:
what they wait for is sent late, or never. Nothing faults or hangs: every wait ends by its limit, and the
cluster's own barrier is reached by all threads whatever the waits found."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cuda_runtime.h>

#include "dyt_cluster.cuh"
#include "dyt_steal.cuh"

constexpr int kShort = 64;  // polls of a wait that is to run out

// One warp in each of two CTAs. of: out[cta * 8 + k].
__global__ void __cluster_dims__(2) meet(float *out) {
  __shared__ dyt::Meet m;
  const int lane = threadIdx.x;
  const int cta = (int)dyt::cluster_rank();
  float *o = out + cta * 8;
  m.init(lane, 32);
  dyt::cluster_sync();
  if (cta == 0) {  // the other CTA sends nothing yet
    m.put(0, 1.0f, lane, 32);
    bool any = false;
    for (int i = 0; i < 3; ++i) any |= m.wait<kShort>(0, lane, 32);
    if (lane == 0) o[0] = any;
  }
  dyt::cluster_sync();
  if (cta == 1) m.put(0, 2.0f, lane, 32);
  // now all comes, within the ordinary limit: the barrier is as it was before the waits that ran out
  const bool first = m.wait(0, lane, 32);
  if (lane == 0) o[1] = first, o[2] = m.of[0][0], o[3] = m.of[0][1];
  for (int it = 1; it < 5; ++it) {  // and so for the steps behind it, the same places again
    m.put(it, it * 10.0f + cta, lane, 32);
    const bool more = m.wait(it, lane, 32);
    if (lane == 0 && it == 4) o[4] = more, o[5] = m.of[0][0], o[6] = m.of[0][1];
    if (lane == 0 && it == 3) o[7] = more && m.of[1][0] == 30.0f && m.of[1][1] == 31.0f;
  }
  dyt::cluster_sync();
}

// An answer that was not asked for does not come.
__global__ void steal(float *out) {
  __shared__ dyt::Steal queue;
  if (threadIdx.x == 0) queue.init();
  __syncthreads();
  const int64_t got = queue.take<kShort>(0);
  if (threadIdx.x == 0) out[16] = got == dyt::Steal::kLost;
}

extern "C" int run(float *out, void *stream) {
  meet<<<2, 32, 0, (cudaStream_t)stream>>>(out);
  steal<<<1, 64, 0, (cudaStream_t)stream>>>(out);
  return (int)cudaGetLastError();
}
"""


def test_waits_that_run_out_leave_their_barrier_whole(tmp_path):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from elementwise_reduction_b200 import build
    src, lib = tmp_path / "waits.cu", tmp_path / "waits.so"
    src.write_text(PROGRAM)
    subprocess.run([build.nvcc(), *build.NVCC_FLAGS, "-shared", "-o", str(lib), str(src)], check=True)
    call = ctypes.CDLL(str(lib)).run
    call.argtypes, call.restype = [ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int
    out = torch.full((17,), -1.0, device="cuda")
    assert call(out.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    got = out.tolist()
    assert got[0] == 0, "a wait for what was not sent found it"
    for cta in (0, 1):
        o = got[8 * cta:8 * cta + 8]
        assert o[1:4] == [1, 1, 2] and o[4:7] == [1, 40, 41] and o[7] == 1, o
    assert got[16] == 1
