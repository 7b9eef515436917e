"""First calls of a process from several host threads at once: kernels that are launched
with more than one size of shared memory, layer norm's and the policy loss's."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys, threading
sys.path.insert(0, sys.argv[1])
import torch
import elementwise_reduction_b200 as dyt

g = torch.Generator("cuda").manual_seed(1)
r = lambda *s: torch.randn(*s, device="cuda", generator=g)

def norm(M, N, dtype):
    x, dy, gamma = r(M, N).to(dtype), r(M, N).to(dtype), r(N)
    def call():
        y, mean, rstd = dyt.layer_norm_forward(x, gamma, gamma)
        return (y, *dyt.layer_norm_backward(x, dy, mean, rstd, gamma, gamma))
    return call

def loss(M, N, dtype):
    z, old, adv = r(M, N).to(dtype), r(M) - 8, r(M)
    tokens = torch.randint(0, N, (M,), device="cuda", generator=g)
    return lambda: dyt.policy_loss_forward(z, tokens, old, adv)

calls = []
for t in (torch.float32, torch.bfloat16):
    # blocks of 128 and 512 threads, groups of several widths, ragged rows; parts of few and of many rows
    calls += [norm(3, 64, t), norm(4000, 64, t), norm(300, 4096, t), norm(300, 1000, t), norm(300, 1001, t),
              norm(3, 65, t), loss(1, 700, t), loss(40, 9000, t), loss(3000, 4000, t)]
torch.cuda.synchronize()
got, failed = [None] * len(calls), []
start = threading.Barrier(len(calls))

def work(i):
    stream = torch.cuda.Stream()
    start.wait()
    try:
        with torch.cuda.stream(stream):
            got[i] = calls[i]()
    except Exception as e:
        failed.append((i, repr(e)))

threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
for t in threads: t.start()
for t in threads: t.join()
torch.cuda.synchronize()
assert not failed, failed
for i, call in enumerate(calls):  # every size, again, after all of the first calls
    for a, b in zip(got[i], call()):
        assert torch.equal(a, b), i
torch.cuda.synchronize()
print("ok")
"""


@pytest.mark.parametrize("attempt", range(3))
def test_first_calls_from_many_threads(attempt):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout[-2000:] + r.stderr[-2000:]
