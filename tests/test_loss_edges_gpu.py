"""The policy loss's kernels where its other tests do not reach: parts of few weighted
rows, vocabularies beyond 70000, in place on ragged rows, sliced batches."""
from __future__ import annotations

import pytest
import torch

from tests import row_helpers as R
from tests.test_loss_gpu import Case, dyt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")


def parts_written(c, parts):
    """How many partial sums a call writes. They lie at the workspace's start, with room for at least 16
    a row (of rows of 16 batches or more)."""
    ws = dyt().policy_loss_workspace(c.z.t)
    ws.fill_(255)
    c.forward(ws=ws)
    M = c.z.t.shape[0]
    return int((ws[:M * max(parts, 16) * 8].view(torch.int32).view(-1, 2) != -1).any(-1).sum())


@pytest.mark.parametrize("M,N,dtype", [(64, 131072, "bf16"), (32, 152064, "bf16"), (37, 131072, "f16"),
                                       (40, 100000, "f32"), (300, 40000, "bf16")])
def test_weights_leave_few_long_rows_their_parts(M, N, dtype):
    # the same rows with and without weights: as many parts, whichever way the kernel finds the rows
    c = Case(M, N, dtype)
    c.forward()
    parts = dyt().dyt_last_launch_info()["col_chunks"]
    assert parts > 4
    assert parts_written(c, parts) == M * parts
    c.weight = torch.full((M,), 1.0 / M, device="cuda")
    got, info = c.check_forward()
    assert info["col_chunks"] == parts and parts_written(c, parts) == M * parts
    c.check_backward(got, grad=100.0)
    c.weight[1::2] = 0  # half of them
    c.tokens[1::2] = -100
    got, _ = c.check_forward()
    assert parts_written(c, parts) >= M // 2 * parts // 2
    c.check_backward(got, grad=100.0)


def test_the_last_position_of_every_sequence():
    # [:, -1:] and [:, k]: rows a whole sequence apart, read where they lie
    B, S, N = 5, 7, 1003
    z = torch.randn(B, S, N, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(torch.bfloat16)
    tokens = torch.arange(B, device="cuda") * 100
    adv = torch.linspace(-1, 1, B, device="cuda")
    flat = z[:, -1].contiguous()
    old = torch.full((B,), -7.0, device="cuda")
    want = dyt().policy_loss_forward(flat, tokens, old, adv)
    dwant = dyt().policy_loss_backward(flat, tokens, want[2], want[3])
    for v, shape in ((z[:, -1:], (B, 1)), (z[:, -1], (B,))):
        t, o, a = tokens.view(shape), old.view(shape), adv.view(shape)
        got = dyt().policy_loss_forward(v, t, o, a)
        assert got[1].shape == shape and got[2].shape == (*shape, 2)
        assert all(torch.equal(p.flatten(), q.flatten()) for p, q in zip(got, want))
        d = dyt().policy_loss_backward(v, t, got[2], got[3])
        assert d.shape == v.shape and torch.equal(d.reshape(B, N), dwant)
    x = z[:, 2:3]
    assert torch.equal(dyt().layer_norm_forward(x)[0], dyt().layer_norm_forward(x.contiguous())[0])


@pytest.mark.parametrize("M,N,dtype,pad", [(1, 131072, "bf16", 0), (64, 131072, "bf16", 0), (300, 50001, "f16", 3),
                                           (148, 32000, "bf16", 0), (9, 5003, "f32", 1)])
def test_the_gradients_of_few_rows_take_no_more_parts_than_fit(M, N, dtype, pad):
    # five CTAs an SM: a part of a row for each, in one go
    c = Case(M, N, dtype, pitch=N + pad)
    got, _ = c.check_forward()
    info = c.check_backward(got, grad=100.0)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert info["path"] == 2 and info["grid"] == M * info["col_chunks"] <= 5 * sms
    assert info["col_chunks"] > 1
