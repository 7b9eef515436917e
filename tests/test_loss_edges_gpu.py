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


@pytest.mark.parametrize("M,N,dtype,pitch,offset", [(3, 151936, "bf16", None, 0), (300, 151936, "bf16", None, 0),
                                                    (5, 256000, "f16", None, 0), (40, 256000, "bf16", 256003, 1),
                                                    (2, 500001, "f32", None, 3), (1, 2000003, "bf16", None, 1)])
def test_large_vocabularies(M, N, dtype, pitch, offset):
    c = Case(M, N, dtype, pitch=pitch, offset=offset, T=0.9, masked=0.3 if M > 3 else 0.0)
    got, _ = c.check_forward()
    c.check_backward(got, grad=1000.0)
    c.check_backward(got, grad=1000.0, out_pitch=N + 5, out_offset=2)  # the output at other offsets


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,pitch,offset", [(9, 5003, 5003, 3), (2000, 77, 77, 1), (1300, 1001, 1008, 0),
                                              (5, 70001, 70003, 5), (700, 9, 9, 2)])
def test_gradients_in_place_on_ragged_rows(M, N, pitch, offset, dtype):
    c = Case(M, N, dtype, pitch=pitch, offset=offset, masked=0.2)
    got, _ = c.check_forward()
    dz = dyt().policy_loss_backward(c.z.t, c.tokens, got[2], got[3])
    assert dyt().policy_loss_backward(c.z.t, c.tokens, got[2], got[3], dlogits=c.z.t) is c.z.t
    want = R.Guarded(M, N, c.z.t.dtype, pitch, offset)
    dyt().policy_loss_backward(Case(M, N, dtype, pitch=pitch, offset=offset, masked=0.2).z.t, c.tokens, got[2], got[3],
                               dlogits=want.t)
    assert torch.equal(c.z.t, dz) and torch.equal(c.z.t, want.t)
    c.z.assert_surroundings_untouched("dlogits")


def test_a_batch_cut_by_one_position():
    # a causal model's logits predict the next token: logits[:, :-1] has no single pitch, is refused by the
    # function and copied by the module; with weight 0 at the last position the whole logits are taken as they
    # lie, those rows unread, for the same loss and gradient
    B, S, N = 4, 30, 1003
    g = torch.Generator("cuda").manual_seed(5)
    z = torch.randn(B, S, N, device="cuda", generator=g).to(torch.bfloat16)
    ids = torch.randint(0, N, (B, S), device="cuda", generator=g)
    adv = torch.randn(B, 1, device="cuda", generator=g).expand(B, S - 1)
    old = torch.full((B, S - 1), -7.0, device="cuda")
    weight = torch.full((B, S - 1), 1.0 / (B * (S - 1)), device="cuda")
    with pytest.raises(ValueError):
        dyt().policy_loss_forward(z[:, :-1], ids[:, 1:].contiguous(), old, adv.contiguous())
    loss = dyt().PolicyLoss()
    a = z.clone().requires_grad_()
    cut = loss(a[:, :-1], ids[:, 1:], old, adv, weight=weight)
    cut.backward()
    b = z.clone()
    b[:, -1] = float("nan")
    b.requires_grad_()
    last = lambda t, v: torch.cat([t, torch.full_like(t[:, :1], v)], 1)  # noqa: E731
    whole = loss(b, ids.roll(-1, 1), last(old, 0.0), last(adv, 0.0), weight=last(weight, 0.0))
    whole.backward()
    # the row sums are those of other parts and lanes: each loss is within its own bound of the formula
    flat = z[:, :-1].reshape(-1, N)
    want, tol = R.loss_forward(flat, ids[:, 1:].reshape(-1), old.reshape(-1), adv.reshape(-1),
                               weight=weight.reshape(-1))
    for v in (cut, whole):
        R.assert_close(v.detach(), want[0], tol[0], "loss")
    wdz, tdz = R.loss_backward(flat, ids[:, 1:].reshape(-1), want[2], want[3])
    # (the rows' own statistics and coefficients are rounded: their bounds, by the gradient's derivatives)
    extra = wdz.abs() * (tol[2][:, 1:] + 2 * R.U) + tol[3][:, None]
    for v in (a, b):
        got = v.grad[:, :-1].reshape(-1, N)
        R.assert_close(got, wdz, tdz + extra + R.half_step(got.dtype, wdz), "dlogits")
        assert torch.equal(v.grad[:, -1], torch.zeros_like(v.grad[:, -1]))


@pytest.mark.parametrize("M,N,masked", [(4736, 33000, 0.6), (4737, 33000, 0.6), (6000, 32768, 0.3), (8192, 20000, 0.9),
                                        (8192, 17000, 0.9)])
def test_rows_listed_or_looked_up_one_by_one(M, N, masked):
    # both sides of what a warp can look up in the list: 32 items, rows times the room for parts
    c = Case(M, N, "bf16", masked=masked)
    got, _ = c.check_forward()
    c.check_backward(got, grad=1000.0)
    M1 = M // 8
    c.weight = torch.zeros_like(c.weight)
    c.weight[:M1] = 1.0 / M1  # all of them side by side
    c.tokens = torch.randint(0, N, (M,), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    c.check_forward()
