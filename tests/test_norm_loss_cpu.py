"""Layer norm and the policy loss without a GPU: the plain formulas the GPU tests
compare with against autograd and differences, and the entry points' refusals,
which come before any CUDA call."""
from __future__ import annotations

import pytest
import torch

import elementwise_reduction_b200 as dyt
from tests import row_helpers as R

A = 1 << 20  # a 16-byte aligned stand-in for a device address


def test_norm_formulas_agree_with_autograd():
    torch.manual_seed(0)
    x = torch.randn(5, 11, dtype=torch.float64, requires_grad=True)
    g = torch.rand(11, dtype=torch.float64, requires_grad=True)
    b = torch.randn(11, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(5, 11, dtype=torch.float64)
    y = torch.nn.functional.layer_norm(x, (11,), g, b, 1e-3)
    (y * dy).sum().backward()
    (mine, mean, rstd), _ = R.norm_forward(x.detach(), g.detach(), b.detach(), 1e-3)
    assert torch.allclose(mine, y, rtol=1e-12, atol=1e-12)
    (dx, dgamma, dbeta), _ = R.norm_backward(x.detach(), dy, mean, rstd, g.detach())
    for got, want in ((dx, x.grad), (dgamma, g.grad), (dbeta, b.grad)):
        assert torch.allclose(got, want, rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("T", [1.0, 0.7])
def test_loss_formulas_agree_with_autograd(T):
    torch.manual_seed(1)
    M, N = 40, 13
    z = torch.randn(M, N, dtype=torch.float64, requires_grad=True)
    tokens = torch.randint(0, N, (M,))
    adv, weight = torch.randn(M, dtype=torch.float64), torch.rand(M, dtype=torch.float64)
    weight[::5] = 0
    lp = (z / T).log_softmax(-1).gather(1, tokens[:, None])[:, 0]
    old = lp.detach() + 0.3 * torch.randn(M, dtype=torch.float64)
    ref = lp.detach() + 0.3 * torch.randn(M, dtype=torch.float64)
    r, q = (lp - old).exp(), ref - lp
    each = -torch.minimum(r * adv, r.clamp(0.8, 1.3) * adv) + 0.1 * (q.exp() - q - 1)
    loss = (each * weight).sum()
    loss.backward()
    (mine, logp, stats, coef), _ = R.loss_forward(z.detach(), tokens, old, adv, ref, weight, 0.2, 0.3, 0.1, T)
    assert torch.allclose(mine, loss, rtol=1e-12)
    assert torch.allclose(logp, torch.where(weight != 0, lp, torch.zeros_like(lp)), rtol=1e-12)
    dz, _ = R.loss_backward(z.detach(), tokens, stats, coef, 1.0, T)
    assert torch.allclose(dz, z.grad, rtol=1e-10, atol=1e-13)
    v, t = torch.randn(M, N, dtype=torch.float64), 1e-6
    f = lambda a: float(R.loss_forward(a, tokens, old, adv, ref, weight, 0.2, 0.3, 0.1, T)[0][0])  # noqa: E731
    slope = (f(z.detach() + t * v) - f(z.detach() - t * v)) / (2 * t)
    assert abs(slope - float((dz * v).sum())) < 1e-6


def norm_fwd(x=A, ldx=8, g=A, b=A, eps=1e-5, y=A, ldy=8, mean=A, rstd=A, M=4, N=8, xd=0, gd=0, bd=0):
    return dyt.dyt_layer_norm_forward(x, ldx, g, b, eps, y, ldy, mean, rstd, M, N, xd, gd, bd, None)


def norm_bwd(x=A, ldx=8, dy=A, lddy=8, g=A, mean=A, rstd=A, dx=A, lddx=8, dg=A, db=A, M=4, N=8, xd=0, gd=0, bd=0,
             ws=A, n=1 << 20):
    return dyt.dyt_layer_norm_backward(x, ldx, dy, lddy, g, mean, rstd, dx, lddx, dg, db, M, N, xd, gd, bd, ws, n,
                                       None)


def test_norm_refusals():
    for kw in ({"M": -1}, {"N": -1}, {"N": 2**31, "ldx": 2**31, "ldy": 2**31}, {"M": 2**62}, {"ldx": 7}, {"ldy": 7},
               {"ldx": 2**61}, {"x": 0}, {"y": 0}, {"x": A + 2}, {"y": A + 1}, {"g": A + 2}, {"b": A + 1},
               {"mean": A + 2}, {"rstd": A + 3}, {"eps": -1e-5}, {"eps": float("nan")}, {"eps": float("inf")}):
        assert norm_fwd(**kw) == 1, kw
    for kw in ({"xd": 3}, {"xd": -1}, {"gd": 5}, {"bd": 9}):
        assert norm_fwd(**kw) == 2 and norm_bwd(**kw) == 2, kw
    for kw in ({"M": -1}, {"N": -1}, {"ldx": 7}, {"lddy": 7}, {"lddx": 7}, {"x": 0}, {"dy": 0}, {"dx": 0},
               {"mean": 0}, {"rstd": 0}, {"ws": 0}, {"ws": A + 8}, {"x": A + 1}, {"dy": A + 2}, {"dx": A + 3},
               {"g": A + 1}, {"dg": A + 2}, {"db": A + 1}, {"mean": A + 1}):
        assert norm_bwd(**kw) == 1, kw
    assert norm_fwd(x=0, y=0, M=0) == 0 and norm_fwd(x=0, y=0, N=0, ldx=0, ldy=0) == 0
    assert dyt.dyt_last_launch_info()["kernels"] == 0 and dyt.dyt_last_launch_info()["op"] == 5
    assert norm_bwd(x=0, M=0, dg=None, db=None) == 0
    for M, N, xd in ((-1, 4, 0), (0, 4, 0), (4, 0, 0), (4, 4, 7)):
        assert dyt.dyt_layer_norm_backward_workspace_bytes(M, N, xd) == 0


def loss_fwd(z=A, ld=8, tok=A, tb=8, old=A, ref=A, adv=A, w=A, lo=0.2, hi=0.2, kl=0.1, T=1.0, loss=A, logp=A, stats=A,
             coef=A, M=4, N=8, dt=0, ws=A, n=1 << 20):
    return dyt.dyt_policy_loss_forward(z, ld, tok, tb, old, ref, adv, w, lo, hi, kl, T, loss, logp, stats, coef, M, N,
                                       dt, ws, n, None)


def loss_bwd(z=A, ld=8, tok=A, tb=8, stats=A, coef=A, grad=A, T=1.0, dz=A, lddz=8, M=4, N=8, dt=0):
    return dyt.dyt_policy_loss_backward(z, ld, tok, tb, stats, coef, grad, T, dz, lddz, M, N, dt, None)


def test_loss_refusals():
    nan, inf = float("nan"), float("inf")
    for kw in ({"M": -1}, {"N": -1}, {"N": 0, "ld": 0}, {"ld": 7}, {"tb": 2}, {"tb": 0}, {"z": 0}, {"tok": 0},
               {"old": 0}, {"adv": 0}, {"loss": 0}, {"logp": 0}, {"stats": 0}, {"coef": 0}, {"ws": 0}, {"ws": A + 8},
               {"z": A + 2}, {"tok": A + 4}, {"tok": A + 2, "tb": 4}, {"old": A + 1}, {"ref": A + 2}, {"w": A + 2},
               {"stats": A + 4}, {"loss": A + 2}, {"lo": -0.1}, {"lo": nan}, {"hi": inf}, {"hi": -1.0}, {"kl": nan},
               {"kl": inf}, {"T": 0.0}, {"T": -1.0}, {"T": nan}, {"T": inf}, {"T": 1e-60}, {"T": 1e300}):
        assert loss_fwd(**kw) == 1, kw
    assert loss_fwd(dt=3) == 2 and loss_bwd(dt=-1) == 2
    for kw in ({"M": -1}, {"N": -1}, {"ld": 7}, {"lddz": 7}, {"tb": 3}, {"z": 0}, {"tok": 0}, {"stats": 0},
               {"coef": 0}, {"dz": 0}, {"z": A + 2}, {"dz": A + 1}, {"stats": A + 4}, {"coef": A + 2},
               {"grad": A + 1}, {"T": 0.0}, {"T": inf}):
        assert loss_bwd(**kw) == 1, kw
    assert loss_bwd(z=0, M=0) == 0 and loss_bwd(z=0, N=0, ld=0, lddz=0) == 0
    for M, N, d in ((-1, 4, 0), (0, 4, 0), (4, 0, 0), (4, 4, 7)):
        assert dyt.dyt_policy_loss_workspace_bytes(M, N, d) == 0


def test_tensors_must_be_on_a_gpu():
    x = torch.randn(3, 8)
    for call in (lambda: dyt.layer_norm_forward(x), lambda: dyt.layer_norm_backward(x, x, x[:, 0], x[:, 0]),
                 lambda: dyt.policy_loss_forward(x, x[:, 0].long(), x[:, 0], x[:, 0]),
                 lambda: dyt.policy_loss_backward(x, x[:, 0].long(), x[:, :2], x[:, 0])):
        with pytest.raises(ValueError):
            call()
