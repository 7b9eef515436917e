"""The root-mean-square norm without a GPU: the plain formulas the GPU tests compare with against autograd, and
the entry points' refusals, which come before any CUDA call."""
from __future__ import annotations

import pytest
import torch

import elementwise_reduction_b200 as dyt
from tests import rms_helpers as S

A = 1 << 20  # a 16-byte aligned stand-in for a device address


def test_norm_formulas_agree_with_autograd():
    torch.manual_seed(0)
    x, r = (torch.randn(5, 11, dtype=torch.float64, requires_grad=True) for _ in range(2))
    g = torch.rand(11, dtype=torch.float64, requires_grad=True)
    uy, uh = (torch.randn(5, 11, dtype=torch.float64) for _ in range(2))
    h = x + r
    y = h / (h.square().mean(-1, keepdim=True) + 1e-3).sqrt() * g
    ((y * uy).sum() + (h * uh).sum()).backward()
    (mine, sum_, rstd), _ = S.forward(x.detach(), r.detach(), g.detach(), 1e-3)
    assert torch.allclose(mine, y, rtol=1e-12, atol=1e-12) and torch.equal(sum_, h.detach())
    (dx, dgamma), _ = S.backward(sum_, uy, rstd, g.detach(), uh)
    for got, want in ((dx, x.grad), (dx, r.grad), (dgamma, g.grad)):
        assert torch.allclose(got, want, rtol=1e-11, atol=1e-12)


def test_the_check_of_an_8_bit_output_finds_mistakes():
    # the plain rounding passes, a value one step off, a wrong scale and a smaller largest value do not
    torch.manual_seed(1)
    x, g = torch.randn(4, 300), 1 + 0.1 * torch.randn(300)
    y = S.groups_of(S.forward(x, None, g, 1e-6)[0][0], 128)
    scale = y.abs().amax(-1) / S.QMAX
    q = (y / scale[..., None]).flatten(-2)[:, :300].float().to(torch.float8_e4m3fn)
    ok = lambda q, s: S.assert_quantized(q, s.float(), x, None, g, 1e-6, 128)  # noqa: E731
    ok(q, scale)
    for row, col in ((0, 5), (3, 299)):
        bad = q.clone()
        bad.view(torch.uint8)[row, col] ^= 1
        with pytest.raises(AssertionError):
            ok(bad, scale)
    for factor in (1.001, 0.999):
        with pytest.raises(AssertionError):
            ok(q, scale * factor)


def rms_fwd(x=A, ldx=8, r=A, ldr=8, g=A, eps=1e-5, y=A, ldy=8, h=A, ldh=8, rstd=A, M=4, N=8, xd=0, gd=0):
    return dyt.dyt_rms_norm_forward(x, ldx, r, ldr, g, eps, y, ldy, h, ldh, rstd, M, N, xd, gd, None)


def rms_q8(x=A, ldx=8, r=A, ldr=8, g=A, eps=1e-5, group=0, q=A, ldq=8, s=A, h=A, ldh=8, M=4, N=8, xd=0, gd=0):
    return dyt.dyt_rms_norm_quantize(x, ldx, r, ldr, g, eps, group, q, ldq, s, h, ldh, M, N, xd, gd, None)


def rms_bwd(h=A, ldh=8, dy=A, lddy=8, rstd=A, g=A, dh=A, lddh=8, dx=A, lddx=8, dg=A, M=4, N=8, xd=0, gd=0, ws=A,
            n=1 << 20):
    return dyt.dyt_rms_norm_backward(h, ldh, dy, lddy, rstd, g, dh, lddh, dx, lddx, dg, M, N, xd, gd, ws, n, None)


def test_norm_refusals():
    nan, inf = float("nan"), float("inf")
    for call in (rms_fwd, rms_q8):
        for kw in ({"M": -1}, {"N": -1}, {"N": 2**31, "ldx": 2**31}, {"M": 2**62}, {"ldx": 7}, {"ldr": 7}, {"ldh": 7},
                   {"ldx": 2**61}, {"ldr": 2**61}, {"x": 0}, {"h": 0}, {"x": A + 2}, {"r": A + 1}, {"h": A + 2},
                   {"g": A + 2}, {"eps": -1e-5}, {"eps": nan}, {"eps": inf}):
            assert call(**kw) == 1, kw
        for kw in ({"xd": 3}, {"xd": -1}, {"gd": 5}):
            assert call(**kw) == 2, kw
        assert call(x=0, M=0) == 0 and call(x=0, N=0) == 0
        assert dyt.dyt_last_launch_info()["kernels"] == 0
    for kw in ({"y": 0}, {"y": A + 1}, {"ldy": 7}, {"rstd": A + 2}):
        assert rms_fwd(**kw) == 1, kw
    for kw in ({"q": 0}, {"ldq": 7}, {"s": 0}, {"s": A + 2}, {"group": 64}, {"group": -128}, {"group": 1}):
        assert rms_q8(**kw) == 1, kw
    for kw in ({"M": -1}, {"N": -1}, {"ldh": 7}, {"lddy": 7}, {"lddh": 7}, {"lddx": 7}, {"h": 0}, {"dy": 0}, {"dx": 0},
               {"rstd": 0}, {"ws": 0}, {"ws": A + 8}, {"h": A + 1}, {"dy": A + 2}, {"dh": A + 2}, {"dx": A + 3},
               {"g": A + 1}, {"dg": A + 2}, {"rstd": A + 1}):
        assert rms_bwd(**kw) == 1, kw
    assert rms_bwd(xd=3) == 2 and rms_bwd(gd=-1) == 2
    assert rms_bwd(h=0, M=0, dg=None) == 0
    for M, N, xd in ((-1, 4, 0), (0, 4, 0), (4, 0, 0), (4, 4, 7)):
        assert dyt.dyt_rms_norm_backward_workspace_bytes(M, N, xd) == 0


def test_tensors_must_be_on_a_gpu():
    x = torch.randn(3, 8)
    for call in (lambda: dyt.rms_norm_forward(x), lambda: dyt.rms_norm_quantize(x),
                 lambda: dyt.rms_norm_backward(x, x, x[:, 0])):
        with pytest.raises(ValueError):
            call()
