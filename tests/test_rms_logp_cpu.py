"""The root-mean-square norm and the log probabilities without a GPU: the plain formulas
the GPU tests compare with against autograd, and the entry points' refusals, which come
before any CUDA call."""
from __future__ import annotations

import pytest
import torch

import elementwise_reduction_b200 as dyt
from tests import logp_helpers as L
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


def rms_fwd(x=A, ldx=8, r=A, ldr=8, g=A, eps=1e-5, y=A, ldy=8, h=2 * A, ldh=8, rstd=A, M=4, N=8, xd=0, gd=0):
    return dyt.dyt_rms_norm_forward(x, ldx, r, ldr, g, eps, y, ldy, h, ldh, rstd, M, N, xd, gd, None)


def rms_q8(x=A, ldx=8, r=A, ldr=8, g=A, eps=1e-5, group=0, q=A, ldq=8, s=A, h=2 * A, ldh=8, M=4, N=8, xd=0, gd=0):
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
    for kw in ({"y": 0}, {"y": A + 1}, {"ldy": 7}, {"rstd": A + 2}, {"h": A}):
        assert rms_fwd(**kw) == 1, kw
    for kw in ({"q": 0}, {"ldq": 7}, {"s": 0}, {"s": A + 2}, {"group": 64}, {"group": -128}, {"group": 1}):
        assert rms_q8(**kw) == 1, kw
    for kw in ({"M": -1}, {"N": -1}, {"ldh": 7}, {"lddy": 7}, {"lddh": 7}, {"lddx": 7}, {"h": 0}, {"dy": 0}, {"dx": 0},
               {"rstd": 0}, {"ws": 0, "M": 4000},
               {"ws": 0, "N": 9000, "ldh": 9000, "lddy": 9000, "lddh": 9000, "lddx": 9000},
               {"ws": 0, "N": 70000, "ldh": 70000, "lddy": 70000, "lddh": 70000, "lddx": 70000},
               {"ws": A + 8}, {"h": A + 1}, {"dy": A + 2}, {"dh": A + 2}, {"dx": A + 3},
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


@pytest.mark.parametrize("T", [1.0, 0.7])
def test_log_probability_formulas_agree_with_autograd(T):
    torch.manual_seed(2)
    M, N = 30, 17
    z = torch.randn(M, N, dtype=torch.float64, requires_grad=True)
    tokens = torch.randint(0, N, (M,))
    tokens[::4] = -100
    on = tokens != -100
    a, b = torch.randn(M, dtype=torch.float64), torch.randn(M, dtype=torch.float64)
    lp = (z / T).log_softmax(-1)
    entropy = -(lp.exp() * lp).sum(-1)
    hit = lp.gather(1, tokens.clamp(min=0)[:, None])[:, 0]
    ((hit * a)[on].sum() + (entropy * b)[on].sum()).backward()
    (logp, ent, best, ids, stats), _ = L.forward(z.detach(), tokens, 3, T)
    keep = on.double()
    assert torch.allclose(logp, hit.detach() * keep, rtol=1e-12) and torch.allclose(ent, entropy.detach() * keep)
    assert torch.equal(ids[on], z.detach().topk(3).indices[on]) and (ids[~on] == -1).all()
    assert torch.allclose(best[on], lp.detach().topk(3).values[on]) and (stats[~on] == 0).all()
    dz, _ = L.backward(z.detach(), tokens, stats, ent, a, b, T)
    assert torch.allclose(dz, z.grad, rtol=1e-10, atol=1e-13)
    v, t = torch.randn(M, N, dtype=torch.float64), 1e-6
    def f(y):
        out = L.forward(y, tokens, 0, T)[0]
        return float((out[0] * a + out[1] * b).sum())
    slope = (f(z.detach() + t * v) - f(z.detach() - t * v)) / (2 * t)
    assert abs(slope - float((dz * v).sum())) < 1e-6


def test_alternatives_go_by_column_and_leave_nan_out():
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([[1.0, 2.0, 2.0, 0.0], [nan, -inf, nan, -inf], [0.0, -0.0, nan, inf], [nan] * 4])
    assert L.alternatives(z, 3).tolist() == [[1, 2, 0], [1, 3, -1], [3, 0, 1], [-1, -1, -1]]


def logp_fwd(z=A, ld=8, tok=A, tb=8, ignore=-100, top=3, T=1.0, logp=A, ent=A, best=A, ids=A, stats=A, M=4, N=8, dt=0,
             ws=A, n=1 << 20):
    return dyt.dyt_log_probs_forward(z, ld, tok, tb, ignore, top, T, logp, ent, best, ids, stats, M, N, dt, ws, n,
                                     None)


def logp_bwd(z=A, ld=8, tok=A, tb=8, ignore=-100, stats=A, ent=A, da=A, db=A, T=1.0, dz=A, lddz=8, M=4, N=8, dt=0):
    return dyt.dyt_log_probs_backward(z, ld, tok, tb, ignore, stats, ent, da, db, T, dz, lddz, M, N, dt, None)


def test_log_probability_refusals():
    nan, inf = float("nan"), float("inf")
    for kw in ({"M": -1}, {"N": -1}, {"N": 0, "ld": 0}, {"ld": 7}, {"tb": 2}, {"tb": 0}, {"z": 0}, {"logp": 0},
               {"ent": 0}, {"stats": 0}, {"best": 0}, {"ids": 0}, {"ws": 0, "M": 4000}, {"ws": A + 8}, {"z": A + 2},
               {"tok": A + 4}, {"tok": A + 2, "tb": 4}, {"logp": A + 2}, {"ent": A + 1}, {"best": A + 2},
               {"ids": A + 4}, {"stats": A + 4}, {"top": -1}, {"top": 9}, {"top": 33, "N": 64, "ld": 64}, {"T": 0.0},
               {"T": -1.0}, {"T": nan}, {"T": inf}, {"T": 1e-60}, {"T": 1e300}):
        assert logp_fwd(**kw) == 1, kw
    assert logp_fwd(dt=3) == 2 and logp_bwd(dt=-1) == 2
    for kw in ({"M": -1}, {"N": -1}, {"ld": 7}, {"lddz": 7}, {"tb": 3}, {"z": 0}, {"stats": 0}, {"dz": 0},
               {"z": A + 2}, {"dz": A + 1}, {"stats": A + 4}, {"ent": 0}, {"tok": 0}, {"ent": A + 2}, {"da": A + 2},
               {"db": A + 1}, {"T": 0.0}, {"T": inf}):
        assert logp_bwd(**kw) == 1, kw
    assert logp_fwd(z=0, M=0) == 0 and logp_bwd(z=0, M=0) == 0 and logp_bwd(z=0, N=0, ld=0, lddz=0) == 0
    for M, N, top, d in ((-1, 4, 0, 0), (0, 4, 0, 0), (4, 0, 0, 0), (4, 4, 0, 7), (4, 4, 5, 0), (4, 64, 33, 0)):
        assert dyt.dyt_log_probs_workspace_bytes(M, N, top, d) == 0


def test_logits_must_be_on_a_gpu():
    x = torch.randn(3, 8)
    for call in (lambda: dyt.log_probs_forward(x), lambda: dyt.log_probs_workspace(x),
                 lambda: dyt.log_probs_backward(x, None, x[:, :2])):
        with pytest.raises(ValueError):
            call()
