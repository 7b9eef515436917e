"""Layer norm's kernels where its other tests do not reach: rows far from zero, constant
rows whose sum rounds, column sums over several runs, in place on ragged rows, frozen
parameters, parameters that the call before has written, calls from two host threads."""
from __future__ import annotations

import pytest
import torch

from tests import row_helpers as R
from tests.test_norm_gpu import check

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")


def dyt():
    import elementwise_reduction_b200 as d
    return d


# widths that leave lanes or parts of vectors without elements: rows in a part of a warp, a warp, several warps
@pytest.mark.parametrize("N", [20, 24, 100, 101, 300, 301, 1000, 1001, 4100, 9000])
@pytest.mark.parametrize("xd", ["f32", "bf16"])
def test_rows_far_from_zero_have_finite_gradients(N, xd):
    # x = mean in every place, mean * rstd beyond binary32: h is 0 in the row and dx = rstd (g - c1)
    M = 7
    g = torch.Generator("cuda").manual_seed(N)
    value = torch.tensor([2e36, -2e36, 3e38, 1.0, 0.0, 5e37, 1e36], device="cuda").to(R.DT[xd])
    x = value[:, None].expand(M, N).contiguous()
    dy = torch.randn(M, N, device="cuda", generator=g).to(R.DT[xd])
    gamma = 1 + 0.2 * torch.randn(N, device="cuda", generator=g)
    mean, rstd = value.float(), torch.full((M,), EPS, device="cuda").rsqrt()
    assert torch.isinf(mean * rstd).any()
    dx, dgamma, dbeta = dyt().layer_norm_backward(x, dy, mean, rstd, gamma, gamma)
    want, tol = R.norm_backward(x, dy, mean, rstd, gamma)
    assert torch.isfinite(want[0]).all()
    R.assert_close(dx, want[0], tol[0] + R.half_step(dx.dtype, want[0]), "dx")
    assert torch.equal(dgamma, torch.zeros_like(dgamma))
    R.assert_close(dbeta, want[2], tol[2] + R.half_step(dbeta.dtype, want[2]), "dbeta")


def test_rows_cut_across_a_dimension_of_one_step():
    # [:, :, :2] of (3, 1, 5, N) has no single pitch: refused, and copied by the modules
    x = torch.randn(3, 1, 5, 40, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    v = x[:, :, :2]
    with pytest.raises(ValueError):
        dyt().layer_norm_forward(v)
    assert torch.equal(dyt().LayerNorm(40, affine=False)(v), dyt().layer_norm_forward(v.contiguous())[0])
    layer = dyt().DyT(40, device="cuda")
    assert torch.equal(layer(v), layer(v.contiguous()))


@pytest.mark.parametrize("N", [64, 1000, 4100, 9001])
def test_parameters_that_the_kernel_before_has_written(N):
    # gamma, beta and the upstream gradient straight from the calls before, with no other kernel between them
    g = torch.Generator("cuda").manual_seed(N)
    x = torch.randn(300, N, device="cuda", generator=g)
    a = torch.randn(1, N, device="cuda", generator=g)
    outs = []
    for wait in (True, False):
        got = []
        rest = lambda: torch.cuda.synchronize() if wait else None  # noqa: E731
        gamma = torch.zeros(1, N, device="cuda")
        y, dgamma = torch.zeros_like(x), torch.zeros(N, device="cuda")
        stats = [torch.zeros(300, device="cuda") for _ in range(2)]
        ws = dyt().layer_norm_workspace(x)
        rest()
        for step in range(4):
            dyt().layer_norm_forward(a * (step + 1.0) if step == 0 else y[:1], out=gamma)
            rest()
            dyt().layer_norm_forward(x, gamma.view(N), gamma.view(N), out=y, mean=stats[0], rstd=stats[1])
            rest()
            dyt().layer_norm_backward(x, y, stats[0], stats[1], gamma.view(N), dx=y, dgamma=dgamma, ws=ws)
            rest()
            dyt().layer_norm_forward(y, dgamma, gamma.view(N), out=y)
            rest()
            got += [y.clone(), dgamma.clone()]
            rest()
        outs.append(got)
    assert all(torch.equal(p, q) for p, q in zip(*outs))


@pytest.mark.parametrize("N", [96, 1001, 9000])
@pytest.mark.parametrize("want_gamma", [True, False])
@pytest.mark.parametrize("want_beta", [True, False])
def test_frozen_parameters(N, want_gamma, want_beta):
    # no gradient, and no kernel for the gradients where none is wanted
    g = torch.Generator("cuda").manual_seed(N)
    x, up = (torch.randn(33, N, device="cuda", generator=g) for _ in range(2))
    full, part = (dyt().LayerNorm(N, device="cuda") for _ in range(2))
    part.gamma.requires_grad_(want_gamma)
    part.beta.requires_grad_(want_beta)
    grads = []
    for layer in (full, part):
        with torch.no_grad():
            layer.gamma.copy_(torch.linspace(0.5, 1.5, N, device="cuda"))
        a = x.clone().requires_grad_()
        layer(a).backward(up)
        grads.append((a.grad, layer.gamma.grad, layer.beta.grad))
    assert torch.equal(grads[1][0], grads[0][0])
    for want, i in ((want_gamma, 1), (want_beta, 2)):
        assert torch.equal(grads[1][i], grads[0][i]) if want else grads[1][i] is None


@pytest.mark.parametrize("N", [96, 9000])
def test_a_frozen_gamma_and_its_refusals(N):
    g = torch.Generator("cuda").manual_seed(N)
    x, dy = (torch.randn(20, N, device="cuda", generator=g) for _ in range(2))
    gamma = torch.rand(N, device="cuda", generator=g)
    _, mean, rstd = dyt().layer_norm_forward(x, gamma, gamma, EPS)
    want = dyt().layer_norm_backward(x, dy, mean, rstd, gamma, gamma)
    kernels = dyt().dyt_last_launch_info()["kernels"]
    got = dyt().layer_norm_backward(x, dy, mean, rstd, gamma, frozen=True)
    assert torch.equal(got[0], want[0]) and got[1] is None and got[2] is None
    assert dyt().dyt_last_launch_info()["kernels"] == kernels - 1
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dyt().layer_norm_backward(x, dy, mean, rstd, gamma, gamma, stream=s, frozen=True)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and got[1] is None and torch.equal(got[2], want[2])
    with pytest.raises(ValueError):
        dyt().layer_norm_backward(x, dy, mean, rstd, gamma, dgamma=gamma.clone(), frozen=True)


# rows side by side in a CTA: part of a warp, a warp and several warps per row, whole vectors and ragged
@pytest.mark.parametrize("N,xd,rows", [(96, "bf16", 64), (30, "f32", 128), (512, "f16", 16), (509, "bf16", 16),
                                       (1024, "bf16", 8), (1021, "f16", 8), (8192, "f32", 1), (7001, "bf16", 1)])
@pytest.mark.parametrize("runs,more", [(2, 3), (1, 1)])
def test_column_sums_over_several_runs(N, xd, rows, runs, more):
    # runs of 128 rows a lane, then `more` rows, of which most rows of the grid do not make the last one
    step = torch.cuda.get_device_properties(0).multi_processor_count * rows
    M = step * (runs * 128 + more - 1) + (rows * 5 + 3 if rows > 1 else 5)
    _, bwd = check(M, N, xd)
    assert bwd["rows_per_step"] == rows and bwd["grid"] * rows == step
    assert -(-M // step) == runs * 128 + more and M % step


@pytest.mark.parametrize("N,xd", [(9000, "bf16"), (9001, "bf16"), (20000, "f32")])
def test_column_sums_of_long_rows_over_several_runs(N, xd):
    # the second pass's row groups take every row_groups-th row
    _, bwd = check(1, N, xd)
    groups = (torch.cuda.get_device_properties(0).multi_processor_count * 4
              // -(-(N // (16 // R.DT[xd].itemsize) if N % 8 == 0 else N) // 256))
    M = groups * (2 * 128 + 3) + 1
    _, bwd = check(M, N, xd)
    assert bwd["row_groups"] == groups and M > 256 * groups


@pytest.mark.parametrize("xd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [3, 61, 300, 513, 1001, 4099, 8192, 9001, 20000])
def test_constant_rows_whose_sum_rounds(N, xd):
    # The mean of N times c is off by the sum's rounding alone: D u |c| (D additions, see row_helpers.chain),
    # two halves of a step more. eps bounds what is left: |y| <= |mean error| / sqrt(eps).
    value = torch.tensor([0.1, -0.3, 1 / 3, 1e-3, 7.7, 0.0], device="cuda").to(R.DT[xd])
    x = value[:, None].expand(6, N).contiguous()
    gamma = torch.ones(N, device="cuda")
    y, mean, rstd = dyt().layer_norm_forward(x, gamma, None, EPS)
    v = value.double()
    off = (R.chain(N) + 2) * R.U * v.abs()
    R.assert_close(mean, v, off, "mean")
    # the variance that is computed is at most the square of the mean's error
    want = torch.full_like(v, EPS ** -0.5)
    R.assert_close(rstd, want, want * (off.square() / EPS / 2 + 4 * R.U), "rstd")
    t = (off * want)[:, None] * (1 + 4 * R.U)
    R.assert_close(y, torch.zeros_like(y, dtype=torch.float64), t + R.half_step(y.dtype, t), "y")
    assert torch.equal(y[5], torch.zeros_like(y[5]))
    # the gradient with those statistics, against the formula with the same
    dy = torch.randn(6, N, device="cuda", generator=torch.Generator("cuda").manual_seed(N)).to(R.DT[xd])
    dx, dgamma, dbeta = dyt().layer_norm_backward(x, dy, mean, rstd, gamma, gamma)
    want, tol = R.norm_backward(x, dy, mean, rstd, gamma)
    for got, w, b, name in ((dx, want[0], tol[0], "dx"), (dgamma, want[1], tol[1], "dgamma"),
                            (dbeta, want[2], tol[2], "dbeta")):
        R.assert_close(got, w, b + R.half_step(got.dtype, w), name)


@pytest.mark.parametrize("xd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,pitch,offset", [(1500, 9, 9, 1), (1500, 61, 64, 3), (700, 255, 255, 1), (700, 509, 512, 0),
                                              (400, 1001, 1001, 5), (400, 1001, 1008, 0), (50, 8191, 8191, 1),
                                              (20, 9001, 9003, 1), (20, 20001, 20001, 3)])
def test_in_place_on_ragged_rows(M, N, pitch, offset, xd):
    # rows at any offset, one after the other or NaN between them; the output over x, and over dy
    g = torch.Generator("cuda").manual_seed(N)
    v = [torch.randn(M, N, device="cuda", generator=g) for _ in range(2)]
    gamma, beta = (torch.randn(N, device="cuda", generator=g) for _ in range(2))
    make = lambda t: R.Guarded(M, N, R.DT[xd], pitch, offset)  # noqa: E731
    x, dy = make(0), make(0)
    x.set(v[0])
    dy.set(v[1])
    y = make(0)
    _, mean, rstd = dyt().layer_norm_forward(x.t, gamma, beta, EPS, out=y.t)
    dx = make(0)
    want = dyt().layer_norm_backward(x.t, dy.t, mean, rstd, gamma, beta, dx=dx.t)
    for _ in range(3):
        a = make(0)
        a.set(v[0])
        got = dyt().layer_norm_forward(a.t, gamma, beta, EPS, out=a.t)
        assert torch.equal(a.t, y.t) and torch.equal(got[1], mean) and torch.equal(got[2], rstd)
        a.assert_surroundings_untouched("y")
        for which in (0, 1):
            a, b = make(0), make(0)
            a.set(v[0])
            b.set(v[1])
            out = (a, b)[which]
            got = dyt().layer_norm_backward(a.t, b.t, mean, rstd, gamma, beta, dx=out.t)
            assert torch.equal(out.t, dx.t) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
            out.assert_surroundings_untouched("dx")


def test_dyt_on_the_last_position_of_every_sequence():
    g = torch.Generator("cuda").manual_seed(9)
    x, dy = (torch.randn(6, 5, 72, device="cuda", generator=g)[:, -1:] for _ in range(2))
    alpha, gamma, beta = torch.tensor([0.7], device="cuda"), torch.rand(72, device="cuda"), torch.rand(72, device="cuda")
    y = dyt().forward(x, alpha, gamma, beta)
    assert y.shape == x.shape and torch.equal(y, dyt().forward(x.contiguous(), alpha, gamma, beta))
    got = dyt().backward(x, dy, alpha, gamma, beta)
    want = dyt().backward(x.contiguous(), dy.contiguous(), alpha, gamma, beta)
    assert torch.equal(got[0], want[0])
    for a, b in zip(got[1:], want[1:]):  # sums of six rows in binary64, rounded once; another plan may add in another order
        assert torch.allclose(a, b, rtol=4 * R.U, atol=0)
