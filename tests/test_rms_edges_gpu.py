"""Root-mean-square norm, where its definition leaves one answer: the 8-bit values are the
rounded quotients of the norm by its scale, bit for bit, one column's gamma reaches no
other column's group, and a row's bits go by its layout alone."""
from __future__ import annotations

import pytest
import torch

from tests import rms_helpers as S
from tests import row_helpers as R
from tests.rms_helpers import LEAST, QMAX, groups_of
from tests.test_rms_gpu import EPS, INF, NAN, dyt, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")


def quantized(x, residual, gamma, group):
    """(q, scale) from the forward's factors, each operation in binary32 rounded once: the products with the factor
    and with gamma, the largest one's product with the rounded 1 / 448, the quotients, their rounding to 8 bits."""
    rstd = dyt().rms_norm_forward(x, gamma, residual, EPS)[2]
    h = x.float() if residual is None else x.float() + residual.float()
    y = h * rstd[:, None] * gamma.float()
    g = groups_of(y, group)
    scale = torch.maximum(g.abs().amax(-1), y.new_tensor(LEAST)) * y.new_tensor(1 / QMAX)
    q = (g / scale[..., None]).flatten(1)[:, :x.shape[1]].to(torch.float8_e4m3fn)
    return q, scale if group else scale[:, 0], y


def assert_bits(got, want, what):
    a, b = (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t.view(torch.int32) for t in (got, want))
    differ = int((a != b).sum())
    assert differ == 0, f"{what}: {differ} of {a.numel()} differ"


# less than a warp, half of one, a warp, several, clusters of 2 and 4, rows that are read several times
SHAPES = [(20000, 16, "bf16"), (20000, 100, "bf16"), (9000, 255, "f32"), (9000, 256, "bf16"), (5000, 700, "f16"),
          (4096, 1001, "f16"), (3000, 1024, "f32"), (1000, 4096, "bf16"), (1000, 8191, "bf16"), (300, 20480, "bf16"),
          (300, 20481, "f16"), (300, 16384, "f32"), (200, 40000, "bf16"), (100, 70000, "bf16"), (100, 40001, "f32")]


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("M,N,xd", SHAPES)
def test_8_bit_values_are_the_rounded_quotients(M, N, xd, group):
    for res in (False, True):
        x, r, _, gamma = inputs(M, N, xd, xd, res, seed=N)
        rt = None if r is None else r.t
        got = dyt().rms_norm_quantize(x.t, gamma, rt, EPS, group)
        q, scale, _ = quantized(x.t, rt, gamma, group)
        assert_bits(got[1], scale, "scale")
        assert_bits(got[0], q, "q")


@pytest.mark.parametrize("N", [100, 1024, 8192, 20000, 40000])
def test_gamma_whose_product_with_the_sum_passes_binary32(N):
    """The norm is finite although gamma times the sum is not: so are its scales."""
    x, r, _, _ = inputs(50, N, "f32")
    x.t.mul_(1e15)
    r.t.mul_(1e15)
    gamma = torch.full((N,), 1e25, device="cuda")
    for group in (0, 128):
        got = dyt().rms_norm_quantize(x.t, gamma, r.t, EPS, group)
        q, scale, y = quantized(x.t, r.t, gamma, group)
        assert torch.isfinite(y).all() and torch.isfinite(scale).all()
        assert_bits(got[1], scale, "scale")
        assert_bits(got[0], q, "q")


@pytest.mark.parametrize("value", [INF, NAN])
@pytest.mark.parametrize("N,xd", [(100, "bf16"), (1000, "f32"), (4100, "f16"), (20000, "bf16"), (20001, "bf16"),
                                  (40001, "f32"), (40004, "f32"), (65672, "f16"), (70003, "bf16")])
def test_gamma_that_is_not_finite_keeps_to_its_group(N, xd, value):
    """The first column's gamma, with a last group of 128 that is not full."""
    for res in (False, True):
        x, r, dy, gamma = inputs(7, N, xd, res=res)
        rt = None if r is None else r.t
        y0, _, rstd = dyt().rms_norm_forward(x.t, gamma, rt, EPS)
        q0, s0, _ = dyt().rms_norm_quantize(x.t, gamma, rt, EPS, 128)
        h = x.t if rt is None else dyt().rms_norm_forward(x.t, gamma, rt, EPS)[1]
        _, d0 = dyt().rms_norm_backward(h, dy.t, rstd, gamma)
        bad = gamma.clone()
        bad[0] = value
        y, _, again = dyt().rms_norm_forward(x.t, bad, rt, EPS)
        assert torch.equal(y[:, 1:], y0[:, 1:]) and torch.equal(again, rstd) and not torch.isfinite(y[:, 0]).any()
        q, s, _ = dyt().rms_norm_quantize(x.t, bad, rt, EPS, 128)
        assert_bits(s[:, 1:], s0[:, 1:], "scale")
        assert_bits(q[:, 128:], q0[:, 128:], "q")
        q1, s1, _ = dyt().rms_norm_quantize(x.t, bad, rt, EPS, 0)
        if value == INF:  # the group's scale is infinite, and its finite values 0 by it
            assert torch.isinf(s[:, 0]).all() and torch.isinf(s1).all()
            assert (q.float()[:, 1:128] == 0).all() and torch.isnan(q.float()[:, 0]).all()
            assert (q1.float()[:, 1:] == 0).all() and torch.isnan(q1.float()[:, 0]).all()
        else:
            assert torch.isnan(s[:, 0]).all() and torch.isnan(q[:, :128].float()).all()
            assert torch.isnan(s1).all() and torch.isnan(q1.float()).all()
        dx, dg = dyt().rms_norm_backward(h, dy.t, rstd, bad)
        assert torch.equal(dg, d0)  # (gamma is no factor of its own gradient)
        # the row's sum c is not finite, and rstd (g - n c) neither
        assert not torch.isfinite(dx).any()


@pytest.mark.parametrize("N,xd", [(100, "bf16"), (255, "f32"), (1000, "bf16"), (1000, "f32"), (4096, "f16"),
                                  (20000, "bf16")])
def test_the_same_bits_at_every_offset_of_ragged_rows(N, xd):
    """Rows 1, 2, ... elements past a 16-byte boundary, and rows an odd pitch apart: spread over lanes alike."""
    M = 700
    once = None
    for offset, pitch in ((1, N), (2, N), (3, N + 8), (3, N + 1), (1, N + 3), (0, N + 5)):
        x, r, dy, gamma = inputs(M, N, xd, pitch=pitch, offset=offset)
        fwd = dyt().rms_norm_forward(x.t, gamma, r.t, EPS)
        assert dyt().dyt_last_launch_info()["shifted"] == 1
        back = dyt().rms_norm_backward(x.t, dy.t, fwd[2], gamma, r.t)
        eight = [t.view(torch.uint8) for k in (0, 128) for t in dyt().rms_norm_quantize(x.t, gamma, r.t, EPS, k)[:2]]
        all_of = (*fwd, *back, *eight)
        once = once or all_of
        assert all(torch.equal(a, b) for a, b in zip(once, all_of)), (offset, pitch)


@pytest.mark.parametrize("N,xd", [(12288, "bf16"), (20480, "f16"), (9217, "bf16"), (20481, "f16"), (12290, "f32")])
def test_a_row_alone_and_among_others_backward(N, xd):
    """Their clusters, and so the order of the row's sum, may differ: both are within the bound, and they are equal in
    every bit where the launch spreads the row alike."""
    M = 4000
    x, r, dy, gamma = inputs(M, N, xd)
    rstd = dyt().rms_norm_forward(x.t, gamma, r.t, EPS)[2]
    among, _ = dyt().rms_norm_backward(x.t, dy.t, rstd, gamma, r.t)
    many = dyt().dyt_last_launch_info()
    at = [0, 1, 149, 2000, M - 1]
    exact, tol = S.backward(x.t[at], dy.t[at], rstd[at], gamma, r.t[at])
    tol = tol[0] + R.half_step(x.t.dtype, exact[0])
    R.assert_close(among[at], exact[0], tol, "dx among others")
    for k, n in enumerate(at):
        row = slice(n, n + 1)
        alone, _ = dyt().rms_norm_backward(x.t[row], dy.t[row], rstd[row], gamma, r.t[row])
        one = dyt().dyt_last_launch_info()
        R.assert_close(alone, exact[0][k:k + 1], tol[k:k + 1], "dx alone")
        lanes = [(i["col_chunks"], i["block"] // i["row_lanes"]) for i in (one, many)]
        if lanes[0] == lanes[1]:
            assert torch.equal(alone, among[row])
