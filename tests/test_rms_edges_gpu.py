"""Root-mean-square norm, where its definition leaves one answer: the 8-bit values are the
rounded quotients of the norm by its scale, bit for bit, and one column's gamma reaches no
other column's group."""
from __future__ import annotations

import pytest
import torch

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
