"""Layer norm's kernels where its other tests do not reach: rows far from zero, constant
rows whose sum rounds, column sums over several runs, in place on ragged rows, frozen
parameters, parameters that the call before has written, calls from two host threads."""
from __future__ import annotations

import pytest
import torch

from tests import row_helpers as R

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
