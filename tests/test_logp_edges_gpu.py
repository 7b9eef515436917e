"""Log probabilities where rows lie far apart: every output and the gradient, in place and
elsewhere, against the binary64 forms at element offsets past 2^31."""
from __future__ import annotations

import pytest
import torch

from tests import logp_helpers as L
from tests import row_helpers as R
from tests.test_logp_gpu import dyt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")


# few rows, in one kernel; rows in two kernels, with and without alternatives
@pytest.mark.parametrize("M,N,pitch,top,kernels", [(3, 3001, (1 << 30) + 8, 10, 1), (5, 70001, (1 << 29) + 1, 20, 1),
                                                  (300, 131072, (1 << 23) + 8, 8, 2),
                                                  (300, 131071, (1 << 23) + 3, 0, 2)])
def test_values_at_offsets_beyond_32_bits(M, N, pitch, top, kernels):
    gen = torch.Generator("cuda").manual_seed(N)

    def wide():
        return torch.empty((M - 1) * pitch + N, dtype=torch.bfloat16, device="cuda").as_strided((M, N), (pitch, 1))

    assert (M - 1) * pitch >= 1 << 31
    z = wide()
    z.copy_(2 * torch.randn(M, N, device="cuda", generator=gen))
    tokens = torch.randint(0, N, (M,), device="cuda", generator=gen)
    tokens[0], tokens[M - 1] = 0, N - 1
    da, db = (torch.randn(M, device="cuda", generator=gen) for _ in range(2))
    got = dyt().log_probs_forward(z, tokens, top)
    assert dyt().dyt_last_launch_info()["kernels"] == kernels
    want, tol = L.forward(z, tokens, top)
    for g, w, t, name in zip(got, want, tol, ("logp", "entropy", "top_logp", "top_tokens", "stats")):
        if g is None:
            assert top == 0 and name.startswith("top")
        elif t is None:
            assert torch.equal(g, w), name
        else:
            R.assert_close(g, w, t, name)
    back, tol = L.backward(z.clone(), tokens, got[4], got[1], da, db)
    tol = tol + R.half_step(z.dtype, back)
    for dz in (wide(), z):  # elsewhere, then in place of the logits
        if dz is not z:
            dz.fill_(7.0)
        assert dyt().log_probs_backward(z, tokens, got[4], got[1], da, db, dlogits=dz) is dz
        R.assert_close(dz, back, tol, "dlogits")
