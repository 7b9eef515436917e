"""Plain binary64 forms of the root-mean-square norm with bounds on the rounding of
the kernels' arithmetic (see row_helpers: u = 2^-24 a rounding, D the additions behind
a row's sum).

rsqrtf is within 2 units in the last place: 4 u. An e4m3 value is off by at most half
a step: 2^-4 of the power of two below it, or 2^-10 below 2^-6.
"""
from __future__ import annotations

import torch

from tests.row_helpers import U, chain

LEAST, QMAX = 2.0 ** -100, 448.0


def forward(x, residual, gamma, eps):
    """(y, h, rstd) in binary64, and bounds (y's and h's without their last rounding)."""
    h = x.double() if residual is None else x.double() + residual.double()
    N = h.shape[-1]
    g = torch.ones(N, dtype=torch.float64, device=x.device) if gamma is None else gamma.double()
    rstd = 1 / torch.sqrt((h * h).mean(-1) + eps)
    # a row's sum of squares is a binary32 number: beyond its range the factor is 0
    rstd = torch.where((h * h).sum(-1) > torch.finfo(torch.float32).max, torch.zeros_like(rstd), rstd)
    y = h * rstd[..., None] * g
    # the squares: the sum's rounding twice, the product, D additions; 1 / N, the fused addition of eps;
    # half of all that after the root, and rsqrtf's own
    rr = (chain(N) + 5) * U / 2 + 4 * U
    du = 0 if residual is None else U
    return (y, h, rstd), (y.abs() * (rr + du + 2 * U), h.abs() * du, rstd * rr)


def groups_of(v, group):
    """v with its columns in groups (zeros behind the last one): [..., groups, columns]."""
    N = v.shape[-1]
    group = group or N
    pad = torch.zeros(*v.shape[:-1], -N % group, dtype=v.dtype, device=v.device)
    return torch.cat([v, pad], -1).unflatten(-1, (-1, group))


def assert_quantized(q, scale, x, residual, gamma, eps, group):
    """q and scale stand for the norm: each value within half a step and the arithmetic's rounding, each
    group's largest at 448."""
    (y, _, _), (dy, _, _) = forward(x, residual, gamma, eps)
    y, dy, v = groups_of(y, group), groups_of(dy, group), groups_of(q.double(), group)
    a = y.abs().amax(-1)
    s = scale.double().reshape(a.shape)
    assert scale.dtype == torch.float32 and q.dtype == torch.float8_e4m3fn
    none = torch.isnan(a)  # a NaN leaves its group nothing else
    assert torch.equal(torch.isnan(s), none) and torch.isnan(v[none][..., 0]).all(), "NaN"
    y, dy, v, s, a = y[~none], dy[~none], v[~none], s[~none], a[~none]
    want = a.clamp(min=LEAST) / QMAX
    # the largest value's error, its product with the rounded 1 / 448
    assert ((s - want).abs() <= dy.amax(-1) / QMAX + 3 * U * want).all(), "scale"
    # the quotient and the product before the conversion, and the scale's own rounding
    # (next to a power of two the arithmetic may reach the wider step: the value is then that power, all but exactly)
    at = (y.abs() / s[..., None]).nan_to_num().frexp()
    half = torch.ldexp(torch.ones_like(y), at.exponent - 5).clamp(min=2.0 ** -10) * s[..., None]
    off = (v * s[..., None] - y).abs()
    tol = dy + 6 * U * y.abs() + half
    assert (off <= tol).all(), f"q: off by up to {float((off - tol).max()):.3g} over the bound"
    top = v.abs().amax(-1)
    assert torch.equal(top, torch.where(a > LEAST, torch.full_like(top, QMAX), top)), "the largest value is not 448"


def overflowed(want, t):
    """want as type t holds it: from half a step past its largest value on, infinite (fp16: 65504 + 16)."""
    f = torch.finfo(t)
    return torch.where(want.abs() >= f.max * (1 + f.eps / (4 - 2 * f.eps)), want.sign() * float("inf"), want)


def backward(h, dy, rstd, gamma, dres=None):
    """(dx, dgamma) in binary64, and bounds (without the last rounding)."""
    h, dy, rstd = h.double(), dy.double(), rstd.double().reshape(-1, 1)
    N = h.shape[-1]
    g = torch.ones(N, dtype=torch.float64, device=h.device) if gamma is None else gamma.double()
    n, gd = h * rstd, g * dy
    c = (gd * n).mean(-1, keepdim=True)
    dx = rstd * (gd - n * c)
    # the product's factors and 1 / N: 4 u, D additions
    dc = (chain(N) + 5) * U * (gd * n).abs().mean(-1, keepdim=True)
    ddx = rstd * (3 * U * gd.abs() + n.abs() * (dc + 3 * U * c.abs())) + 2 * U * dx.abs()
    if dres is not None:
        dx = dx + dres.double()
        ddx = ddx + U * dx.abs()
    # columns: runs of at most 128 rows and 5 levels of lanes in binary32; n is within u
    return (dx, (dy * n).sum(0)), (ddx, 136 * U * (dy * n).abs().sum(0))
