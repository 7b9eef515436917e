"""Plain binary64 forms of layer norm and of the clipped policy loss, with bounds
on the rounding of the kernels' arithmetic, and tensors with guarded surroundings.

u = 2^-24 is binary32's half step. Each bound adds what the kernels round: sums of
n values reached through at most D additions each are off by at most D u sum |v|
(to first order), each product or difference by u relative, the final rounding to a
type t by torch.finfo(t).eps / 2 relative (half its smallest step near 0).
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
EX2 = 2.0 ** -22  # the bound of ex2.approx.ftz.f32, relative
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def half_step(t: torch.dtype, v: torch.Tensor) -> torch.Tensor:
    """Half a step of t at v (binary64 values)."""
    f = torch.finfo(t)
    return v.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def assert_close(got: torch.Tensor, want: torch.Tensor, tol: torch.Tensor, what: str) -> None:
    """got (any type) against want within tol (binary64), NaN and infinities in the same places."""
    g = got.double()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(g), torch.isnan(want)), f"{what}: NaN in other places"
    inf = ~fine & ~torch.isnan(want)
    assert torch.equal(g[inf], want[inf]), f"{what}: infinities differ"
    if fine.any():
        over = ((g - want).abs() - tol.expand_as(want))[fine]
        worst = float(over.max())
        assert worst <= 0, (f"{what}: {int((over > 0).sum())} of {over.numel()} values over the bound, "
                            f"by up to {worst:.3g} (error up to {float((g - want).abs()[fine].max()):.3g})")


class Guarded:
    """M rows of N elements, `pitch` apart, `offset` elements past a 16-byte boundary,
    in a buffer filled with `fill` (also between the rows)."""

    def __init__(self, M, N, dtype, pitch=None, offset=0, fill=float("nan"), device="cuda"):
        self.M, self.N, self.pitch = M, N, N if pitch is None else pitch
        self.front = 64 + offset
        size = self.front + (max(M, 1) - 1) * self.pitch + N + 64
        self.fill = fill
        self.buf = torch.full((size,), fill, dtype=dtype, device=device)
        self.t = self.buf.as_strided((M, N), (self.pitch, 1), self.front)

    def set(self, v: torch.Tensor) -> torch.Tensor:
        self.t.copy_(v)
        return self.t

    def assert_surroundings_untouched(self, what: str) -> None:
        inside = torch.zeros(self.buf.shape, dtype=torch.bool, device=self.buf.device)
        inside.as_strided((self.M, self.N), (self.pitch, 1), self.front).fill_(True)
        out = self.buf[~inside]
        want = torch.full_like(out, self.fill)
        assert torch.equal(out.view(torch.uint8), want.view(torch.uint8)), f"{what}: written outside its rows"


# ---- layer norm ----------------------------------------------------------------------------

def chain(N: int) -> int:
    """Additions behind a row sum, at most: a lane's own elements (up to 32 in registers,
    N / 1024 and a vector's 8 more in the long rows' kernels) and 10 levels."""
    return 48 + N // 1024


def norm_forward(x, gamma, beta, eps):
    """(y, mean, rstd) in binary64 and bounds on the kernels' errors in them (y's
    without its last rounding)."""
    x = x.double()
    N = x.shape[-1]
    g = torch.ones(N, dtype=torch.float64, device=x.device) if gamma is None else gamma.double()
    b = torch.zeros(N, dtype=torch.float64, device=x.device) if beta is None else beta.double()
    mean = x.mean(-1, keepdim=True)
    c = x - mean
    var = (c * c).mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    h = c * rstd
    y = g * h + b
    D = chain(N)
    dm = (D + 2) * U * x.abs().mean(-1, keepdim=True)  # the mean's error, also of 1 / N
    # the centred squares: D for their sum, 6 for the differences, the square, 1 / N, the root and
    # the quotient, and the shifted mean's own square
    rr = (D + 8) * U / 2 + 4 * U + (rstd * dm) ** 2
    dh = h.abs() * (rr + 3 * U) + rstd * dm
    dy = g.abs() * dh + 2 * U * ((g * h).abs() + b.abs())
    return (y, mean[..., 0], rstd[..., 0]), (dy, (dm + U * mean.abs())[..., 0], (rstd * (rr + U))[..., 0])


def norm_backward(x, dy, mean, rstd, gamma):
    """(dx, dgamma, dbeta) in binary64, and bounds (without the last rounding)."""
    x, dy = x.double(), dy.double()
    mean, rstd = mean.double().reshape(-1, 1), rstd.double().reshape(-1, 1)
    N = x.shape[-1]
    g = torch.ones(N, dtype=torch.float64, device=x.device) if gamma is None else gamma.double()
    h = (x - mean) * rstd
    gd = g * dy
    c1, c2 = gd.mean(-1, keepdim=True), (gd * h).mean(-1, keepdim=True)
    dx = rstd * (gd - c1 - h * c2)
    D = chain(N)
    d1 = (D + 3) * U * gd.abs().mean(-1, keepdim=True)
    d2 = (D + 6) * U * (gd * h).abs().mean(-1, keepdim=True)
    ddx = rstd * (6 * U * gd.abs() + d1 + h.abs() * (d2 + 4 * U * c2.abs()) + 4 * U * c1.abs()) + 2 * U * dx.abs()
    # columns: runs of at most 128 rows and 5 levels of lanes in binary32; h is within 2 u
    dgamma, dbeta = (dy * h).sum(0), dy.sum(0)
    sg, sb = (dy * h).abs().sum(0), dy.abs().sum(0)
    return (dx, dgamma, dbeta), (ddx, 136 * U * sg, 134 * U * sb)


# ---- policy loss -----------------------------------------------------------------------------

def loss_forward(z, tokens, old, adv, ref=None, weight=None, lo=0.2, hi=0.2, kl=0.0, T=1.0):
    """(loss, logp, stats, coef) in binary64, and bounds on the kernels' errors."""
    z = z.double()
    M, N = z.shape
    w = torch.full((M,), 1.0 / M, dtype=torch.float64, device=z.device) if weight is None else weight.double()
    on = w != 0
    m = z.amax(-1)
    e = (z - m[:, None]) / T
    x = e.exp()
    total = x.sum(-1)
    s = total.log()
    ok = (tokens >= 0) & (tokens < N)
    hit = z.gather(1, tokens.clamp(0, N - 1).long()[:, None])[:, 0]
    lp = torch.where(ok, (hit - m) / T - s, float("nan"))
    A, old = adv.double(), old.double()
    r = (lp - old).exp()
    c = r.clamp(1 - lo, 1 + hi)
    held = r * A > c * A
    each = torch.where(held, -c * A, -r * A)
    d = torch.where(held, torch.zeros_like(A), -r * A)
    steep = (r * A).abs()
    if ref is not None and kl != 0:
        q = ref.double() - lp
        each = each + kl * (torch.expm1(q) - q)
        d = d - kl * torch.expm1(q)
        steep = steep + kl * q.exp()
    zero = torch.zeros_like(lp)
    loss = torch.where(on, w * each, zero).sum()
    # The sum: each term is off by ex2's bound and by its exponent's rounding (the product's and the
    # constant's, u each of the exponent's size), each term passes N / 1024 + 48 additions and as many
    # rescalings by ex2 at most.
    spread = torch.nan_to_num((x * e.abs()).nan_to_num().sum(-1) / total) / 0.69
    ds = (48 + N / 1024) * (U + EX2) + 3 * U * spread
    stats = torch.stack([m, s], -1)
    dcoef = torch.where(on, w.abs() * steep * ds + 2 * U * (w * d).abs(), zero)
    dloss = (w.abs() * steep * ds)[on].nan_to_num().sum() + 2 * U * loss.abs()
    return ((loss, torch.where(on, lp, zero), torch.where(on[:, None], stats, torch.zeros_like(stats)),
             torch.where(on, w * d, zero)),
            # a row that does not count is exactly 0
            (dloss, torch.where(on, ds + 2 * U * lp.abs(), zero),
             torch.stack([zero, torch.where(on, ds + 2 * U * s.abs(), zero)], -1), dcoef))


def loss_backward(z, tokens, stats, coef, grad=1.0, T=1.0):
    """dlogits in binary64, and a bound (without the last rounding)."""
    z, stats, a = z.double(), stats.double(), grad * coef.double()[:, None] / T
    e = (z - stats[:, :1]) / T - stats[:, 1:]
    p = e.exp()
    hit = (torch.arange(z.shape[1], device=z.device) == tokens[:, None]).double()
    dz = torch.where(a == 0, torch.zeros_like(p), a * (hit - p))
    # p: ex2's bound, its exponent's rounding and the constant's, the factor's two roundings
    rel = EX2 + 4 * U + 3 * U * (e.abs() + stats[:, 1:].abs() + ((z - stats[:, :1]) / T).abs()) / 0.69
    return dz, (a.abs() * (p * rel + 2 * U * hit)).nan_to_num() + U * dz.abs()
