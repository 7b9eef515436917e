"""Plain binary64 forms of the log probabilities, entropy and alternatives, with bounds
on the rounding of the kernels' arithmetic (see row_helpers)."""
from __future__ import annotations

import torch

from tests.row_helpers import EX2, U


def alternatives(z, top):
    """The `top` largest logits' columns, NaN left out, the lower column first among equal ones; -1 where
    there are none."""
    v = z.double()
    nan = torch.isnan(v)
    order = torch.where(nan, -float("inf"), v).sort(dim=-1, descending=True, stable=True).indices
    last = nan.gather(1, order).to(torch.uint8).sort(dim=-1, stable=True).indices
    ids = order.gather(1, last)[:, :top]
    return torch.where(torch.arange(top, device=z.device) < (~nan).sum(-1, keepdim=True), ids, -1)


def forward(z, tokens, top=0, T=1.0, ignore=-100):
    """(logp, entropy, top_logp, top_tokens, stats) in binary64, and bounds on the kernels' errors."""
    ids = alternatives(z, top)
    z = z.double()
    M, N = z.shape
    on = torch.ones(M, dtype=torch.bool, device=z.device) if tokens is None else tokens != ignore
    m = z.amax(-1)
    m = torch.where(torch.isnan(z).any(-1), torch.where(torch.isnan(z), -float("inf"), z).amax(-1), m)
    e = (z - m[:, None]) / T
    x = e.exp()
    total = x.sum(-1)
    s = total.log()
    xe = torch.where(x == 0, torch.zeros_like(x), x * e)
    entropy = s - xe.sum(-1) / total
    lp = e - s[:, None]
    logp = None
    if tokens is not None:
        ok = (tokens >= 0) & (tokens < N)
        logp = torch.where(ok, lp.gather(1, tokens.clamp(0, N - 1).long()[:, None])[:, 0], float("nan"))
    best = torch.where(ids >= 0, lp.gather(1, ids.clamp(min=0)), float("nan"))
    # The sum, as in the policy loss: each term is off by ex2's bound and its exponent's rounding (3 u of the
    # exponent's size), and passes at most 48 + N / 1024 additions and rescalings.
    many = 48 + N / 1024
    a1 = xe.abs().sum(-1) / total
    a2 = torch.where(x == 0, torch.zeros_like(x), x * e * e).sum(-1) / total
    ds = many * (U + EX2) + 3 * U * a1 / 0.69
    # The second sum's terms are all of one sign: 3 u for the exponent in front and 6 u for each rescaling more;
    # its terms' exponents move it by 3 u of their squares. Divided by the first sum, which is off by ds of it.
    dh = ds * (1 + a1) + a1 * (many * (6 * U + EX2) + 3 * U) + 3 * U * a2
    keep = lambda v: torch.where(on.reshape(-1, *[1] * (v.dim() - 1)), v, torch.zeros_like(v))  # noqa: E731
    out = (None if logp is None else keep(logp), keep(entropy), keep(best),
           torch.where(on[:, None], ids, -1), keep(torch.stack([m, s], -1)))
    tol = (None if logp is None else keep(ds + 2 * U * logp.abs()), keep(dh + 2 * U * entropy.abs()),
           keep(ds[:, None] + 2 * U * best.abs()), None,
           keep(torch.stack([torch.zeros_like(s), ds + 2 * U * s.abs()], -1)))
    return out, tol


def backward(z, tokens, stats, entropy, da, db, T=1.0, ignore=-100):
    """dlogits in binary64, and a bound (without the last rounding)."""
    z, m, s = z.double(), stats.double()[:, :1], stats.double()[:, 1:]
    M, N = z.shape
    zero = torch.zeros(M, 1, dtype=torch.float64, device=z.device)
    a = zero if da is None else da.double()[:, None] / T
    b = zero if db is None else db.double()[:, None] / T
    h = zero if entropy is None or db is None else entropy.double()[:, None]
    if tokens is None:
        off, hit = torch.zeros_like(zero, dtype=torch.bool), zero
    else:
        off = (tokens == ignore)[:, None]
        hit = (torch.arange(N, device=z.device) == tokens[:, None]).double()
        bad = ((tokens < 0) | (tokens >= N))[:, None] & ~off & (a != 0)
        a = torch.where(bad, float("nan"), a)
    off = off | ((a == 0) & (b == 0))
    e = (z - m) / T
    p = (e - s).exp()
    gone = p < 1e-55  # the kernels' exponents end at -200 (base 2)
    lp = torch.where(gone, torch.zeros_like(e), e - s)
    p = torch.where(gone, torch.zeros_like(p), p)
    e = torch.where(gone, torch.zeros_like(e), e)
    f = a + b * (lp + h)
    dz = torch.where(off, torch.zeros_like(p), a * hit - p * f)
    # p: ex2's bound, its exponent's rounding and the constant's, expf's 2 units; the factor: its terms' roundings
    rel = EX2 + 8 * U + 3 * U * (lp.abs() + s.abs() + e.abs()) / 0.69
    size = a.abs() + b.abs() * (h.abs() + s.abs() + e.abs())
    # ex2.approx.ftz gives 0 for powers below 2^-126: that much of the factor is lost at most
    flushed = 2.0 ** -126 * size
    tol = flushed + p * (rel * f.abs() + 8 * U * size) + 2 * U * (a * hit).abs()
    return dz, torch.where(off, torch.zeros_like(tol), tol + U * dz.abs())
