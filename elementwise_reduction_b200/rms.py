"""Root-mean-square norm with the addition of a residual stream: forward, an output
in 8 bits with scales, backward, autograd module.

    h = x + residual      (x itself without a residual)
    y = gamma * h * rstd,  rstd = (mean(h^2) + eps)^(-1/2)      (x: [..., N]; rstd: per row; gamma: [N])

y is computed from the sum before it is rounded to h. Row layouts, dtypes and
streams are those of layer norm.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _abi
from ._tensors import (DTYPE_CODE, _bytes, _code, _current, _elsewhere, _fresh, _fresh_matrix, _fresh_rows, _like,
                       _pitch, _rows_of, _scratch, _there, _vector, _workspace, row_pitch)
from .norm import _shape

_F32 = (torch.float32,)
_PARAM = DTYPE_CODE
_FORWARD, _QUANTIZE = _abi.lib.dyt_rms_norm_forward, _abi.lib.dyt_rms_norm_quantize
_BACKWARD, _SIZE = _abi.lib.dyt_rms_norm_backward, "dyt_rms_norm_backward_workspace_bytes"
SCALE_COLUMNS = 128  # columns of a group of the 8-bit output


def rms_norm_forward(x: torch.Tensor, gamma: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                     eps: float = 1e-6, out: torch.Tensor | None = None, residual_out: torch.Tensor | None = None,
                     rstd: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """(y, h, rstd): y and the new residual stream h in x's dtype (without a residual h
    is x), the rows' factors in float32 (one kernel launch). x, residual, out and
    residual_out may be row-strided views (dense rows, evenly spaced): no copy is made.
    gamma may have its own dtype, or be left out. residual_out may be residual or x,
    and so may out, but not the same tensor as residual_out. (Without a residual, out = x
    leaves no h: what is returned as h then holds y.)"""
    index = x.get_device()
    if _elsewhere(index, stream):
        with _there(x, stream):
            return rms_norm_forward(x, gamma, residual, eps, out, residual_out, rstd)
    M, N, ldx, code = _rows_of(x, "x")
    gp, gd, rp, ldr, hp, ldh, h = None, code, None, N, None, N, x
    if gamma is not None:
        gp, gd = _vector(gamma, "gamma", N, index, _PARAM), DTYPE_CODE[gamma.dtype]
    if residual is not None:
        rp, ldr = residual.data_ptr(), _like(residual, "residual", x)
        if residual_out is None:
            h = _fresh(x)
        else:
            h, ldh = residual_out, _like(residual_out, "residual_out", x)
        hp = h.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if out is None:
        y, ldy = _fresh(x), N
    else:
        y, ldy = out, _like(out, "out", x)
    if rstd is None:
        rstd = _fresh_rows(x.shape[:-1], x.device)
    else:
        _vector(rstd, "rstd", x.shape[:-1].numel(), index, _F32)
    st = _FORWARD(x.data_ptr(), ldx, rp, ldr, gp, eps, y.data_ptr(), ldy, hp, ldh, rstd.data_ptr(), M, N, code, gd,
                  _current(index))
    if st:
        _abi._check(st, "dyt_rms_norm_forward")
    if N == 0:  # no elements: no statistics, and no kernel that would write them
        rstd.fill_(float("nan"))
    return y, h, rstd


def rms_norm_quantize(x: torch.Tensor, gamma: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                      eps: float = 1e-6, group: int = 0, out: torch.Tensor | None = None,
                      scale: torch.Tensor | None = None, residual_out: torch.Tensor | None = None,
                      stream: torch.cuda.Stream | None = None):
    """(q, scale, h): the norm as float8_e4m3fn values q that stand for q * scale, and
    the new residual stream h as in rms_norm_forward (one kernel launch). group 0: a
    float32 scale per row ([...]); group 128: one for each 128 columns ([...,
    ceil(N / 128)]). The largest value of a scale's columns becomes 448; q is the
    quotient of rms_norm_forward's y, before that is rounded, by its scale. out may be a
    row-strided view. No gradient: this is the input of an 8-bit product."""
    index = x.get_device()
    if _elsewhere(index, stream):
        with _there(x, stream):
            return rms_norm_quantize(x, gamma, residual, eps, group, out, scale, residual_out)
    if group not in (0, SCALE_COLUMNS):
        raise ValueError(f"group must be 0 (a scale per row) or {SCALE_COLUMNS}, not {group}")
    M, N, ldx, code = _rows_of(x, "x")
    rows, dev = x.shape[:-1], x.device
    gp, gd, rp, ldr, hp, ldh, h = None, code, None, N, None, N, x
    if gamma is not None:
        gp, gd = _vector(gamma, "gamma", N, index, _PARAM), DTYPE_CODE[gamma.dtype]
    if residual is not None:
        rp, ldr = residual.data_ptr(), _like(residual, "residual", x)
        if residual_out is None:
            h = _fresh(x)
        else:
            h, ldh = residual_out, _like(residual_out, "residual_out", x)
        hp = h.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if out is None:
        q, ldq = _fresh_matrix(rows, N, torch.float8_e4m3fn, dev), N
    else:
        q = out
        if q.shape != x.shape or q.dtype != torch.float8_e4m3fn or q.get_device() != index:
            raise ValueError("out must match x in shape and device, in float8_e4m3fn")
        ldq = _pitch(q, "out")
    groups = -(-N // group) if group else 1
    if scale is None:
        scale = _fresh_matrix(rows, groups, torch.float32, dev) if group else _fresh_rows(rows, dev)
    else:
        _vector(scale, "scale", rows.numel() * groups, index, _F32)
    st = _QUANTIZE(x.data_ptr(), ldx, rp, ldr, gp, eps, group, q.data_ptr(), ldq, scale.data_ptr(), hp, ldh, M, N, code,
                   gd, _current(index))
    if st:
        _abi._check(st, "dyt_rms_norm_quantize")
    if N == 0:
        scale.fill_(2.0 ** -100 / 448)  # the largest of no values is 0
    return q, scale, h


def rms_norm_workspace(x: torch.Tensor) -> torch.Tensor:
    """A device workspace large enough for rms_norm_backward on x's shape and device."""
    if _elsewhere(x.get_device(), None):
        with _there(x, None):
            return rms_norm_workspace(x)
    M, N = _shape(x)
    return _scratch(_bytes(_SIZE, x.get_device(), M, N, _code(x, "x")), x.device)


def rms_norm_backward(h: torch.Tensor, dy: torch.Tensor, rstd: torch.Tensor, gamma: torch.Tensor | None = None,
                      dresidual: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                      dgamma: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                      stream: torch.cuda.Stream | None = None, frozen: bool = False):
    """(dx, dgamma) from the forward's h and rstd: dx, the gradient of x and of the
    residual alike, in h's dtype, and dgamma in gamma's (None without gamma).
    dresidual: the gradient that h itself received; it is added to dx. h, dy, dresidual
    and dx may be row-strided views; dx may be any of the others. frozen: gamma's
    gradient is not wanted (None; dx alone then takes one kernel launch less)."""
    index = h.get_device()
    if _elsewhere(index, stream):
        with _there(h, stream):
            return rms_norm_backward(h, dy, rstd, gamma, dresidual, dx, dgamma, ws, frozen=frozen)
    M, N, ldh, code = _rows_of(h, "h")
    lddy = _like(dy, "dy", h)
    rp, lddr = (None, N) if dresidual is None else (dresidual.data_ptr(), _like(dresidual, "dresidual", h))
    if dx is None:
        dx, lddx = _fresh(h), N
    else:
        lddx = _like(dx, "dx", h)
    gp = gg = None
    gd = code
    if (gamma is None or frozen) and dgamma is not None:
        raise ValueError("dgamma needs its parameter, and one that is not frozen")
    if gamma is not None:
        gp, gd = _vector(gamma, "gamma", N, index, _PARAM), DTYPE_CODE[gamma.dtype]
        if frozen:
            pass
        elif dgamma is None:
            dgamma = torch.empty_like(gamma)
            gg = dgamma.data_ptr()
        else:
            gg = _vector(dgamma, "dgamma", N, index, (gamma.dtype,))
    if ws is None:
        n, wp = _bytes(_SIZE, index, M, N, code), None
        if n > 16:  # (few rows need none)
            ws = _scratch(n, h.device)
            wp = ws.data_ptr()
    else:
        wp, n = _workspace(ws, index), ws.numel()
    st = _BACKWARD(
        h.data_ptr(), ldh, dy.data_ptr(), lddy, _vector(rstd, "rstd", h.shape[:-1].numel(), index, _F32), gp, rp,
        lddr, dx.data_ptr(), lddx, gg, M, N, code, gd, wp, n, _current(index))
    if st:
        _abi._check(st, "dyt_rms_norm_backward")
    return dx, dgamma


class RMSNormFunction(torch.autograd.Function):
    """Autograd wrapper: the sum and the rows' factors are saved, the rest is recomputed. Returns y, or
    (y, h) with a residual."""

    @staticmethod
    def forward(ctx, x, residual, gamma, eps):
        gamma = None if gamma is None else gamma.contiguous()
        x, residual = (t if t is None or row_pitch(t) is not None else t.contiguous() for t in (x, residual))
        y, h, rstd = rms_norm_forward(x, gamma, residual, eps)
        ctx.save_for_backward(h, rstd, gamma)
        ctx.set_materialize_grads(False)
        return y if residual is None else (y, h)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, rstd, gamma = ctx.saved_tensors
        want_x, want_residual, want_gamma, _ = ctx.needs_input_grad
        if dy is None:  # y was not used
            return dh if want_x else None, dh if want_residual else None, None, None
        dy, dh = (t if t is None or row_pitch(t) is not None else t.contiguous() for t in (dy, dh))
        dx, dgamma = rms_norm_backward(h, dy, rstd, gamma, dh, frozen=not want_gamma)
        return dx if want_x else None, dx if want_residual else None, dgamma, None


class RMSNorm(torch.nn.Module):
    """gamma * h * rstd over the last dimension, h = x or x + residual.

    forward(x) returns y; forward(x, residual) returns (y, h), h being the residual
    stream for the next block. gamma has one entry per channel and lives in
    ``param_dtype``; its gradient comes back in that dtype. ``affine=False`` leaves
    it out.
    """

    def __init__(self, num_features: int, eps: float = 1e-6, affine: bool = True, param_dtype=torch.float32,
                 device=None):
        super().__init__()
        self.num_features, self.eps = num_features, eps
        self.register_parameter("gamma", torch.nn.Parameter(
            torch.ones(num_features, dtype=param_dtype, device=device)) if affine else None)

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        if x.shape[-1:] != (self.num_features,):
            raise ValueError(f"x's last dimension {tuple(x.shape)} must be {self.num_features}")
        return RMSNormFunction.apply(x, residual, self.gamma, self.eps)
