"""Layer norm, the layer that DyT takes the place of: forward, backward, autograd module.

    y = gamma * (x - mean) * rstd + beta      (x: [..., N]; mean, rstd: per row; gamma/beta: [N])

Row layouts, dtypes and streams are those of DyT's forward and backward.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _abi
from ._tensors import (DTYPE_CODE, _code, _current, _elsewhere, _fresh, _fresh_rows, _like, _pitch, _scratch, _there,
                       _vector, _workspace, row_pitch)

_F32 = (torch.float32,)
_PARAM = DTYPE_CODE


def _shape(x: torch.Tensor) -> tuple[int, int]:
    if x.dim() == 0:
        raise ValueError("x must have at least one dimension")
    N = x.shape[-1]
    return (x.numel() // N if N else 0), N


def layer_norm_forward(x: torch.Tensor, gamma: torch.Tensor | None = None, beta: torch.Tensor | None = None,
                       eps: float = 1e-5, out: torch.Tensor | None = None, mean: torch.Tensor | None = None,
                       rstd: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """(y, mean, rstd): y in x's dtype, the rows' statistics in float32 (one kernel
    launch). x and out may be row-strided views (dense rows, evenly spaced): no copy
    is made. gamma and beta may each have their own dtype, or be left out. out may
    be x."""
    index = x.get_device()
    if _elsewhere(index, stream):
        with _there(x, stream):
            return layer_norm_forward(x, gamma, beta, eps, out, mean, rstd)
    M, N = _shape(x)
    ldx, code, dev = _pitch(x, "x"), _code(x, "x"), x.device
    gp = None if gamma is None else _vector(gamma, "gamma", N, index, _PARAM)
    bp = None if beta is None else _vector(beta, "beta", N, index, _PARAM)
    if out is None:
        y, ldy = _fresh(x), N
    else:
        y, ldy = out, _like(out, "out", x)
    rows = x.shape[:-1]
    if mean is None:
        mean = _fresh_rows(rows, dev)
    else:
        _vector(mean, "mean", rows.numel(), index, _F32)
    if rstd is None:
        rstd = _fresh_rows(rows, dev)
    else:
        _vector(rstd, "rstd", rows.numel(), index, _F32)
    st = _abi.lib.dyt_layer_norm_forward(
        x.data_ptr(), ldx, gp, bp, eps, y.data_ptr(), ldy, mean.data_ptr(), rstd.data_ptr(), M, N, code,
        code if gamma is None else DTYPE_CODE[gamma.dtype], code if beta is None else DTYPE_CODE[beta.dtype],
        _current(index))
    if st:
        _abi._check(st, "dyt_layer_norm_forward")
    if N == 0:  # no elements: no statistics, and no kernel that would write them
        mean.fill_(float("nan"))
        rstd.fill_(float("nan"))
    return y, mean, rstd


def layer_norm_workspace(x: torch.Tensor) -> torch.Tensor:
    """A device workspace large enough for layer_norm_backward on x's shape and device."""
    if _elsewhere(x.get_device(), None):
        with _there(x, None):
            return layer_norm_workspace(x)
    M, N = _shape(x)
    n = _abi.lib.dyt_layer_norm_backward_workspace_bytes(M, N, _code(x, "x"))
    return _scratch(n, x.device)


def layer_norm_backward(x: torch.Tensor, dy: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        gamma: torch.Tensor | None = None, beta: torch.Tensor | None = None,
                        dx: torch.Tensor | None = None, dgamma: torch.Tensor | None = None,
                        dbeta: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                        stream: torch.cuda.Stream | None = None, frozen: bool = False):
    """(dx, dgamma, dbeta) from the forward's statistics: dx in x's dtype and each
    parameter's gradient in its parameter's dtype (None for a parameter that is not
    given; beta's values are not read). x, dy and dx may be row-strided views; dx may
    be x or dy. frozen: gamma's gradient is not wanted (None; dx alone then takes one
    kernel launch less)."""
    index = x.get_device()
    if _elsewhere(index, stream):
        with _there(x, stream):
            return layer_norm_backward(x, dy, mean, rstd, gamma, beta, dx, dgamma, dbeta, ws, frozen=frozen)
    M, N = _shape(x)
    ldx, code, dev = _pitch(x, "x"), _code(x, "x"), x.device
    lddy = _like(dy, "dy", x)
    if dx is None:
        dx, lddx = _fresh(x), N
    else:
        lddx = _like(dx, "dx", x)
    gp = None if gamma is None else _vector(gamma, "gamma", N, index, _PARAM)
    if beta is not None:
        _vector(beta, "beta", N, index, _PARAM)
    if ((gamma is None or frozen) and dgamma is not None) or (beta is None and dbeta is not None):
        raise ValueError("dgamma and dbeta need their parameters, and dgamma one that is not frozen")
    gd = bd = code
    gg = bg = None
    if gamma is not None:
        gd = DTYPE_CODE[gamma.dtype]
        if frozen:
            pass
        elif dgamma is None:
            dgamma = torch.empty_like(gamma)
            gg = dgamma.data_ptr()
        else:
            gg = _vector(dgamma, "dgamma", N, index, (gamma.dtype,))
    if beta is not None:
        bd = DTYPE_CODE[beta.dtype]
        if dbeta is None:
            dbeta = torch.empty_like(beta)
            bg = dbeta.data_ptr()
        else:
            bg = _vector(dbeta, "dbeta", N, index, (beta.dtype,))
    rows = x.shape[:-1].numel()
    if ws is None:
        n = _abi.lib.dyt_layer_norm_backward_workspace_bytes(M, N, code)
        ws = _scratch(n, dev)
        wp = ws.data_ptr()
    else:
        wp, n = _workspace(ws, index), ws.numel()
    st = _abi.lib.dyt_layer_norm_backward(
        x.data_ptr(), ldx, dy.data_ptr(), lddy, gp, _vector(mean, "mean", rows, index, _F32),
        _vector(rstd, "rstd", rows, index, _F32), dx.data_ptr(), lddx, gg, bg, M, N, code, gd, bd, wp, n,
        _current(index))
    if st:
        _abi._check(st, "dyt_layer_norm_backward")
    return dx, dgamma, dbeta


class LayerNormFunction(torch.autograd.Function):
    """Autograd wrapper: x and the rows' statistics are saved, the rest is recomputed."""

    @staticmethod
    def forward(ctx, x, gamma, beta, eps):
        gamma, beta = (None if t is None else t.contiguous() for t in (gamma, beta))
        x = x if row_pitch(x) is not None else x.contiguous()
        y, mean, rstd = layer_norm_forward(x, gamma, beta, eps)
        ctx.save_for_backward(x, mean, rstd, gamma, beta)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, mean, rstd, gamma, beta = ctx.saved_tensors
        dy = dy if row_pitch(dy) is not None else dy.contiguous()
        _, want_gamma, want_beta, _ = ctx.needs_input_grad
        dx, dgamma, dbeta = layer_norm_backward(x, dy, mean, rstd, gamma, beta if want_beta else None,
                                                frozen=not want_gamma)
        return dx, dgamma, dbeta, None


class LayerNorm(torch.nn.Module):
    """gamma * (x - mean) * rstd + beta over the last dimension.

    gamma and beta have one entry per channel and live in ``param_dtype``; each
    gradient comes back in that dtype. ``affine=False`` leaves both out,
    ``bias=False`` beta alone.
    """

    def __init__(self, num_features: int, eps: float = 1e-5, affine: bool = True, bias: bool = True,
                 param_dtype=torch.float32, device=None):
        super().__init__()
        self.eps = eps
        make = lambda fill: torch.nn.Parameter(torch.full((num_features,), fill, dtype=param_dtype,  # noqa: E731
                                                          device=device))
        self.num_features = num_features
        self.register_parameter("gamma", make(1.0) if affine else None)
        self.register_parameter("beta", make(0.0) if affine and bias else None)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1:] != (self.num_features,):
            raise ValueError(f"x's last dimension {tuple(x.shape)} must be {self.num_features}")
        return LayerNormFunction.apply(x, self.gamma, self.beta, self.eps)
