"""The clipped policy loss with a KL term, from the logits: forward, backward, autograd module.

    lp   = log softmax(logits / temperature)[token]
    r    = exp(lp - old_logp),  q = ref_logp - lp
    loss = sum_i weight_i (-min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) + kl_coef (exp(q) - q - 1))

logits: [..., N], the other inputs one value per row; rows of weight 0 (padding,
prompts) do not count and are not read. No tensor of the logits' size besides
the gradient is made, for logits whose rows are dense and evenly spaced. A batch
cut by one position, logits[:, :-1], is not: the module copies it and the
functions refuse it. Take the whole logits instead, with weight 0 at the last
position: those rows are not read either.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _abi
from ._tensors import (_code, _current, _elsewhere, _fresh, _fresh_rows, _like, _pitch, _scratch, _there, _vector,
                       _workspace, row_pitch)

_F32 = (torch.float32,)
_TOKEN = (torch.int64, torch.int32)


def _shape(logits: torch.Tensor) -> tuple[int, int]:
    if logits.dim() == 0 or logits.shape[-1] == 0:
        raise ValueError("logits must have a vocabulary in their last dimension")
    return logits.numel() // logits.shape[-1], logits.shape[-1]


def policy_loss_workspace(logits: torch.Tensor) -> torch.Tensor:
    """A device workspace large enough for policy_loss_forward on the logits' shape and device."""
    if _elsewhere(logits.get_device(), None):
        with _there(logits, None):
            return policy_loss_workspace(logits)
    M, N = _shape(logits)
    n = _abi.lib.dyt_policy_loss_workspace_bytes(M, N, _code(logits, "logits"))
    return _scratch(n, logits.device)


def policy_loss_forward(logits: torch.Tensor, tokens: torch.Tensor, old_logp: torch.Tensor, advantage: torch.Tensor,
                        ref_logp: torch.Tensor | None = None, weight: torch.Tensor | None = None,
                        clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0,
                        temperature: float = 1.0, ws: torch.Tensor | None = None,
                        stream: torch.cuda.Stream | None = None):
    """(loss, logp, stats, coef) in float32: the loss (no dimension), each row's log
    probability of its token, and what policy_loss_backward needs: each row's maximum
    and log of its sum ([..., 2]) and the loss's derivative by its log probability.
    logits may be a row-strided view; tokens are int64 or int32, the other inputs
    float32, contiguous. Without weight every row weighs 1 / rows; without ref_logp
    (or with kl_coef 0) there is no KL term."""
    index = logits.get_device()
    if _elsewhere(index, stream):
        with _there(logits, stream):
            return policy_loss_forward(logits, tokens, old_logp, advantage, ref_logp, weight, clip_low, clip_high,
                                       kl_coef, temperature, ws)
    M, N = _shape(logits)
    ld, code, dev, rows = _pitch(logits, "logits"), _code(logits, "logits"), logits.device, logits.shape[:-1]
    if ws is None:
        n = _abi.lib.dyt_policy_loss_workspace_bytes(M, N, code)
        ws = _scratch(n, dev)
        wp = ws.data_ptr()
    else:
        wp, n = _workspace(ws, index), ws.numel()
    loss = torch.empty_strided((), (), dtype=torch.float32, device=dev)
    logp, coef = _fresh_rows(rows, dev), _fresh_rows(rows, dev)
    stats = (torch.empty_strided((M, 2), (2, 1), dtype=torch.float32, device=dev) if len(rows) == 1 else
             torch.empty((*rows, 2), dtype=torch.float32, device=dev))
    st = _abi.lib.dyt_policy_loss_forward(
        logits.data_ptr(), ld, _vector(tokens, "tokens", M, index, _TOKEN), tokens.element_size(),
        _vector(old_logp, "old_logp", M, index, _F32),
        None if ref_logp is None else _vector(ref_logp, "ref_logp", M, index, _F32),
        _vector(advantage, "advantage", M, index, _F32),
        None if weight is None else _vector(weight, "weight", M, index, _F32), clip_low, clip_high, kl_coef,
        temperature, loss.data_ptr(), logp.data_ptr(), stats.data_ptr(), coef.data_ptr(), M, N, code,
        wp, n, _current(index))
    if st:
        _abi._check(st, "dyt_policy_loss_forward")
    return loss, logp, stats, coef


def policy_loss_backward(logits: torch.Tensor, tokens: torch.Tensor, stats: torch.Tensor, coef: torch.Tensor,
                         grad: torch.Tensor | None = None, temperature: float = 1.0,
                         dlogits: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """The loss's gradient by the logits, in their dtype (one kernel launch), from what
    policy_loss_forward returned at the same temperature. grad: the loss's own gradient
    (one float32 value on the device; left out: 1). logits and dlogits may be
    row-strided views; dlogits may be logits."""
    index = logits.get_device()
    if _elsewhere(index, stream):
        with _there(logits, stream):
            return policy_loss_backward(logits, tokens, stats, coef, grad, temperature, dlogits)
    M, N = _shape(logits)
    ld, code, dev = _pitch(logits, "logits"), _code(logits, "logits"), logits.device
    if dlogits is None:
        dlogits, lddl = _fresh(logits), N
    else:
        lddl = _like(dlogits, "dlogits", logits)
    st = _abi.lib.dyt_policy_loss_backward(
        logits.data_ptr(), ld, _vector(tokens, "tokens", M, index, _TOKEN), tokens.element_size(),
        _vector(stats, "stats", 2 * M, index, _F32), _vector(coef, "coef", M, index, _F32),
        None if grad is None else _vector(grad, "grad", 1, index, _F32), temperature, dlogits.data_ptr(), lddl, M, N,
        code, _current(index))
    if st:
        _abi._check(st, "dyt_policy_loss_backward")
    return dlogits


class PolicyLossFunction(torch.autograd.Function):
    """Autograd wrapper: the logits and three numbers a row are saved (a copy of logits that have no row
    pitch); the gradient goes to the logits alone."""

    @staticmethod
    def forward(ctx, logits, tokens, old_logp, advantage, ref_logp, weight, clip_low, clip_high, kl_coef,
                temperature):
        tokens, old_logp, advantage, ref_logp, weight = (
            None if t is None else t.contiguous() for t in (tokens, old_logp, advantage, ref_logp, weight))
        logits = logits if row_pitch(logits) is not None else logits.contiguous()
        loss, _, stats, coef = policy_loss_forward(logits, tokens, old_logp, advantage, ref_logp, weight, clip_low,
                                                   clip_high, kl_coef, temperature)
        ctx.save_for_backward(logits, tokens, stats, coef)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        logits, tokens, stats, coef = ctx.saved_tensors
        dlogits = policy_loss_backward(logits, tokens, stats, coef, grad.contiguous(), ctx.temperature)
        return (dlogits,) + (None,) * 9


class PolicyLoss(torch.nn.Module):
    """The clipped policy loss with a KL term (see the top of this file) as a module
    that holds its constants; returns the loss."""

    def __init__(self, clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0, temperature: float = 1.0):
        super().__init__()
        self.clip_low, self.clip_high, self.kl_coef, self.temperature = clip_low, clip_high, kl_coef, temperature

    def forward(self, logits: torch.Tensor, tokens: torch.Tensor, old_logp: torch.Tensor, advantage: torch.Tensor,
                ref_logp: torch.Tensor | None = None, weight: torch.Tensor | None = None) -> torch.Tensor:
        return PolicyLossFunction.apply(logits, tokens, old_logp, advantage, ref_logp, weight, self.clip_low,
                                        self.clip_high, self.kl_coef, self.temperature)
