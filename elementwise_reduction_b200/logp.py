"""Log probabilities of given tokens, with the entropy and the best alternatives of each
row, from the logits: forward, backward, autograd module.

    lp      = log softmax(logits / temperature)
    logp    = lp[token],  entropy = -sum exp(lp) lp
    top     = the largest logits' columns and lp, of equal logits the lower column first

logits: [..., N], tokens one per row. These are the policy loss's old_logp and ref_logp,
and what a sampler reports of its choice. Rows whose token is ignore_index (padding,
prompts) do not count and are not read. No tensor of the logits' size besides the
gradient is made; row layouts are those of the policy loss.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _abi
from ._tensors import (_bytes, _code, _current, _elsewhere, _fresh, _fresh_matrix, _fresh_rows, _like, _pitch,
                       _scratch, _there, _vector, _workspace, row_pitch)
from .loss import _shape

_F32 = (torch.float32,)
_TOKEN = (torch.int64, torch.int32)
_FORWARD, _BACKWARD = _abi.lib.dyt_log_probs_forward, _abi.lib.dyt_log_probs_backward
_SIZE = "dyt_log_probs_workspace_bytes"


def _top(top: int, N: int) -> None:
    if not 0 <= top <= min(_abi.MAX_TOP, N):
        raise ValueError(f"top must be from 0 to {min(_abi.MAX_TOP, N)}, not {top}")


def log_probs_workspace(logits: torch.Tensor, top: int = 0) -> torch.Tensor:
    """A device workspace large enough for log_probs_forward on the logits' shape and device."""
    if _elsewhere(logits.get_device(), None):
        with _there(logits, None):
            return log_probs_workspace(logits, top)
    M, N = _shape(logits)
    _top(top, N)
    return _scratch(_bytes(_SIZE, logits.get_device(), M, N, top, _code(logits, "logits")), logits.device)


def log_probs_forward(logits: torch.Tensor, tokens: torch.Tensor | None = None, top: int = 0,
                      temperature: float = 1.0, ignore_index: int = -100, ws: torch.Tensor | None = None,
                      stream: torch.cuda.Stream | None = None):
    """(logp, entropy, top_logp, top_tokens, stats): logp and entropy per row, the `top`
    (at most 32) largest logits' log probabilities and columns ([..., top], int64), and
    what log_probs_backward needs, each row's maximum and log of its sum ([..., 2]); all
    but the columns in float32. Without tokens logp is None and every row counts, with
    top 0 both top_ are None. logits may be a row-strided view; tokens are int64 or
    int32, contiguous. A row whose token is ignore_index has zeros (columns: -1)."""
    index = logits.get_device()
    if _elsewhere(index, stream):
        with _there(logits, stream):
            return log_probs_forward(logits, tokens, top, temperature, ignore_index, ws)
    M, N = _shape(logits)
    _top(top, N)
    ld, code, dev, rows = _pitch(logits, "logits"), _code(logits, "logits"), logits.device, logits.shape[:-1]
    if ws is None:
        n, wp = _bytes(_SIZE, index, M, N, top, code), None
        if n > 16:  # (few rows need none)
            ws = _scratch(n, dev)
            wp = ws.data_ptr()
    else:
        wp, n = _workspace(ws, index), ws.numel()
    logp = tp = None
    token_bytes = 8
    if tokens is not None:
        tp, token_bytes = _vector(tokens, "tokens", M, index, _TOKEN), tokens.element_size()
        logp = _fresh_rows(rows, dev)
    entropy = _fresh_rows(rows, dev)
    stats = _fresh_matrix(rows, 2, torch.float32, dev)
    best = ids = None
    if top:
        best, ids = _fresh_matrix(rows, top, torch.float32, dev), _fresh_matrix(rows, top, torch.int64, dev)
    st = _FORWARD(
        logits.data_ptr(), ld, tp, token_bytes, ignore_index, top, temperature,
        None if logp is None else logp.data_ptr(), entropy.data_ptr(), None if best is None else best.data_ptr(),
        None if ids is None else ids.data_ptr(), stats.data_ptr(), M, N, code, wp, n, _current(index))
    if st:
        _abi._check(st, "dyt_log_probs_forward")
    return logp, entropy, best, ids, stats


def log_probs_backward(logits: torch.Tensor, tokens: torch.Tensor | None, stats: torch.Tensor,
                       entropy: torch.Tensor | None = None, grad_logp: torch.Tensor | None = None,
                       grad_entropy: torch.Tensor | None = None, temperature: float = 1.0, ignore_index: int = -100,
                       dlogits: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """The gradient by the logits, in their dtype (one kernel launch), from the forward's
    stats and entropy at the same temperature and ignore_index, and the gradients of logp
    and of entropy (one float32 value per row each; left out: 0). logits and dlogits may
    be row-strided views; dlogits may be logits."""
    index = logits.get_device()
    if _elsewhere(index, stream):
        with _there(logits, stream):
            return log_probs_backward(logits, tokens, stats, entropy, grad_logp, grad_entropy, temperature,
                                      ignore_index, dlogits)
    M, N = _shape(logits)
    ld, code = _pitch(logits, "logits"), _code(logits, "logits")
    if grad_logp is not None and tokens is None:
        raise ValueError("grad_logp needs the tokens")
    if grad_entropy is not None and entropy is None:
        raise ValueError("grad_entropy needs the forward's entropy")
    if dlogits is None:
        dlogits, lddl = _fresh(logits), N
    else:
        lddl = _like(dlogits, "dlogits", logits)
    st = _BACKWARD(
        logits.data_ptr(), ld, None if tokens is None else _vector(tokens, "tokens", M, index, _TOKEN),
        8 if tokens is None else tokens.element_size(), ignore_index, _vector(stats, "stats", 2 * M, index, _F32),
        None if entropy is None else _vector(entropy, "entropy", M, index, _F32),
        None if grad_logp is None else _vector(grad_logp, "grad_logp", M, index, _F32),
        None if grad_entropy is None else _vector(grad_entropy, "grad_entropy", M, index, _F32), temperature,
        dlogits.data_ptr(), lddl, M, N, code, _current(index))
    if st:
        _abi._check(st, "dyt_log_probs_backward")
    return dlogits


class LogProbsFunction(torch.autograd.Function):
    """Autograd wrapper: the logits and three numbers a row are saved (a copy of logits that have no row
    pitch); logp and entropy have gradients, the alternatives none."""

    @staticmethod
    def forward(ctx, logits, tokens, top, temperature, ignore_index):
        tokens = None if tokens is None else tokens.contiguous()
        logits = logits if row_pitch(logits) is not None else logits.contiguous()
        logp, entropy, best, ids, stats = log_probs_forward(logits, tokens, top, temperature, ignore_index)
        ctx.save_for_backward(logits, tokens, stats, entropy)
        ctx.temperature, ctx.ignore_index = temperature, ignore_index
        ctx.set_materialize_grads(False)
        if best is not None:
            ctx.mark_non_differentiable(best, ids)
        return logp, entropy, best, ids

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_logp, grad_entropy, *_):
        logits, tokens, stats, entropy = ctx.saved_tensors
        if grad_logp is None and grad_entropy is None:
            return (None,) * 5
        grad_logp, grad_entropy = (None if g is None else g.contiguous() for g in (grad_logp, grad_entropy))
        dlogits = log_probs_backward(logits, tokens, stats, entropy, grad_logp, grad_entropy, ctx.temperature,
                                     ctx.ignore_index)
        return (dlogits,) + (None,) * 4


class LogProbs(torch.nn.Module):
    """Log probabilities, entropy and alternatives (see the top of this file) as a module
    that holds its constants; returns (logp, entropy, top_logp, top_tokens), None for what
    was not asked for."""

    def __init__(self, top: int = 0, temperature: float = 1.0, ignore_index: int = -100):
        super().__init__()
        self.top, self.temperature, self.ignore_index = top, temperature, ignore_index

    def forward(self, logits: torch.Tensor, tokens: torch.Tensor | None = None):
        return LogProbsFunction.apply(logits, tokens, self.top, self.temperature, self.ignore_index)
