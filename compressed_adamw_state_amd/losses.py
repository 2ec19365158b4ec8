"""Losses over rows of logits, with gradients the fused steps consume
(include/flashopt_lm.h): log probabilities of given tokens with entropy and
top alternatives, and distillation from a teacher's top alternatives.

Logits are [..., vocab] in BF16, FP16 or FP32; the leading dimensions are the
rows and every output has them.  Two forms of each loss:

* token_logprobs, distill_loss: differentiable (torch.autograd), for losses
  whose upstream gradient is known only after the forward pass;
* token_logprobs_grad, distill_grad: the outputs and the gradient with
  respect to the logits in one call, for upstream gradients known beforehand
  (a mean over tokens); hand it on with logits.backward(grad).  inplace=True
  lets the gradient replace the logits (no second buffer of rows x vocab).

A run of distillation:

    t = token_logprobs(teacher_logits, top=64, temperature=T)
    loss, grad = distill_grad(student_logits, t.top_id, t.top_logprob, weight, temperature=T)
    student_logits.backward(grad)

Inside a HIP graph, capture the *_grad forms (they need no autograd).  This
module only marshals: every sum runs in the HIP library.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import flashopt as F


class TokenLogprobs(NamedTuple):
    logprob: Optional[torch.Tensor]       # [...] FP32; None without targets
    entropy: torch.Tensor                 # [...] FP32
    top_logprob: Optional[torch.Tensor]   # [..., top] FP32, largest first; None for top = 0
    top_id: Optional[torch.Tensor]        # [..., top] int64


class TokenLogprobsGrad(NamedTuple):
    logprob: torch.Tensor
    entropy: torch.Tensor
    grad: torch.Tensor


def _rows(logits: torch.Tensor) -> torch.Tensor:
    """The logits as rows x vocab, without a copy."""
    if not logits.is_cuda:
        raise ValueError("expected device tensors")
    if logits.dim() == 2:
        return logits
    if logits.dim() == 0 or logits.shape[-1] == 0:
        raise ValueError("logits need a vocabulary dimension")
    try:
        return logits.view(-1, logits.shape[-1])
    except RuntimeError:
        raise ValueError("the logits' leading dimensions must flatten without a copy") from None


def _per_row(t: torch.Tensor, shape, device, dtype, name: str) -> torch.Tensor:
    if t.dtype != dtype or t.shape != shape or t.device != device:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)} on {device}")
    F.no_tangent(t, name)
    return t if t.is_contiguous() else t.contiguous()


def _check_temperature(temperature: float) -> float:
    temperature = float(temperature)
    if not 2.0 ** -126 <= temperature <= 2.0 ** 126:
        raise ValueError(f"temperature = {temperature} is outside its range")
    return temperature


def _upstream(g: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    if g is None:
        return None
    if g.dtype != torch.float32:
        g = g.float()
    return g if g.is_contiguous() else g.contiguous()


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _empty(shape, device, dtype=torch.float32) -> torch.Tensor:
    return torch.empty(shape, dtype=dtype, device=device)


def _workspace(need: int, device) -> Optional[torch.Tensor]:
    return _empty(need, device, torch.uint8) if need else None


# Below, the library is called with the addresses of tensors that the checks
# above have seen or that were just made here.

def _forward(logits, lead, targets, top, temperature, keep):
    x, ty, rows, vocab, stride = F._logits(_rows(logits))
    dev = logits.device
    logprob = None if targets is None else _empty(lead, dev)
    entropy = _empty(lead, dev)
    stats = _empty((rows, 4), dev) if keep else None
    tl = ti = None
    if top:
        tl, ti = _empty(lead + (top,), dev), _empty(lead + (top,), dev, torch.int64)
    need = F.lib().flashopt_logprob_workspace_bytes(ty, rows, vocab, top)
    ws = _workspace(need, dev)
    F._call("flashopt_logprob", dev, None, x, ty, rows, vocab, stride, temperature, _at(targets),
            top, _at(ws), need, _at(logprob), entropy.data_ptr(), _at(stats), _at(tl), _at(ti))
    return logprob, entropy, stats, tl, ti


class _Logprob(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, lead, targets, top, temperature):
        logprob, entropy, stats, tl, ti = _forward(logits, lead, targets, top, temperature, True)
        ctx.save_for_backward(logits, targets, stats)
        ctx.temperature = temperature
        ctx.set_materialize_grads(False)
        if top:
            ctx.mark_non_differentiable(tl, ti)
        return logprob, entropy, tl, ti

    @staticmethod
    @once_differentiable
    def backward(ctx, g_logprob, g_entropy, _tl, _ti):
        logits, targets, stats = ctx.saved_tensors
        if g_logprob is None and g_entropy is None:
            return None, None, None, None, None
        g_logprob, g_entropy = _upstream(g_logprob), _upstream(g_entropy)
        x, ty, rows, vocab, stride = F._logits(_rows(logits))
        dev = logits.device
        grad = _empty(logits.shape, dev, logits.dtype)
        F._call("flashopt_logprob_backward", dev, None, x, ty, rows, vocab, stride,
                ctx.temperature, _at(targets), stats.data_ptr(), _at(g_logprob), _at(g_entropy),
                grad.data_ptr(), vocab)
        return grad, None, None, None, None


def token_logprobs(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, top: int = 0,
                   temperature: float = 1.0) -> TokenLogprobs:
    """Per row: the log probability of targets (int64; an id outside the
    vocabulary, such as -100, gives 0 without a gradient), the entropy, and
    the `top` most likely tokens (0 to 64; equal logits by lowest id), of
    softmax(logits / temperature).  logprob and entropy are differentiable."""
    temperature = _check_temperature(temperature)
    F.no_tangent(logits, "logits")
    if top < 0 or top > F.TOP_MAX or top > logits.shape[-1]:
        raise ValueError(f"top = {top} is outside 0 .. {min(F.TOP_MAX, logits.shape[-1])}")
    lead = logits.shape[:-1]
    if targets is not None:
        targets = _per_row(targets, lead, logits.device, torch.int64, "targets")
    if logits.requires_grad and torch.is_grad_enabled():
        return TokenLogprobs(*_Logprob.apply(logits, lead, targets, top, temperature))
    logprob, entropy, _, tl, ti = _forward(logits, lead, targets, top, temperature, False)
    return TokenLogprobs(logprob, entropy, tl, ti)


def _grad_buffer(logits: torch.Tensor, inplace: bool):
    """(the gradient, its row stride)"""
    if inplace:
        return logits.detach(), F.row_stride(_rows(logits))
    return _empty(logits.shape, logits.device, logits.dtype), logits.shape[-1]


def _replaced(logits: torch.Tensor, inplace: bool) -> None:
    """After the call: torch then refuses a backward pass that would read the logits' values."""
    if inplace:
        torch.autograd.graph.increment_version(logits)


def token_logprobs_grad(logits: torch.Tensor, targets: torch.Tensor, grad_logprob: torch.Tensor,
                        grad_entropy: Optional[torch.Tensor] = None, temperature: float = 1.0,
                        inplace: bool = False) -> TokenLogprobsGrad:
    """logprob, entropy and the gradient of sum(grad_logprob * logprob +
    grad_entropy * entropy) with respect to the logits (grad_*: FP32, one per
    row).  inplace: the gradient takes the logits' place, whose values nothing
    else may need any more."""
    temperature = _check_temperature(temperature)
    F.no_tangent(logits, "logits")
    lead, dev = logits.shape[:-1], logits.device
    targets = _per_row(targets, lead, dev, torch.int64, "targets")
    grad_logprob = _per_row(grad_logprob, lead, dev, torch.float32, "grad_logprob")
    if grad_entropy is not None:
        grad_entropy = _per_row(grad_entropy, lead, dev, torch.float32, "grad_entropy")
    x, ty, rows, vocab, stride = F._logits(_rows(logits))
    logprob, entropy = _empty(lead, dev), _empty(lead, dev)
    grad, grad_stride = _grad_buffer(logits, inplace)
    need = F.lib().flashopt_logprob_workspace_bytes(ty, rows, vocab, 0)
    ws = _workspace(need, dev)
    F._call("flashopt_logprob_grad", dev, None, x, ty, rows, vocab, stride, temperature,
            targets.data_ptr(), grad_logprob.data_ptr(), _at(grad_entropy), _at(ws), need,
            logprob.data_ptr(), entropy.data_ptr(), grad.data_ptr(), grad_stride)
    _replaced(logits, inplace)
    return TokenLogprobsGrad(logprob, entropy, grad)


def _distill_forward(logits, lead, top_id, top_logprob, tail, temperature):
    x, ty, rows, vocab, stride = F._logits(_rows(logits))
    dev = logits.device
    loss, stats = _empty(lead, dev), _empty((rows, 8), dev)
    need = F.lib().flashopt_distill_workspace_bytes(ty, rows, vocab)
    ws = _workspace(need, dev)
    F._call("flashopt_distill", dev, None, x, ty, rows, vocab, stride, temperature,
            top_id.data_ptr(), top_logprob.data_ptr(), top_id.shape[-1], tail, _at(ws), need,
            loss.data_ptr(), stats.data_ptr())
    return loss, stats


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, lead, top_id, top_logprob, tail, temperature):
        loss, stats = _distill_forward(logits, lead, top_id, top_logprob, tail, temperature)
        ctx.save_for_backward(logits, top_id, top_logprob, stats)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        logits, top_id, top_logprob, stats = ctx.saved_tensors
        g = _upstream(g)
        x, ty, rows, vocab, stride = F._logits(_rows(logits))
        dev = logits.device
        grad = _empty(logits.shape, dev, logits.dtype)
        F._call("flashopt_distill_backward", dev, None, x, ty, rows, vocab, stride,
                ctx.temperature, top_id.data_ptr(), top_logprob.data_ptr(), top_id.shape[-1],
                stats.data_ptr(), g.data_ptr(), grad.data_ptr(), vocab)
        return grad, None, None, None, None, None


def _teacher(logits, lead, top_id, top_logprob):
    top = top_id.shape[-1] if top_id.dim() else 0
    if top < 1 or top > F.TOP_MAX or top > logits.shape[-1]:
        raise ValueError(f"{top} alternatives are outside 1 .. {min(F.TOP_MAX, logits.shape[-1])}")
    if top_logprob.requires_grad and torch.is_grad_enabled():
        raise ValueError("the teacher's log probabilities have no gradient here: detach them")
    shape = lead + (top,)
    return (_per_row(top_id, shape, logits.device, torch.int64, "top_id"),
            _per_row(top_logprob, shape, logits.device, torch.float32, "top_logprob"))


def distill_loss(logits: torch.Tensor, top_id: torch.Tensor, top_logprob: torch.Tensor,
                 tail: bool = True, temperature: float = 1.0) -> torch.Tensor:
    """Per row: the divergence KL(teacher || student) of softmax(logits /
    temperature) from a teacher's top alternatives (token_logprobs' top_id and
    top_logprob at the same temperature).  tail=True treats the rest of the
    vocabulary as one more outcome; tail=False takes the alternatives as the
    whole.  Differentiable in the logits; multiply by temperature ** 2 for
    the customary weight."""
    temperature = _check_temperature(temperature)
    F.no_tangent(logits, "logits")
    lead = logits.shape[:-1]
    top_id, top_logprob = _teacher(logits, lead, top_id, top_logprob)
    if logits.requires_grad and torch.is_grad_enabled():
        return _Distill.apply(logits, lead, top_id, top_logprob, bool(tail), temperature)
    return _distill_forward(logits, lead, top_id, top_logprob, bool(tail), temperature)[0]


def distill_grad(logits: torch.Tensor, top_id: torch.Tensor, top_logprob: torch.Tensor,
                 grad_loss: torch.Tensor, tail: bool = True, temperature: float = 1.0,
                 inplace: bool = False):
    """(loss, gradient of sum(grad_loss * loss) with respect to the logits);
    grad_loss: FP32, one per row; inplace as in token_logprobs_grad."""
    temperature = _check_temperature(temperature)
    F.no_tangent(logits, "logits")
    lead, dev = logits.shape[:-1], logits.device
    top_id, top_logprob = _teacher(logits, lead, top_id, top_logprob)
    grad_loss = _per_row(grad_loss, lead, dev, torch.float32, "grad_loss")
    x, ty, rows, vocab, stride = F._logits(_rows(logits))
    loss = _empty(lead, dev)
    grad, grad_stride = _grad_buffer(logits, inplace)
    need = F.lib().flashopt_distill_workspace_bytes(ty, rows, vocab)
    ws = _workspace(need, dev)
    F._call("flashopt_distill_grad", dev, None, x, ty, rows, vocab, stride, temperature,
            top_id.data_ptr(), top_logprob.data_ptr(), top_id.shape[-1], bool(tail),
            grad_loss.data_ptr(), _at(ws), need, loss.data_ptr(), grad.data_ptr(), grad_stride)
    _replaced(logits, inplace)
    return loss, grad
