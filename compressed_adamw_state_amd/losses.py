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


def _per_row(t: torch.Tensor, logits: torch.Tensor, dtype, name: str, last=()) -> torch.Tensor:
    if t.dtype != dtype or t.shape != logits.shape[:-1] + tuple(last):
        raise ValueError(f"{name} must be {dtype} of shape {tuple(logits.shape[:-1]) + tuple(last)}")
    return t if t.is_contiguous() else t.contiguous()


def _check_temperature(temperature: float) -> float:
    temperature = float(temperature)
    if not 2.0 ** -126 <= temperature <= 2.0 ** 126:
        raise ValueError(f"temperature = {temperature} is outside its range")
    return temperature


def _upstream(g: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    return None if g is None else g.to(torch.float32).contiguous()


def _forward(logits, targets, top, temperature, keep):
    x = _rows(logits)
    lead, dev = logits.shape[:-1], logits.device
    logprob = None if targets is None else torch.empty(lead, dtype=torch.float32, device=dev)
    entropy = torch.empty(lead, dtype=torch.float32, device=dev)
    stats = torch.empty((x.shape[0], 4), dtype=torch.float32, device=dev) if keep else None
    tl = ti = None
    if top:
        tl = torch.empty(lead + (top,), dtype=torch.float32, device=dev)
        ti = torch.empty(lead + (top,), dtype=torch.int64, device=dev)
    F.flashopt_logprob(x, targets, top, temperature, logprob, entropy, stats, tl, ti)
    return logprob, entropy, stats, tl, ti


class _Logprob(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, top, temperature):
        logprob, entropy, stats, tl, ti = _forward(logits, targets, top, temperature, True)
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
            return None, None, None, None
        grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        F.flashopt_logprob_backward(_rows(logits), targets, stats, _upstream(g_logprob),
                                    _upstream(g_entropy), _rows(grad), ctx.temperature)
        return grad, None, None, None


def token_logprobs(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, top: int = 0,
                   temperature: float = 1.0) -> TokenLogprobs:
    """Per row: the log probability of targets (int64; an id outside the
    vocabulary, such as -100, gives 0 without a gradient), the entropy, and
    the `top` most likely tokens (0 to 64; equal logits by lowest id), of
    softmax(logits / temperature).  logprob and entropy are differentiable."""
    temperature = _check_temperature(temperature)
    if not 0 <= top <= min(F.TOP_MAX, logits.shape[-1]):
        raise ValueError(f"top = {top} is outside 0 .. {min(F.TOP_MAX, logits.shape[-1])}")
    if targets is not None:
        targets = _per_row(targets, logits, torch.int64, "targets")
    if torch.is_grad_enabled() and logits.requires_grad:
        return TokenLogprobs(*_Logprob.apply(logits, targets, top, temperature))
    logprob, entropy, _, tl, ti = _forward(logits, targets, top, temperature, False)
    return TokenLogprobs(logprob, entropy, tl, ti)


def _grad_buffer(logits: torch.Tensor, inplace: bool) -> torch.Tensor:
    if inplace:
        return logits.detach()
    return torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)


@torch.no_grad()
def token_logprobs_grad(logits: torch.Tensor, targets: torch.Tensor, grad_logprob: torch.Tensor,
                        grad_entropy: Optional[torch.Tensor] = None, temperature: float = 1.0,
                        inplace: bool = False) -> TokenLogprobsGrad:
    """logprob, entropy and the gradient of sum(grad_logprob * logprob +
    grad_entropy * entropy) with respect to the logits (grad_*: FP32, one per
    row)."""
    temperature = _check_temperature(temperature)
    targets = _per_row(targets, logits, torch.int64, "targets")
    grad_logprob = _per_row(grad_logprob, logits, torch.float32, "grad_logprob")
    if grad_entropy is not None:
        grad_entropy = _per_row(grad_entropy, logits, torch.float32, "grad_entropy")
    x = _rows(logits)
    lead, dev = logits.shape[:-1], logits.device
    logprob = torch.empty(lead, dtype=torch.float32, device=dev)
    entropy = torch.empty(lead, dtype=torch.float32, device=dev)
    stats = torch.empty((x.shape[0], 4), dtype=torch.float32, device=dev)
    grad = _grad_buffer(logits, inplace)
    F.flashopt_logprob_grad(x, targets, grad_logprob, grad_entropy, stats, _rows(grad), logprob,
                            entropy, temperature)
    return TokenLogprobsGrad(logprob, entropy, grad)


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_id, top_logprob, tail, temperature):
        loss, stats = _distill_forward(logits, top_id, top_logprob, tail, temperature)
        ctx.save_for_backward(logits, top_id, top_logprob, stats)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        logits, top_id, top_logprob, stats = ctx.saved_tensors
        grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        top = top_id.shape[-1]
        F.flashopt_distill_backward(_rows(logits), top_id.view(-1, top), top_logprob.view(-1, top),
                                    stats, _upstream(g), _rows(grad), ctx.temperature)
        return grad, None, None, None, None


def _distill_forward(logits, top_id, top_logprob, tail, temperature):
    x, top = _rows(logits), top_id.shape[-1]
    loss = torch.empty(logits.shape[:-1], dtype=torch.float32, device=logits.device)
    stats = torch.empty((x.shape[0], 8), dtype=torch.float32, device=logits.device)
    F.flashopt_distill(x, top_id.view(-1, top), top_logprob.view(-1, top), loss, stats, tail,
                       temperature)
    return loss, stats


def _teacher(logits, top_id, top_logprob):
    top = top_id.shape[-1] if top_id.dim() else 0
    if not 1 <= top <= min(F.TOP_MAX, logits.shape[-1]):
        raise ValueError(f"{top} alternatives are outside 1 .. {min(F.TOP_MAX, logits.shape[-1])}")
    if top_logprob.requires_grad and torch.is_grad_enabled():
        raise ValueError("the teacher's log probabilities have no gradient here: detach them")
    return (_per_row(top_id, logits, torch.int64, "top_id", (top,)),
            _per_row(top_logprob, logits, torch.float32, "top_logprob", (top,)))


def distill_loss(logits: torch.Tensor, top_id: torch.Tensor, top_logprob: torch.Tensor,
                 tail: bool = True, temperature: float = 1.0) -> torch.Tensor:
    """Per row: the divergence KL(teacher || student) of softmax(logits /
    temperature) from a teacher's top alternatives (token_logprobs' top_id and
    top_logprob at the same temperature).  tail=True treats the rest of the
    vocabulary as one more outcome; tail=False takes the alternatives as the
    whole.  Differentiable in the logits; multiply by temperature ** 2 for
    the customary weight."""
    temperature = _check_temperature(temperature)
    top_id, top_logprob = _teacher(logits, top_id, top_logprob)
    if torch.is_grad_enabled() and logits.requires_grad:
        return _Distill.apply(logits, top_id, top_logprob, bool(tail), temperature)
    return _distill_forward(logits, top_id, top_logprob, bool(tail), temperature)[0]


@torch.no_grad()
def distill_grad(logits: torch.Tensor, top_id: torch.Tensor, top_logprob: torch.Tensor,
                 grad_loss: torch.Tensor, tail: bool = True, temperature: float = 1.0,
                 inplace: bool = False):
    """(loss, gradient of sum(grad_loss * loss) with respect to the logits);
    grad_loss: FP32, one per row."""
    temperature = _check_temperature(temperature)
    top_id, top_logprob = _teacher(logits, top_id, top_logprob)
    grad_loss = _per_row(grad_loss, logits, torch.float32, "grad_loss")
    x, top = _rows(logits), top_id.shape[-1]
    loss = torch.empty(logits.shape[:-1], dtype=torch.float32, device=logits.device)
    stats = torch.empty((x.shape[0], 8), dtype=torch.float32, device=logits.device)
    grad = _grad_buffer(logits, inplace)
    F.flashopt_distill_grad(x, top_id.view(-1, top), top_logprob.view(-1, top), grad_loss, loss,
                            stats, _rows(grad), bool(tail), temperature)
    return loss, grad
