"""What a layer keeps between its forward and its backward pass, held in 8 bits:
codes with a power of two for each 32 values of a row (include/flashopt_lm.h),
8.25 bits a value, each off by at most 1/127 of its group's largest magnitude
(by 2^-127 where that is below 2^-120).

* linear: a linear layer that keeps its input in 8 bits; its weight's gradient
  comes from the codes, which enter the matrix instructions exactly.  Every call
  holds its input by itself: layers of one input (queries, keys and values; gate
  and up) that are separate calls keep a copy each, so take them as one call
  with their weights stacked, which keeps one;
* gated, activation: an activation function (times a second input), whose
  inputs are held in 8 bits; the output is that of the full inputs;
* save8 and weight_grad, gated_save8 and gated_grad: the same by hand, for a
  program without autograd (inside a HIP graph).

The products with the weight itself (forward, and the input's gradient) are
torch's; everything else runs in the HIP library, and this module only
marshals.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import flashopt as F


class Saved8:
    """A tensor [..., k] held in 8 bits, with the shape and type it had: one uint8 buffer of the
    codes' rows and, behind them, the powers'."""

    def __init__(self, held: torch.Tensor, shape: torch.Size, dtype: torch.dtype):
        self.held, self.shape, self.dtype = held, torch.Size(shape), dtype

    @property
    def device(self) -> torch.device:
        return self.held.device

    @property
    def codes(self) -> torch.Tensor:
        """[rows, flashopt_held_ld(k)] int8"""
        ld = F.lib().flashopt_held_ld(self.shape[-1])
        rows = self.shape[:-1].numel()
        return self.held[:rows * ld].view(torch.int8).view(rows, ld)

    @property
    def powers(self) -> torch.Tensor:
        """[rows, flashopt_held_ld(k) / 32] uint8"""
        ld = F.lib().flashopt_held_ld(self.shape[-1])
        rows = self.shape[:-1].numel()
        return self.held[rows * ld:].view(rows, ld // F.GROUP)

    def load(self, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
        """The values held, in their own type or in FP32."""
        if dtype not in (None, self.dtype, torch.float32):
            raise ValueError(f"held from {self.dtype}: the values are of that type or FP32")
        out = torch.empty(self.shape, dtype=dtype or self.dtype, device=self.device)
        if out.numel():
            F.flashopt_held_values(self.codes, self.powers, out.view(-1, self.shape[-1]))
        return out


def _new_held(rows: int, cols: int, device, count: int = 1) -> torch.Tensor:
    """A buffer of `count` held matrices: the codes of all, then their powers."""
    ld = F.lib().flashopt_held_ld(cols)
    if ld == 0:
        raise ValueError(f"{cols} values a row are outside 1 .. 131072")
    return torch.empty(count * rows * (ld + ld // F.GROUP), dtype=torch.uint8, device=device)


def _addresses(held: Optional[torch.Tensor], count: int = 1) -> list:
    """The addresses of the codes and powers of two held matrices (None for those there are not)."""
    if held is None:
        return [None] * 4
    at, powers = held.data_ptr(), held.numel() // (F.GROUP + 1)
    behind = at + powers * F.GROUP
    if count == 1:
        return [at, behind, None, None]
    return [at, behind, at + powers // 2 * F.GROUP, behind + powers // 2]


def _dense(t: torch.Tensor, cols: int) -> torch.Tensor:
    """t as a matrix with dense rows, copied only where it must be."""
    if t.dim() == 0 or t.shape[-1] != cols:
        raise ValueError(f"expected {cols} values a row")
    if not t.is_cuda:
        raise ValueError("expected device tensors")
    if t.numel() == 0:                           # whatever its strides
        return torch.empty((t.shape[:-1].numel(), cols), dtype=t.dtype, device=t.device)
    if t.dim() != 2:
        try:
            t = t.view(t.shape[:-1].numel(), cols)
        except RuntimeError:
            return t.reshape(-1, cols)
    if (cols > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < cols):
        t = t.contiguous()
    return t


def save8(x: torch.Tensor) -> Saved8:
    """Hold x [..., k] (BF16, FP16 or FP32) in 8 bits.  An infinity or NaN makes its group of
    32 values NaN."""
    F.no_tangent(x, "x")
    F.element_type(x)
    if x.dim() == 0:
        raise ValueError("expected rows of values")
    rows = _dense(x.detach(), x.shape[-1])
    (m, k), dev = rows.shape, x.device
    held = _new_held(m, k, dev)
    F._call("flashopt_hold", dev, None, rows.data_ptr(), F.element_type(x), m, k, F.row_stride(rows),
            *_addresses(held)[:2])
    return Saved8(held, x.shape, x.dtype)


def weight_grad(grad_out: torch.Tensor, saved: Saved8, bias: bool = False):
    """(weight's gradient [n, k], bias's gradient [n] or None) of a linear layer from its
    output's gradient [..., n] and its held input [..., k], both of one type; sums in FP32."""
    F.no_tangent(grad_out, "grad_out")
    if grad_out.dtype != saved.dtype or grad_out.device != saved.device or \
            grad_out.shape[:-1] != saved.shape[:-1]:
        raise ValueError("grad_out must have the held input's type, device and leading dimensions")
    dy = _dense(grad_out.detach(), grad_out.shape[-1])
    (m, n), k, dev, ty = dy.shape, saved.shape[-1], dy.device, F.element_type(dy)
    weight = torch.empty((n, k), dtype=dy.dtype, device=dev)
    b = torch.empty(n, dtype=dy.dtype, device=dev) if bias else None
    need = F.lib().flashopt_held_weight_grad_workspace_bytes(ty, m, n, k)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    F._call("flashopt_held_weight_grad", dev, None, dy.data_ptr(), ty, m, n, F.row_stride(dy),
            *_addresses(saved.held)[:2], k, weight.data_ptr(), k,
            None if b is None else b.data_ptr(), None if ws is None else ws.data_ptr(), need)
    return weight, b


def _product(rows: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor], lead) -> torch.Tensor:
    """torch's product of matrices (of strided leading dimensions it would make a batched one), its
    result a tensor of its own and no view, so that a caller may add to it in place."""
    y = torch.empty(lead + weight.shape[:1], dtype=rows.dtype, device=rows.device)
    out = y.view(rows.shape[0], weight.shape[0])
    if bias is None:
        torch.mm(rows, weight.t(), out=out)
    else:
        torch.addmm(bias, rows, weight.t(), out=out)
    return y


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        rows = _dense(x, x.shape[-1])
        saved = save8(rows) if weight.requires_grad else None
        ctx.save_for_backward(weight, None if saved is None else saved.held)
        ctx.lead, ctx.held = x.shape[:-1], (rows.shape, x.dtype)
        return _product(rows, weight, bias, ctx.lead)

    @staticmethod
    @F.first_order
    def backward(ctx, g):
        weight, held = ctx.saved_tensors
        want_x, want_w, want_b = ctx.needs_input_grad
        g = _dense(g, weight.shape[0])
        dx = dw = db = None
        if want_x:
            dx = g.mm(weight).view(ctx.lead + weight.shape[1:])
        if want_w:
            dw, db = weight_grad(g, Saved8(held, *ctx.held), bias=want_b)
        elif want_b:
            db = g.sum(0)
        return dx, dw, db


def linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """torch.nn.functional.linear, its input kept in 8 bits for the weight's gradient, a copy for
    each call whose weight needs one.  All of one type (BF16, FP16 or FP32)."""
    for t, name in ((x, "x"), (weight, "weight"), (bias, "bias")):
        if t is None:
            continue
        F.no_tangent(t, name)
        if t.dtype != x.dtype or t.device != x.device or not t.is_cuda:
            raise ValueError("x, weight and bias must be of one type on one GPU")
    F.element_type(x)
    if torch.is_autocast_enabled("cuda"):
        raise ValueError("linear works in its inputs' type: call it outside autocast")
    if weight.dim() != 2 or x.dim() == 0 or x.shape[-1] != weight.shape[1] or \
            (bias is not None and bias.shape != weight.shape[:1]):
        raise ValueError("weight must be n x k for x's k features, bias of n")
    if torch.is_grad_enabled():
        return _Linear.apply(x, weight, bias)
    return _product(_dense(x, x.shape[-1]), weight, bias, x.shape[:-1])


def _check_kind(kind: str) -> int:
    if kind not in F.ACTIVATION:
        raise ValueError(f"kind = {kind!r} is none of {sorted(F.ACTIVATION)}")
    return F.ACTIVATION[kind]


def _forward(gate, up, kind, hold, lead):
    (rows, cols), dev, count = gate.shape, gate.device, 1 if up is None else 2
    y = torch.empty(lead + (cols,), dtype=gate.dtype, device=dev)        # no view, as _product's
    held = _new_held(rows, cols, dev, count) if hold else None
    F._call("flashopt_gated", dev, None, gate.data_ptr(), None if up is None else up.data_ptr(),
            F.element_type(gate), kind, rows, cols, F.row_stride(gate),
            0 if up is None else F.row_stride(up), y.data_ptr(), cols, *_addresses(held, count))
    return y, held


def _backward(held, kind, halves, two, shape, g):
    """(gate's gradient, up's): one tensor of both where they lie side by side"""
    cols = shape[-1] // 2 if halves else shape[-1]
    dy = _dense(g, cols)
    dev, size, stride = dy.device, dy.element_size(), shape[-1]
    grad = torch.empty(shape, dtype=dy.dtype, device=dev)
    dup = torch.empty_like(grad) if two and not halves else None
    at = grad.data_ptr()
    second = at + cols * size if halves else None if dup is None else dup.data_ptr()
    F._call("flashopt_gated_backward", dev, None, dy.data_ptr(), F.element_type(dy), kind, dy.shape[0], cols,
            F.row_stride(dy), *_addresses(held, 2 if two else 1), at, stride, second, stride if two else 0)
    return grad, dup


class _Gated(torch.autograd.Function):
    """x: gate, or gate and up side by side where up is None and `halves`."""

    @staticmethod
    def forward(ctx, x, up, kind, halves):
        gate, second = _split(x, up, halves)
        y, held = _forward(gate, second, kind, True, x.shape[:-1])
        ctx.save_for_backward(held)
        ctx.what = kind, halves, second is not None, x.shape
        return y

    @staticmethod
    @F.first_order
    def backward(ctx, g):
        return *_backward(*ctx.saved_tensors, *ctx.what, g), None, None


class SavedGated:
    """What gated_save8 keeps: the inputs in 8 bits, with their function, shape and type."""

    def __init__(self, held: torch.Tensor, kind: int, halves: bool, two: bool, shape: torch.Size,
                 dtype: torch.dtype):
        self.held, self.kind, self.halves, self.two, self.shape, self.dtype = held, kind, halves, two, shape, dtype


def _split(x, up, halves):
    rows = _dense(x, x.shape[-1])
    if halves:
        cols = x.shape[-1] // 2
        return rows[:, :cols], rows[:, cols:]
    return rows, None if up is None else _dense(up, x.shape[-1])


def _check(x, up, kind, halves) -> int:
    kind = _check_kind(kind)
    for t, name in ((x, "x"), (up, "up")):
        if t is not None:
            F.no_tangent(t, name)
            F.element_type(t)
    if up is not None and (up.shape != x.shape or up.dtype != x.dtype or up.device != x.device):
        raise ValueError("up must have the gate's shape, type and device")
    if x.dim() == 0 or x.shape[-1] == 0 or (halves and x.shape[-1] % 2):
        raise ValueError("expected rows of values, an even number where they hold gate and up")
    if not x.is_cuda:
        raise ValueError("expected device tensors")
    return kind


def _apply(x, up, kind, halves):
    kind = _check(x, up, kind, halves)
    if torch.is_grad_enabled() and (x.requires_grad or (up is not None and up.requires_grad)):
        return _Gated.apply(x, up, kind, halves)
    gate, second = _split(x, up, halves)
    return _forward(gate, second, kind, False, x.shape[:-1])[0]


def gated(gate: torch.Tensor, up: Optional[torch.Tensor] = None, kind: str = "silu") -> torch.Tensor:
    """f(gate) * up; without up, gate holds both side by side ([..., 2 h] gives [..., h]).  kind:
    "silu" or "gelu" (its form by tanh).  The gradients use gate and up as held in 8 bits: a group
    of 32 values with an infinity or NaN has gradients NaN."""
    return _apply(gate, up, kind, up is None)


def activation(x: torch.Tensor, kind: str = "gelu") -> torch.Tensor:
    """f(x), its gradient from x as held in 8 bits; kinds as gated's."""
    return _apply(x, None, kind, False)


def gated_save8(gate: torch.Tensor, up: Optional[torch.Tensor] = None, kind: str = "silu",
                halves: bool = False):
    """(y, what gated_grad needs): f(gate) * up, f(gate) without up, or, with halves, gate and up
    side by side in one tensor."""
    if halves and up is not None:
        raise ValueError("halves: gate holds up too")
    code = _check(gate, up, kind, halves)
    first, second = _split(gate.detach(), None if up is None else up.detach(), halves)
    y, held = _forward(first, second, code, True, gate.shape[:-1])
    return y, SavedGated(held, code, halves, second is not None, gate.shape, gate.dtype)


def gated_grad(grad_out: torch.Tensor, saved: SavedGated):
    """The gradients with respect to gate and up (None where there is none, or where one tensor
    holds both) of sum(grad_out * y)."""
    F.no_tangent(grad_out, "grad_out")
    cols = saved.shape[-1] // 2 if saved.halves else saved.shape[-1]
    if grad_out.dtype != saved.dtype or grad_out.device != saved.held.device or \
            grad_out.shape != saved.shape[:-1] + (cols,):
        raise ValueError("grad_out must have the output's shape, type and device")
    return _backward(saved.held, saved.kind, saved.halves, saved.two, saved.shape, grad_out.detach())
