"""Weights in 8 bits for a model that is only read (a teacher, an evaluated or
served model): rows of 8-bit codes with one FP32 scale per output channel, and
the linear layer over them, its input rounded to 8 bits with one scale per
token (include/flashopt_lm.h).

An Int8Weight comes from a weight matrix (from_weight), from the optimizer's
compressed state without an FP32 copy (from_state; FlashAdamW.export_int8),
or from codes made elsewhere (from_codes).  Int8Linear is the module form.

The layer has no gradient: an input that requires one is refused.  This
module only marshals: every product runs in the HIP library.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import flashopt as F


class Int8Weight:
    """n x k codes in rows of ld bytes (k rounded up to 128, zeros behind k)
    and n scales."""

    def __init__(self, codes: torch.Tensor, scale: torch.Tensor, k: int):
        ld = F.lib().flashopt_int8_ld(k)
        if ld == 0:
            raise ValueError(f"k = {k} is outside 1 .. 131072")
        if codes.dtype != torch.int8 or codes.dim() != 2 or codes.shape[1] != ld or \
                not codes.is_contiguous():
            raise ValueError(f"codes must be a contiguous int8 tensor of rows of {ld}")
        if scale.dtype != torch.float32 or scale.shape != codes.shape[:1] or \
                scale.device != codes.device or not scale.is_contiguous():
            raise ValueError("scale must be FP32, one per row of codes, on their device")
        self.codes, self.scale, self.n, self.k = codes, scale, codes.shape[0], k

    @classmethod
    def _empty(cls, n: int, k: int, device) -> "Int8Weight":
        ld = F.lib().flashopt_int8_ld(k)
        return cls(torch.empty((n, ld), dtype=torch.int8, device=device),
                   torch.empty(n, dtype=torch.float32, device=device), k)

    @classmethod
    def from_weight(cls, w: torch.Tensor) -> "Int8Weight":
        """Round the rows of a BF16, FP16 or FP32 matrix (n x k)."""
        w = w.detach()
        out = cls._empty(w.shape[0], w.shape[1], w.device)
        F.flashopt_quantize_rows(w, out.codes, out.scale)
        return out

    @classmethod
    def from_state(cls, st: F.TensorState, k: int) -> "Int8Weight":
        """Round the master weight of a tensor's optimizer state, as rows of k."""
        if k < 1 or st.numel % k:
            raise ValueError(f"{st.numel} elements are not rows of {k}")
        out = cls._empty(st.numel // k, k, st.theta.device)
        F.flashopt_tensor_quantize_rows(st, k, out.codes, out.scale)
        return out

    @classmethod
    def from_codes(cls, codes: torch.Tensor, scale: torch.Tensor) -> "Int8Weight":
        """Lay out n x k codes (values in [-127, 127])."""
        n, k = codes.shape
        ld = F.lib().flashopt_int8_ld(k)
        if ld == 0 or codes.dtype != torch.int8:
            raise ValueError("codes must be int8 with 1 .. 131072 columns")
        rows = torch.zeros((n, ld), dtype=torch.int8, device=codes.device)
        rows[:, :k] = codes
        return cls(rows, scale.to(torch.float32).contiguous(), k)

    def dequantize(self) -> torch.Tensor:
        """The n x k values in FP32."""
        return self.codes[:, :self.k].float() * self.scale[:, None]


def int8_linear(x: torch.Tensor, weight: Int8Weight, bias: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[..., n] = x[..., k] W^T + bias in x's type: x rounded to 8 bits per
    token, an exact integer product, the scales and the bias in FP32, one
    rounding."""
    k, n, dev = weight.k, weight.n, weight.codes.device
    if x.shape[-1] != k:
        raise ValueError(f"x has {x.shape[-1]} features, the weight {k}")
    if (x.requires_grad or (bias is not None and bias.requires_grad)) and torch.is_grad_enabled():
        raise ValueError("int8_linear has no gradient: call it under torch.no_grad()")
    F.no_tangent(x, "x")
    if bias is not None:
        F.no_tangent(bias, "bias")
    if x.device != dev or not x.is_cuda:
        raise ValueError("x and the weight must be on one GPU")
    shape, given = x.shape[:-1] + (n,), out is not None
    if not given:
        out = torch.empty(shape, dtype=x.dtype, device=dev)
    elif out.shape != shape or out.dtype != x.dtype or out.device != dev:
        raise ValueError("out must have x's leading dimensions, type and device, and n features")
    elif out.requires_grad and torch.is_grad_enabled():
        raise ValueError("out requires a gradient, which int8_linear does not have")
    if bias is not None and (bias.dtype != x.dtype or bias.shape != (n,) or bias.device != dev
                             or not bias.is_contiguous()):
        raise ValueError("bias must hold n values of x's type on its device")
    rows, to = _matrix(x, k, "x"), _matrix(out, n, "out")
    m = rows.shape[0]
    need = F.lib().flashopt_int8_workspace_bytes(m, n, k)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    # the weight's arrays were checked when it was made
    F._call("flashopt_int8_linear", dev, None, rows.data_ptr(), F.element_type(x), m, k,
            F.row_stride(rows), weight.codes.data_ptr(), weight.scale.data_ptr(),
            None if bias is None else bias.data_ptr(), n, to.data_ptr(), F.row_stride(to),
            None if ws is None else ws.data_ptr(), need)
    if given:
        # torch then refuses a backward pass that would read out's former values
        torch.autograd.graph.increment_version(out)
    return out


def _matrix(t: torch.Tensor, cols: int, name: str) -> torch.Tensor:
    if t.dim() == 2:
        return t
    try:
        return t.view(t.shape[:-1].numel(), cols)
    except RuntimeError:
        raise ValueError(f"{name}'s leading dimensions must flatten without a copy") from None


class Int8Linear(torch.nn.Module):
    """A torch.nn.Linear whose weight is held in 8 bits (frozen)."""

    def __init__(self, weight: Int8Weight, bias: Optional[torch.Tensor] = None):
        super().__init__()
        self.in_features, self.out_features = weight.k, weight.n
        self.register_buffer("codes", weight.codes)
        self.register_buffer("scale", weight.scale)
        self.register_buffer("bias", None if bias is None else bias.detach())

    @classmethod
    def from_linear(cls, linear: torch.nn.Linear) -> "Int8Linear":
        return cls(Int8Weight.from_weight(linear.weight), linear.bias)

    def _apply(self, fn, recurse: bool = True):
        # a model's .to(dtype), .half() and .bfloat16() change the bias alone:
        # the scales stay the FP32 numbers they are
        scale = self.scale
        super()._apply(fn, recurse)
        if self.scale.dtype != torch.float32:
            self.scale = scale.to(self.scale.device)
        return self

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return int8_linear(x, Int8Weight(self.codes, self.scale, self.in_features), self.bias)
