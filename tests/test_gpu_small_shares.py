"""Activations whose share f / g is below binary32's normal numbers (include/flashopt_lm.h)."""
import math

import pytest
import torch

from compressed_adamw_state_amd import activations as A
from test_gpu_logits import TYPES

pytestmark = pytest.mark.gpu


# f = g s: off by s's own error, at most 2^-126 where s is below it (the hardware's reciprocal gives no
# subnormals), and half a step of the type
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_small_shares(dtype, kind):
    v = torch.linspace(-104, -60, 3000) if kind == "silu" else torch.linspace(-10.6, -8, 3000)
    x = v.to(dtype)
    y = A.activation(x[:, None].repeat(1, 32).cuda(), kind)[:, 0].cpu().double()
    g = x.double()
    z = g if kind == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    f = g / (1 + torch.exp(-z))
    # s is off by (6 |z| + 12) u of itself, as in train_plain.shape
    rel = 2.0 ** -24 * (6 * z.abs() + 14) + torch.finfo(dtype).eps / 2 * (1 + 1e-3)
    tol = f.abs() * rel + g.abs() * 2.0 ** -126 + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    assert bool(((y - f).abs() <= tol).all())
