"""What a layer's small gradients come to (include/flashopt_lm.h): FP32 ones below 2^-110, whose three BF16
parts end at that type's smallest step, and subnormal 16-bit ones, which keep all bits."""
import pytest
import torch

import grad_ways as W
from compressed_adamw_state_amd import activations as A

pytestmark = pytest.mark.gpu

SIZES = [s for sizes in W.SIZES["32"].values() for s in sizes[:1]]


# One token a column of dy and powers of two in x: products and their parts' sums are binary32 numbers.
@pytest.mark.parametrize("m,n,k", SIZES)
def test_small_fp32_gradients(m, n, k):
    g = torch.Generator().manual_seed(n)
    x = torch.exp2(torch.randint(-3, 4, (m, k), generator=g).float()) * (2 * torch.randint(0, 2, (m, k), generator=g) - 1)
    at = (torch.arange(n) * 37 + m - 1) % m
    number = (1 + torch.rand(n, generator=g, dtype=torch.float64)) * torch.exp2(-100 - 48 * torch.rand(n, generator=g, dtype=torch.float64).round(decimals=2))
    number = (number * (2 * torch.randint(0, 2, (n,), generator=g) - 1)).float()
    dy = torch.zeros(m, n)
    dy[at, torch.arange(n)] = number
    step = 2.0 ** -133
    kept = ((number.double() / step).trunc() * step).float()        # towards zero
    assert bool((kept == number)[number.abs() >= 2.0 ** -110].all()) and bool((kept != number).any())
    w, b = A.weight_grad(dy.cuda(), A.save8(x.cuda()), bias=True)
    assert torch.equal(w.cpu(), kept[:, None] * x[at]) and torch.equal(b.cpu(), kept)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_small_16_bit_gradients_are_exact(dtype):
    n = 64
    least = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}[dtype]
    number = (torch.arange(1, n + 1) * least).to(dtype)             # subnormal, all bits
    dy = torch.diag(number)
    w, b = A.weight_grad(dy.cuda(), A.save8(torch.eye(n, dtype=dtype).cuda()), bias=True)
    assert torch.equal(w.cpu(), dy.t()) and torch.equal(b.cpu(), number)
