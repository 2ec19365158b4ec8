"""Weight gradients whose every partial sum is a binary32 number, so that the result is the exact one
rounded once to its type, bit for bit, whatever the order: a token left out or counted twice, a part of
an FP32 gradient lost, a piece joined to another tile all show.  At sizes of every way (grad_ways.py)."""
import pytest
import torch

import grad_ways as W
from compressed_adamw_state_amd import activations as A
from test_gpu_logits import TYPES, place

pytestmark = pytest.mark.gpu

CASES = [(dtype, way, *s) for dtype in TYPES for way, sizes in W.SIZES["32" if dtype == torch.float32 else "16"].items()
         for s in sizes]


def exact(dy, x):
    """In 64 bits (on the GPU), rounded once; both products of integers below 2^53"""
    d, v = dy.cuda().double(), x.cuda().double()
    return (d.t().contiguous() @ v).to(dy.dtype), d.sum(0).to(dy.dtype)


# whole numbers: |dy| <= 4 and |x| <= 7, so all sums stay below m * 28 < 2^24; 8 bits hold x as it is (7 is
# 112 times 2^-4)
@pytest.mark.parametrize("dtype,way,m,n,k", CASES)
def test_whole_numbers(dtype, way, m, n, k):
    assert W.way_of("32" if dtype == torch.float32 else "16", m, n, k)[0] == way and m * 28 < 1 << 24
    g = torch.Generator().manual_seed(m + n + k)
    x = torch.randint(-7, 8, (m, k), generator=g).to(dtype)
    dy = torch.randint(-4, 5, (m, n), generator=g).to(dtype)
    s = A.save8(x.cuda())
    assert torch.equal(s.load().cpu(), x)
    want, sums = exact(dy, x)
    for how in ("dense", "strided"):
        w, b = A.weight_grad(place(dy, how), s, bias=True)
        assert torch.equal(w, want) and torch.equal(b, sums)
        assert torch.equal(A.weight_grad(place(dy, how), s)[0], want)


# each column of dy has one token, all 24 bits of a number, and x powers of two: a product is a binary32
# number, and so is every sum of its parts'
@pytest.mark.parametrize("way,m,n,k", [c[1:] for c in CASES if c[0] == torch.float32])
def test_all_bits_of_fp32_gradients(way, m, n, k):
    assert W.way_of("32", m, n, k)[0] == way
    g = torch.Generator().manual_seed(m * n + k)
    x = torch.exp2(torch.randint(-3, 4, (m, k), generator=g).float()) * (2 * torch.randint(0, 2, (m, k), generator=g) - 1)
    at = (torch.arange(n) * 37 + m - 1) % m                        # the last token first
    dy = torch.zeros(m, n)
    number = (1 << 23) + 2 * torch.randint(0, 1 << 22, (n,), generator=g) + 1
    dy[at, torch.arange(n)] = number.float() * torch.exp2(torch.randint(-60, 60, (n,), generator=g).float())
    s = A.save8(x.cuda())
    assert torch.equal(s.load().cpu(), x)
    w, b = A.weight_grad(dy.cuda(), s, bias=True)
    assert torch.equal(w.cpu(), dy[at, torch.arange(n)][:, None] * x[at]) and torch.equal(b.cpu(), dy.sum(0))
