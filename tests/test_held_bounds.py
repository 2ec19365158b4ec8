"""How far a value held in 8 bits may be off (include/flashopt_lm.h), by the plain codec that the library's
equals bit for bit: ordinary groups, and those at either end of the exponents."""
import pytest
import torch

import train_plain as T

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def errors(x):
    """(each value's error, its group's largest magnitude, its group's e) in 64 bits"""
    codes, powers = T.hold(x)
    v = T.held_values(codes, powers, x.shape[1])
    top = x.double().abs().view(x.shape[0], -1, 32).amax(2).repeat_interleave(32, 1)
    return (v - x.double()).abs(), top, (powers.double() - 127).repeat_interleave(32, 1)[:, :x.shape[1]]


@pytest.mark.parametrize("dtype", TYPES)
def test_bounds_of_held_values(dtype):
    g = torch.Generator().manual_seed(1)
    info = torch.finfo(dtype)
    least, most = T.BOUNDS[dtype]
    lo, hi = (-26, 15) if dtype == torch.float16 else (-134, 127)
    size = torch.randint(lo, hi + 1, (400, 1), generator=g)
    x = ((2 * torch.rand(400, 128, generator=g, dtype=torch.float64) - 1) * torch.exp2(size.double())).to(dtype)
    x[0], x[1], x[2] = info.max, -info.max, info.max * 0.996
    err, top, e = errors(x)
    step = torch.exp2(e)
    ends = (e == most) & (top > 127.5 * step) | (e == least)
    assert bool(ends.any()) and not bool(ends.all())
    assert bool((err <= step / 2)[~ends].all()) and bool((err <= top / 127)[top >= 2.0 ** -120].all())
    high = (e == most) & (top > 127.5 * step)
    # (BF16's largest number is 127.5 steps: off by half a step as ever)
    assert bool((err < step)[high].all()) and bool((err > step / 2)[high].any()) == (dtype != torch.bfloat16)
    low = e == least
    # FP16 is exact there, its own step being 2^-24
    assert bool((err <= (0.0 if dtype == torch.float16 else 2.0 ** -127))[low].all())
    if dtype == torch.float32:
        one = torch.full((1, 32), 2.0 ** -128)                     # held as 0: all of its largest value
        assert errors(one)[0].max().item() == 2.0 ** -128
