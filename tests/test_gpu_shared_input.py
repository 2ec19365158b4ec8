"""Layers that share an input: one call with their weights stacked keeps it once, with the gradients of
separate calls (whole numbers, so that every sum is exact), which keep it once each."""
import pytest
import torch

from compressed_adamw_state_amd import activations as A

pytestmark = pytest.mark.gpu


def kept(call, weights):
    own = {w.data_ptr() for w in weights}
    seen = {}
    with torch.autograd.graph.saved_tensors_hooks(lambda t: seen.setdefault(t.data_ptr(), t), lambda t: t):
        y = call()
    return y, sum(t.numel() * t.element_size() for p, t in seen.items() if p not in own)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_stacked_weights_keep_one_copy(dtype):
    g = torch.Generator().manual_seed(1)
    m, k, n = 200, 256, 96
    x = torch.randint(-7, 8, (m, k), generator=g).to(dtype).cuda()
    stacked = torch.randint(-2, 3, (3 * n, k), generator=g).to(dtype).cuda().requires_grad_()
    parts = [w.clone().requires_grad_() for w in stacked.detach().split(n)]
    up = torch.randint(-4, 5, (m, 3 * n), generator=g).to(dtype).cuda()
    y, one = kept(lambda: A.linear(x, stacked), [stacked])
    z, three = kept(lambda: [A.linear(x, w) for w in parts], parts)
    assert one == m * k * 33 // 32 and three == 3 * one
    whole, = torch.autograd.grad(y, stacked, up)
    separate = torch.autograd.grad(z, parts, list(up.split(n, 1)))
    assert torch.equal(whole, torch.cat(separate))
