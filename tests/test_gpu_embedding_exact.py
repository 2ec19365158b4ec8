"""Gradients of an embedding table whose every partial sum is a binary32 number: the exact sums rounded
once to the type, bit for bit, so that no row of a token may be left out or counted twice."""
import pytest
import torch

from compressed_adamw_state_amd import embedding as E
from test_gpu_logits import TYPES

pytestmark = pytest.mark.gpu


def exact(ids, dy, vocab, scale):
    ok = (ids >= 0) & (ids < vocab)
    grad = torch.zeros(vocab, dy.shape[1], dtype=torch.float64)
    grad.index_add_(0, ids[ok], dy[ok].double())
    return (grad * scale).to(dy.dtype)


# |dy| <= 8: sums below 200000 * 8 < 2^24, the scale a power of two
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [33, 1000, 4097, 20000, 200000])
def test_one_token_throughout(dtype, n):
    g = torch.Generator().manual_seed(n)
    dim = 70 if n < 100000 else 24
    dy = torch.randint(-8, 9, (n, dim), generator=g).to(dtype)
    ids = torch.full((n,), 5)
    for k in (None, n // 3):
        if k is not None:                                          # between two others, in any order
            ids[:k // 2], ids[n - k // 2:] = 4, 9
            ids = ids[torch.randperm(n, generator=g)]
        assert torch.equal(E.embedding_grad(ids.cuda(), dy.cuda(), 11, 0.5).cpu(), exact(ids, dy, 11, 0.5))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,vocab,dim", [(9000, 5000, 16), (20000, 70000, 33), (200000, 3001, 24), (65536, 300001, 8)])
def test_many_tokens(dtype, n, vocab, dim):
    g = torch.Generator().manual_seed(vocab)
    ids = (torch.rand(n, generator=g) ** 4 * vocab).long()         # a few tokens often, most of them never
    ids[torch.rand(n, generator=g) < 0.1] = -100
    dy = torch.randint(-8, 9, (n, dim), generator=g).to(dtype)
    assert torch.equal(E.embedding_grad(ids.cuda(), dy.cuda(), vocab).cpu(), exact(ids, dy, vocab, 1.0))
