"""Arrays side by side in one buffer, and held arrays between a wide matrix's rows: no byte in common, so
the calls that refuse overlaps take them, with the results of buffers apart."""
import pytest
import torch

from compressed_adamw_state_amd import activations as A
from compressed_adamw_state_amd import embedding as E
from compressed_adamw_state_amd import flashopt as F
from compressed_adamw_state_amd.int8 import Int8Weight

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


class Buffer:
    """Pieces of one allocation, each right behind the last (rounded up to `step` bytes)."""

    def __init__(self, size=1 << 20):
        self.bytes, self.at = torch.zeros(size, dtype=torch.uint8, device="cuda"), 0

    def take(self, dtype, *shape, step=1):
        self.at = -(-self.at // step) * step
        n = torch.Size(shape).numel() * dtype.itemsize
        t = self.bytes[self.at:self.at + n].view(dtype).view(shape)
        self.at += n
        return t


@pytest.mark.parametrize("dtype", TYPES)
def test_side_by_side(dtype):
    m, n, k = 8, 24, 128                                           # (all sizes multiples of 16 bytes)
    g = torch.Generator().manual_seed(1)
    b = Buffer()
    x, up, codes, powers, uc, up8 = (b.take(t, *s) for t, s in (
        (dtype, (m, k)), (dtype, (m, k)), (torch.int8, (m, k)), (torch.uint8, (m, k // 32)), (torch.int8, (m, k)),
        (torch.uint8, (m, k // 32))))
    y, dg, du, dy, w, bias, back = (b.take(dtype, *s) for s in ((m, k), (m, k), (m, k), (m, n), (n, k), (n,), (m, k)))
    for t in (x, up, dy):
        t.copy_(torch.randn(t.shape, generator=g))
    s = A.save8(x)
    F.flashopt_hold(x, codes, powers)
    assert torch.equal(codes, s.codes) and torch.equal(powers, s.powers)
    F.flashopt_held_values(codes, powers, back)
    assert torch.equal(back, s.load())
    F.flashopt_held_weight_grad(dy, codes, powers, w, bias)
    want = A.weight_grad(dy, s, bias=True)
    assert torch.equal(w, want[0]) and torch.equal(bias, want[1])
    F.flashopt_gated(x, up, "silu", y, codes, powers, uc, up8)
    z, held = A.gated_save8(x, up)
    assert torch.equal(y, z)
    F.flashopt_gated_backward(y, "silu", codes, powers, dg, uc, up8, du)
    a, c = A.gated_grad(z, held)
    assert torch.equal(dg, a) and torch.equal(du, c)


@pytest.mark.parametrize("dtype", TYPES)
def test_between_the_rows_of_a_wide_matrix(dtype):
    m, k = 3, 96
    wide = torch.zeros(m, 4096, dtype=dtype, device="cuda")
    x = wide[:, :k]
    x.copy_(torch.randn(m, k, generator=torch.Generator().manual_seed(2)))
    s = A.save8(x.contiguous())
    row = wide[1].view(torch.uint8)
    codes, powers = row[1024:1024 + m * 128].view(torch.int8).view(m, 128), row[2048:2048 + m * 4].view(m, 4)
    F.flashopt_hold(x, codes, powers)
    assert torch.equal(codes, s.codes) and torch.equal(powers, s.powers)
    out = wide[:, 2048:2048 + k]
    F.flashopt_held_values(codes, powers, out)
    assert torch.equal(out, s.load())


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_of_a_table_beside_it(dtype):
    q = Int8Weight.from_weight(torch.randn(10, 40, generator=torch.Generator().manual_seed(3)).cuda())
    ids = torch.tensor([3, 9, 0, -100, 3, 7], device="cuda")
    b = Buffer()
    near_ids, w, scale, out = (b.take(t, *s, step=16) for t, s in (
        (torch.int64, (6,)), (torch.int8, tuple(q.codes.shape)), (torch.float32, (10,)), (dtype, (6, 40))))
    for t, v in ((near_ids, ids), (w, q.codes), (scale, q.scale)):
        t.copy_(v)
    F.flashopt_embedding_int8(near_ids, w, scale, out)
    assert torch.equal(out, E.embedding(ids, q, dtype=dtype))
    grad = b.take(dtype, 10, 40)
    F.flashopt_embedding_backward(near_ids, out, grad)
    assert torch.equal(grad, E.embedding_grad(ids, out, 10))
