"""Operators of a training step on arrays of more than 2^32 bytes and 2^31 elements: each element's address
in 64 bits.  The large calls repeat a small one, or are sums of whole numbers (exact in any order)."""
import pytest
import torch

from compressed_adamw_state_amd import activations as A
from compressed_adamw_state_amd import embedding as E
from compressed_adamw_state_amd import losses as L

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def memory():
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GB of device memory")
    yield
    torch.cuda.empty_cache()


def whole(rows, cols, most, seed, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-most, most + 1, (rows, cols), generator=g, device="cuda", dtype=torch.int8).to(dtype)


def test_activations():
    times, rows, cols = 270, 1000, 16384                           # 4.4e9 values
    g = torch.Generator(device="cuda").manual_seed(1)
    gate, up, dy = (torch.randn(rows, cols, generator=g, device="cuda", dtype=BF16) for _ in range(3))
    y0, s0 = A.gated_save8(gate, up)
    a0, b0 = A.gated_grad(dy, s0)
    y, s = A.gated_save8(gate.repeat(times, 1), up.repeat(times, 1))
    assert y.numel() > 1 << 32

    def repeats(big, small):
        return all(torch.equal(part, small) for part in big.view(times, rows, cols))
    assert repeats(y, y0)
    del y
    a, b = A.gated_grad(dy.repeat(times, 1), s)
    assert repeats(a, a0) and repeats(b, b0)


def test_weight_gradient():
    m, n, k, some = 4200001, 1040, 1030, 700
    x = whole(m, k, 7, 2)
    dy = torch.zeros(m, n, dtype=BF16, device="cuda")              # only the first and the last tokens count
    dy[:some], dy[-some:] = whole(some, n, 4, 3), whole(some, n, 4, 4)
    s = A.save8(x)
    assert dy.numel() > 1 << 32 and x.numel() > 1 << 32 and torch.equal(s.load(), x)
    w, b = A.weight_grad(dy, s, bias=True)
    d = torch.cat([dy[:some], dy[-some:]]).double()
    v = torch.cat([x[:some], x[-some:]]).double()
    assert torch.equal(w, (d.t().contiguous() @ v).to(BF16)) and torch.equal(b, d.sum(0).to(BF16))


def test_embedding():
    vocab, dim, n = 524288, 8200, 600001
    w = whole(vocab, dim, 100, 5)
    g = torch.Generator(device="cuda").manual_seed(6)
    ids = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    ids[-3:] = vocab - 1
    ids[:2] = torch.tensor([vocab - 1, -100], device="cuda")
    y = E.embedding(ids, w)
    assert y.numel() > 1 << 32 and w.numel() > 1 << 32 and not y[1].any()
    for i in range(2, n, 60000):
        assert torch.equal(y[i:i + 60000], w[ids[i:i + 60000]])
    grad = E.embedding_grad(ids, y, vocab)                         # each token: its row as often as it is named
    times = torch.bincount(ids.clamp_min(0), minlength=vocab)
    times[0] -= 1                                                  # (the id that is none)
    assert times.max().item() < 20                                 # so that times * w has 11 bits at most
    for i in range(0, vocab, 65536):
        want = (w[i:i + 65536].float() * times[i:i + 65536, None]).to(BF16)
        assert torch.equal(grad[i:i + 65536], want)


def test_log_probabilities():
    period, times = 1 << 20, 2049
    n = period * times
    g = torch.Generator(device="cuda").manual_seed(7)
    lp, old, adv = (torch.randn(period, generator=g, device="cuda") * 0.2 - s for s in (2, 2, 0))
    small = L.policy_loss(lp, old, adv)
    big = L.policy_loss(lp.repeat(times), old.repeat(times), adv.repeat(times))
    assert big.numel() > 1 << 31 and all(torch.equal(part, small) for part in big.view(times, period))
    del big, small, old, adv
    x = torch.full((n,), -2.0 ** -10, device="cuda")               # sums of whole multiples of 2^-10, exact in 64 bits
    x[-3] = -1.0
    offsets = torch.tensor([0, 5, n - 4000, n - 3, n], device="cuda")
    x.requires_grad_()
    r = L.preference_loss(x, offsets, beta=0.5, average=True)
    step = 2.0 ** -10
    want = torch.tensor([[-step, -step], [-step, -(1 + 2 * step) / 3]]).double() * 0.5
    assert torch.equal(r.reward.cpu(), want.float())
    grad, = torch.autograd.grad(r.loss.sum(), x)
    d = want[:, 0] - want[:, 1]
    up = 0.5 * torch.sigmoid(-d)
    lengths = (5, n - 4005, 3997, 3)
    for i, (start, length) in enumerate(zip((0, 5, n - 4000, n - 3), lengths)):
        part = grad[start:start + length]
        assert bool((part == part[0]).all())
        assert part[0].item() == pytest.approx(up[i // 2].item() / length * (1 if i % 2 else -1), rel=2e-7)
