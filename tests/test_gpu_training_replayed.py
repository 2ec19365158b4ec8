"""The whole step of test_gpu_training_run.py with the reference's term, at old and reference log
probabilities near the model's own, so that everything stays finite: eager, and captured and replayed with
the program's own eager work between the replays, equal bit for bit in every parameter and loss."""
import pytest
import torch

from compressed_adamw_state_amd import activations as A
from compressed_adamw_state_amd import embedding as E
from compressed_adamw_state_amd import losses as L
from compressed_adamw_state_amd import optim as O

pytestmark = pytest.mark.gpu

D, H, VOCAB, ROWS = 48, 80, 611, 90


def forward(ids, ps):
    t, a, b, c = ps
    x = E.embedding(ids, t)
    return A.gated(torch.nn.functional.linear(x, a, b)) @ c.t()


@pytest.mark.parametrize("kl", [0.05, 0.5])
def test_replays_equal_eager_steps_and_stay_finite(kl):
    g = torch.Generator().manual_seed(5)
    start = [(torch.randn(*s, generator=g) * f).cuda() for s, f in
             (((VOCAB, D), 1.0), ((2 * H, D), 0.2), ((2 * H,), 0.1), ((VOCAB, H), 0.2))]
    first = [p.to(torch.bfloat16) for p in start]
    data = []
    for _ in range(4):
        i, t = (torch.randint(0, VOCAB, (ROWS,), generator=g).cuda() for _ in range(2))
        lp = L.token_logprobs(forward(i, first), t).logprob
        data.append((i, t, lp + 0.1 * torch.randn(ROWS, generator=g).cuda(), torch.randn(ROWS, generator=g).cuda(),
                     lp + 0.1 * torch.randn(ROWS, generator=g).cuda()))
    ids, targets, old, adv, ref = (v.clone() for v in data[0])
    weight = torch.full((ROWS,), 1.0 / ROWS, device="cuda")
    offsets = torch.tensor([0, 20, 45, 70, ROWS], device="cuda")

    def put(k):
        for t, v in zip((ids, targets, old, adv, ref), data[k]):
            t.copy_(v)

    def make():
        ps = [torch.nn.Parameter(t.clone()) for t in start]
        opt = O.FlashAdamW(ps, lr=1e-3, capturable=True)
        for p in ps:
            p.grad = torch.zeros_like(p)

        @torch.no_grad()
        def step():
            t, a, b, c = ps
            x = E.embedding(ids, t)
            xs = A.save8(x)
            y, held = A.gated_save8(torch.nn.functional.linear(x, a, b), halves=True)
            ys = A.save8(y)
            z = y @ c.t()
            pref = L.preference_grad(z, targets, offsets, ref_logprob=ref)
            r = L.policy_grad(z, targets, old, adv, ref, weight, kl=kl, entropy=0.01, inplace=True)
            gz = r.grad + pref.grad
            gw, _ = A.weight_grad(gz, ys)
            gu, _ = A.gated_grad(gz @ c, held)
            ga, gb = A.weight_grad(gu, xs, bias=True)
            for p, v in zip(ps, (E.embedding_grad(ids, gu @ a, VOCAB), ga, gb, gw)):
                p.grad.copy_(v)
            opt.step()
            return r.loss, pref.loss
        return ps, step
    pa, eager = make()
    pb, captured = make()
    eager()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(pa, pb))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lb = captured()
    for k in (1, 2, 3, 1, 0, 2):
        before = [p.detach().clone() for p in pa]
        put(k)
        la = eager()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*la, *pa), (*lb, *pb)):
            assert bool(torch.isfinite(a).all()) and torch.equal(a, b), k
        assert all(not torch.equal(a, b) for a, b in zip(before, pa)), k
