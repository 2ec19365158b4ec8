"""A run of the language-model operators as they are used together: weights
trained by FlashAdamW, exported in 8 bits from its state, the 8-bit layer's
logits, its top alternatives, the student's distillation gradient, the fused
step on it.  Each stage against its plain 64-bit form on what the stage
before it gave; and the ablation command's study runs."""
import math

import pytest
import torch

import lm_plain as P
from compressed_adamw_state_amd import ablations
from compressed_adamw_state_amd import flashopt as F
from compressed_adamw_state_amd import int8 as I
from compressed_adamw_state_amd import losses as L
from compressed_adamw_state_amd import optim as O

pytestmark = pytest.mark.gpu


def test_one_step_from_an_8_bit_teacher():
    g = torch.Generator().manual_seed(4)
    d, vocab, rows, top, temp = 96, 5003, 70, 12, 2.0
    w = torch.nn.Parameter((torch.randn(vocab, d, generator=g) * 0.2).cuda())
    opt = O.FlashAdamW([w], lr=1e-2)
    for _ in range(3):
        w.grad = torch.randn(vocab, d, generator=g).cuda().to(torch.bfloat16)
        opt.step()
    rows8 = opt.export_int8(w)
    master, _, _ = opt.export_fp32(w)
    q, s = P.row_codes(master.view(vocab, d).cpu())
    assert torch.equal(rows8.codes[:, :d].cpu(), q) and torch.equal(rows8.scale.cpu(), s)

    x = torch.randn(rows, d, generator=g).to(torch.bfloat16)
    logits = I.int8_linear(x.cuda(), rows8)
    xq, xs = P.row_codes(x)
    ref, tol = P.int8_product(xq, xs, q, s, None, torch.bfloat16)
    assert bool(((logits.cpu().double() - ref).abs() <= tol).all())

    t = L.token_logprobs(logits, top=top, temperature=temp)
    ids = P.top(logits.cpu(), top)
    assert torch.equal(t.top_id.cpu(), ids)
    for c in range(top):
        lp, lt, _, _ = P.logprob(logits.cpu(), ids[:, c], temp)
        assert bool(((t.top_logprob[:, c].cpu().double() - lp).abs() <= lt + P.U * lp.abs()).all())

    student = torch.nn.Parameter((torch.randn(vocab, d, generator=g) * 0.2).cuda())
    sopt = O.FlashAdamW([student], lr=1e-2)
    out = x.cuda() @ student.t()
    up = torch.full((rows,), temp * temp / rows)
    loss, grad = L.distill_grad(out.detach(), t.top_id, t.top_logprob, up.cuda(), temperature=temp)
    a, at, b, bt = P.distill(out.detach().cpu(), ids, t.top_logprob.cpu(), True, temp, up)
    assert bool(((loss.cpu().double() - a).abs() <= at + P.U * a.abs()).all())
    half = P.half_step(torch.bfloat16)
    lim = bt * (1 + half) + half * b.abs() + P.smallest(torch.bfloat16)
    assert bool(((grad.cpu().double() - b).abs() <= lim).all())
    # the same gradient by way of torch's graph, and into the weight: a product of
    # BF16 gradients and inputs summed over 70 rows in FP32, rounded to BF16
    auto, = torch.autograd.grad(L.distill_loss(out, t.top_id, t.top_logprob, temperature=temp), out, up.cuda(),
                                retain_graph=True)
    assert bool(((auto.cpu().double() - b).abs() <= lim).all())
    out.backward(grad)
    want = grad.cpu().double().t() @ x.double()
    most = grad.cpu().double().abs().t() @ x.double().abs()
    got = student.grad.cpu().double()
    assert bool(((got - want).abs() <= half * want.abs() + 72 * P.U * most + P.smallest(torch.bfloat16)).all())
    before = student.detach().clone()
    sopt.step()
    assert bool((student != before).any()) and bool(torch.isfinite(student.float()).all())


def test_the_study_runs():
    r = ablations.distillation_study(steps=3, batch=256)
    for side in ("teacher", "student"):
        for name in ("bf16", "int8"):
            assert all(math.isfinite(v) for v in r[side][name].values()), (side, name, r[side][name])
    assert r["teacher"]["bf16"]["same_best"] == 1.0


def test_the_run_captured_and_replayed():
    """The whole step without torch's graph: product in 8 bits, top alternatives, gradient, product for the
    weight's gradient, scheduled fused step; each replay equal to the eager step."""
    g = torch.Generator().manual_seed(9)
    d, vocab, rows = 64, 2001, 40
    teacher = I.Int8Weight.from_weight((torch.randn(vocab, d, generator=g) * 0.3).cuda())
    init = (torch.randn(vocab, d, generator=g) * 0.3).cuda()
    up = torch.full((rows,), 1.0 / rows, device="cuda")
    x = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    inputs = [torch.randn(rows, d, generator=g).to(torch.bfloat16) for _ in range(4)]

    def make():
        w = torch.nn.Parameter(init.clone())
        opt = O.FlashAdamW([w], lr=1e-2, capturable=True)
        w.grad = torch.zeros(vocab, d, dtype=torch.bfloat16, device="cuda")

        @torch.no_grad()
        def step():
            t = L.token_logprobs(I.int8_linear(x, teacher), top=8)
            out = x @ w.t()
            loss, grad = L.distill_grad(out, t.top_id, t.top_logprob, up, inplace=True)
            w.grad.copy_(grad.t() @ x)
            opt.step()
            return loss
        return w, opt, step
    wa, _, eager = make()
    wb, _, captured = make()
    x.copy_(inputs[0])
    la = eager()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(wa, wb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lb = captured()
    for k in (1, 2, 3):
        x.copy_(inputs[k])
        la = eager()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(la, lb) and torch.equal(wa, wb), k
