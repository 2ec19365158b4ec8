"""The losses over rows of logits (include/flashopt_lm.h, losses.py) against
plain 64-bit forms (lm_plain.py, which derives the tolerances): log
probabilities, entropy, top alternatives, distillation, and their gradients,
over types, odd vocabularies around the kernels' chunk sizes, strided and
misaligned rows, masks, ties, and rows whose mask leaves nothing."""
import math

import pytest
import torch

import lm_plain as P
from compressed_adamw_state_amd import flashopt as F
from compressed_adamw_state_amd import losses as L

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
VOCABS = [1, 2, 7, 8, 9, 64, 65, 1000, 4095, 8191, 8193, 16383, 16385, 50257, 131073, 300001]


def near(got, ref, tol, dtype=torch.float32):
    """got (of dtype) is within tol and half a step of ref; equal where ref is not finite."""
    got, ref = got.double().cpu(), ref.cpu()
    fin = torch.isfinite(ref)
    assert torch.equal(got[~fin].nan_to_num(7e300), ref[~fin].nan_to_num(7e300))
    tol = tol.cpu() if torch.is_tensor(tol) else torch.full_like(ref, tol)
    lim = tol * (1 + P.half_step(dtype)) + P.half_step(dtype) * ref.abs() + P.smallest(dtype) + 2.0 ** -126
    bad = fin & ~((got - ref).abs() <= lim)
    if bool(bad.any()):
        k = torch.where(fin, (got - ref).abs() / lim, 0.0).flatten().argmax()
        raise AssertionError(f"{int(bad.sum())} of {ref.numel()} outside; worst at {int(k)}: "
                             f"{got.flatten()[k].item()} for {ref.flatten()[k].item()}, "
                             f"allowed {lim.flatten()[k].item()}")


def draw(rows, vocab, dtype, seed, masked=False, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g) * scale
    if masked:
        x[torch.rand(rows, vocab, generator=g) < 0.5] = -math.inf
    t = torch.randint(0, vocab, (rows,), generator=g)
    if rows > 2:
        t[1] = -100
        t[2] = vocab + 5
    return x.to(dtype), t, g


def place(x, how):
    """The logits on the GPU: dense, or as rows of a wider buffer, or starting one element in."""
    if how == "dense":
        return x.cuda()
    rows, vocab = x.shape
    if how == "strided":
        buf = torch.full((rows, vocab + 13), 1e4 if x.dtype != torch.float32 else 1e30, dtype=x.dtype, device="cuda")
        v = buf[:, 3:3 + vocab]
    else:
        buf = torch.zeros(rows * vocab + 1, dtype=x.dtype, device="cuda")
        v = buf[1:].view(rows, vocab)
    v.copy_(x)
    return v


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", VOCABS)
def test_logprob_entropy_top(dtype, vocab):
    for rows, how, masked, temp in ((1, "dense", False, 1.0), (5, "strided", True, 0.7), (3, "offset", False, 2.5)):
        x, t, _ = draw(rows, vocab, dtype, vocab + rows, masked)
        k = min(64, vocab) if rows == 1 else min(5, vocab)
        r = L.token_logprobs(place(x, how), t.cuda(), top=k, temperature=temp)
        lp, lt, en, et = P.logprob(x, t, temp)
        near(r.logprob, lp, lt)
        near(r.entropy, en, et)
        ids = P.top(x, k)
        assert torch.equal(r.top_id.cpu(), ids)
        for c in range(k):
            v, vt, _, _ = P.logprob(x, ids[:, c], temp)
            near(r.top_logprob[:, c], v, vt)


@pytest.mark.parametrize("dtype", TYPES)
def test_ties_go_to_the_lowest_id(dtype):
    vocab = 40000
    g = torch.Generator().manual_seed(5)
    few = torch.randint(-2, 3, (4, vocab), generator=g).float() * 0.5     # five values, 8000 of each
    few[1] = 0.25                                                         # one value
    few[2] = -math.inf
    few[2, 33333] = 1.0                                                   # one token allowed
    few[3, ::2] = 0.0
    few[3, 1::2] = -0.0                                                   # equal as numbers
    x = few.to(dtype)
    for k in (1, 20, 64):
        r = L.token_logprobs(x.cuda(), top=k)
        assert torch.equal(r.top_id.cpu(), P.top(x, k))
    assert r.logprob is None
    near(r.entropy, P.logprob(x, torch.zeros(4, dtype=torch.int64), 1.0)[2], 1e-4)
    assert r.top_logprob[2, 0].item() == 0.0 and r.top_logprob[2, 1].item() == -math.inf


@pytest.mark.parametrize("dtype", TYPES)
def test_top_in_one_thread(dtype):
    """The largest entries next to each other, and entries in falling and rising order."""
    vocab = 30000
    x = torch.randn(4, vocab, generator=torch.Generator().manual_seed(3))
    x[0, 10000:10064] = torch.arange(64).float() + 10
    x[1] = -torch.arange(vocab).float() / 64
    x[2] = torch.arange(vocab).float() / 64
    x = x.to(dtype)
    for k in (3, 64):
        assert torch.equal(L.token_logprobs(x.cuda(), top=k).top_id.cpu(), P.top(x, k))


@pytest.mark.parametrize("dtype", TYPES)
def test_special_rows(dtype):
    vocab, low = 9000, torch.finfo(dtype).min
    x = torch.randn(8, vocab, generator=torch.Generator().manual_seed(8))
    x[0] = -math.inf                                       # nothing left
    x[1] = low                                             # the lowest value everywhere: uniform
    x[2, 1:] = low                                         # masked by the lowest value
    x[3] = torch.finfo(dtype).max / 2
    x[3, 7] = torch.finfo(dtype).max
    x[4, 100] = math.nan
    x[5, 100] = math.inf
    x[6, 1:] = -math.inf
    x = x.to(dtype)
    t = torch.tensor([3, 4, 0, 7, 5, 5, 0, 11])
    xc = x.cuda().requires_grad_()
    r = L.token_logprobs(xc, t.cuda(), top=4)
    lp, lt, en, et = P.logprob(x, t, 1.0)
    ok = [0, 1, 2, 3, 6, 7]
    near(r.logprob[ok].detach(), lp[ok], lt[ok])
    near(r.entropy[ok].detach(), en[ok], et[ok])
    assert lp[0].item() == -math.inf and abs(en[1].item() - math.log(vocab)) < 1e-9
    assert bool(torch.isnan(r.logprob[[4, 5]]).all()) and bool(torch.isnan(r.entropy[[4, 5]]).all())
    assert torch.equal(r.top_id[ok].cpu(), P.top(x, 4)[ok])
    assert bool(((r.top_id >= 0) & (r.top_id < vocab)).all())
    gl, gh = torch.arange(1.0, 9.0), torch.linspace(-1, 1, 8)
    gr, = torch.autograd.grad((r.logprob, r.entropy), xc, (gl.cuda(), gh.cuda()))
    ref, tol = P.logprob_grad(x[ok], t[ok], gl[ok], gh[ok], 1.0)
    near(gr[ok], ref, tol, dtype)
    assert bool((gr[0] == 0).all())
    ids = torch.tensor([[0, 5, 7, 7, -1]] * 8)
    tlp = torch.log(torch.tensor([[0.3, 0.2, 0.1, 0.1, 0.25]] * 8))
    for tail in (False, True):
        loss, gd = L.distill_grad(xc.detach(), ids.cuda(), tlp.cuda(), gl.cuda(), tail=tail)
        fin = [0, 1, 3, 7]                                 # the rest have infinite loss or NaN
        a, at, b, bt = P.distill(x[fin], ids[fin], tlp[fin], tail, 1.0, gl[fin])
        near(loss[fin], a, at)
        near(gd[fin], b, bt, dtype)
        assert loss[0].item() == 0 and bool((gd[0] == 0).all())
        assert loss[6].item() == math.inf
        assert bool(torch.isnan(loss[[4, 5]]).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", VOCABS)
def test_logprob_gradient(dtype, vocab):
    for rows, how, masked, temp in ((1, "dense", False, 1.0), (5, "strided", True, 0.7), (3, "offset", False, 2.5)):
        x, t, g = draw(rows, vocab, dtype, 3 * vocab + rows, masked)
        gl, gh = torch.randn(rows, generator=g), torch.randn(rows, generator=g)
        xg = place(x, how).requires_grad_()
        r = L.token_logprobs(xg, t.cuda(), temperature=temp)
        for a, b in ((gl, gh), (gl, None), (None, gh)):
            outs = [o for o, u in ((r.logprob, a), (r.entropy, b)) if u is not None]
            ups = [u.cuda() for u in (a, b) if u is not None]
            got, = torch.autograd.grad(outs, xg, ups, retain_graph=True)
            ref, tol = P.logprob_grad(x, t, a, b, temp)
            near(got, ref, tol, dtype)
        one = L.token_logprobs_grad(place(x, how), t.cuda(), gl.cuda(), gh.cuda(), temperature=temp)
        ref, tol = P.logprob_grad(x, t, gl, gh, temp)
        near(one.grad, ref, tol, dtype)
        lp, lt, en, et = P.logprob(x, t, temp)
        near(one.logprob, lp, lt)
        near(one.entropy, en, et)
        dense = place(x, how)                              # the gradient in the logits' place
        around = dense._base.clone() if how == "strided" else None
        two = L.token_logprobs_grad(dense, t.cuda(), gl.cuda(), None, temperature=temp, inplace=True)
        assert two.grad.data_ptr() == dense.data_ptr()
        ref, tol = P.logprob_grad(x, t, gl, None, temp)
        near(dense, ref, tol, dtype)
        if how == "strided":                               # what lies between the rows stays
            assert torch.equal(around[:, :3], dense._base[:, :3])
            assert torch.equal(around[:, 3 + vocab:], dense._base[:, 3 + vocab:])


def teacher(x, k, temp, seed):
    g = torch.Generator().manual_seed(seed)
    z = (x.double() + torch.randn(x.shape, generator=g)) / temp
    v, i = torch.topk(z, k, dim=1)
    return i, (v - torch.logsumexp(z, 1, keepdim=True)).float()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", VOCABS)
def test_distill(dtype, vocab, tail):
    for rows, how, temp, k in ((1, "dense", 1.0, 64), (4, "strided", 0.7, 1), (3, "offset", 2.0, 17)):
        k = min(k, vocab)
        x, _, g = draw(rows, vocab, dtype, 7 * vocab + rows)
        ids, tlp = teacher(x, k, temp, vocab)
        up = torch.randn(rows, generator=g)
        a, at, b, bt = P.distill(x, ids, tlp, tail, temp, up)
        loss, grad = L.distill_grad(place(x, how), ids.cuda(), tlp.cuda(), up.cuda(), tail=tail, temperature=temp)
        near(loss, a, at)
        near(grad, b, bt, dtype)
        xg = place(x, how).requires_grad_()
        lo = L.distill_loss(xg, ids.cuda(), tlp.cuda(), tail=tail, temperature=temp)
        near(lo.detach(), a, at)
        got, = torch.autograd.grad(lo, xg, up.cuda())
        near(got, b, bt, dtype)
        here = place(x, how)
        L.distill_grad(here, ids.cuda(), tlp.cuda(), up.cuda(), tail=tail, temperature=temp, inplace=True)
        near(here, b, bt, dtype)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_distill_odd_lists(dtype, tail):
    """Repeated ids, skipped ids, none at all, all of the vocabulary, a student far from the teacher."""
    vocab, rows = 20000, 6
    x, _, g = draw(rows, vocab, dtype, 77, scale=2.0)
    ids, tlp = teacher(x, 8, 1.0, 5)
    ids[0, 3] = ids[0, 1]
    ids[0, 7] = ids[0, 1]
    ids[1, 0], ids[1, 5] = -100, vocab
    ids[2, :] = -1
    x[3, ids[3]] = -30.0                                   # the student finds them unlikely
    x[4] = -30.0
    x[4, ids[4]] = 30.0                                    # the student finds nothing else likely
    tlp[5] = -math.inf
    tlp[5, 2] = 0.0                                        # the teacher knows one token
    up = torch.randn(rows, generator=g)
    a, at, b, bt = P.distill(x, ids, tlp, tail, 1.0, up)
    loss, grad = L.distill_grad(x.cuda(), ids.cuda(), tlp.cuda(), up.cuda(), tail=tail)
    near(loss, a, at)
    near(grad, b, bt, dtype)
    assert loss[2].item() == 0 and bool((grad[2] == 0).all())
    whole = torch.arange(50).repeat(2, 1)
    y = torch.randn(2, 50, generator=g).to(dtype)
    t = torch.log_softmax(torch.randn(2, 50, generator=g).double(), 1).float()
    a, at, b, bt = P.distill(y, whole, t, tail, 1.0, up[:2])
    loss, grad = L.distill_grad(y.cuda(), whole.cuda(), t.cuda(), up[:2].cuda(), tail=tail)
    near(loss, a, at)
    near(grad, b, bt, dtype)


def test_gradients_against_differences():
    """Central differences of the library's own losses in FP32, h = 2^-5: the
    third derivatives of these losses are below 2 (weights at most 1), so the
    difference is off by h^2 / 3 < 4e-4, and the losses' own rounding of at
    most 2e-5 adds 2e-5 / h = 7e-4."""
    vocab, h = 37, 2.0 ** -5
    g = torch.Generator().manual_seed(1)
    x = torch.randn(1, vocab, generator=g)
    both = torch.cat([x + h * torch.eye(vocab), x - h * torch.eye(vocab)]).cuda()
    t = torch.full((2 * vocab,), 5)
    r = L.token_logprobs(both, t.cuda())
    f = 0.5 * r.logprob + 0.25 * r.entropy
    diff = (f[:vocab] - f[vocab:]) / (2 * h)
    one = L.token_logprobs_grad(x.cuda(), t[:1].cuda(), torch.tensor([0.5]).cuda(), torch.tensor([0.25]).cuda())
    assert (diff - one.grad[0]).abs().max().item() < 1.1e-3
    ids, tlp = teacher(x, 6, 1.0, 2)
    for tail in (False, True):
        f = L.distill_loss(both, ids.repeat(2 * vocab, 1).cuda(), tlp.repeat(2 * vocab, 1).cuda(), tail=tail)
        diff = (f[:vocab] - f[vocab:]) / (2 * h)
        _, grad = L.distill_grad(x.cuda(), ids.cuda(), tlp.cuda(), torch.ones(1).cuda(), tail=tail)
        assert (diff - grad[0]).abs().max().item() < 1.1e-3


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [4101, 8193, 8203, 12301, 16387, 24580, 32768, 32771, 40000, 50257, 65536, 65543])
def test_rows_of_one_block(dtype, vocab):
    """256 rows and more: each held or streamed by one block (more rows than blocks at once for the
    small vocabularies), with rows that need the exceptional paths."""
    rows = 1100 if vocab < 16000 else 300
    x, t, g = draw(rows, vocab, dtype, vocab)
    x[3] = -math.inf                                       # nothing left
    x[4, :vocab - 2] = -math.inf                           # the row's last entries only
    x[5] = torch.finfo(dtype).min                          # the lowest value everywhere
    x[6, vocab // 2] = 300.0                               # far above what comes first
    x[7, vocab - 1] = 60000.0                              # the last entry far above all
    x[8, ::3] = -math.inf
    x[9] = x[9].sort()[0]                                  # rising
    x[10] = -math.inf
    x[10, 1] = -2.0
    x[11] *= 1000                                          # large magnitudes
    t[4], t[7], t[10] = vocab - 1, vocab - 1, 1
    gl, gh = torch.randn(rows, generator=g), torch.randn(rows, generator=g)
    xc, tc, glc, ghc = x.cuda(), t.cuda(), gl.cuda(), gh.cuda()
    for temp, b in ((1.0, None), (0.7, ghc)):
        r = L.token_logprobs_grad(xc, tc, glc, b, temperature=temp)
        ref, tol = P.logprob_grad(xc, tc, glc, b, temp)
        near(r.grad, ref, tol, dtype)
        lp, lt, en, et = P.logprob(xc, tc, temp)
        near(r.logprob, lp, lt)
        near(r.entropy, en, et)
        wide = place(x, "strided")
        two = L.token_logprobs_grad(wide, tc, glc, b, temperature=temp, inplace=True)
        near(wide, ref, tol, dtype)
        assert torch.equal(two.logprob, r.logprob)
        del ref, tol
    r = L.token_logprobs(xc, tc, top=20)
    near(r.logprob, *P.logprob(xc, tc, 1.0)[:2])
    assert torch.equal(r.top_id, P.top(xc, 20))
    xc[13, 5], xc[14, vocab - 1] = math.nan, math.inf      # and nothing but those rows is lost
    r = L.token_logprobs_grad(xc, tc, glc)
    bad = torch.isnan(r.grad).any(1)
    assert bad.nonzero().flatten().tolist() == [13, 14] and torch.isnan(r.entropy[[13, 14]]).all()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [1003, 16385, 50257, 131075])
def test_distill_rows_of_one_block(dtype, vocab, tail):
    rows = 260
    x, _, g = draw(rows, vocab, dtype, vocab + 1)
    x[3] = -math.inf
    x[5] = torch.finfo(dtype).min
    x[6, vocab // 2] = 300.0
    x[11] *= 100
    xc = x.cuda()
    z = xc.double() + torch.randn(rows, vocab, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    z[3] = 0.0
    v, ids = torch.topk(z, 30, dim=1)
    tlp = (v - torch.logsumexp(z, 1, keepdim=True)).float()
    up = torch.randn(rows, generator=g).cuda()
    a, at, b, bt = P.distill(xc, ids, tlp, tail, 1.0, up)
    loss, grad = L.distill_grad(xc, ids, tlp, up, tail=tail)
    near(loss, a, at)
    near(grad, b, bt, dtype)
    wide = place(x, "strided")
    loss2, _ = L.distill_grad(wide, ids, tlp, up, tail=tail, inplace=True)
    near(wide, b, bt, dtype)
    assert torch.equal(loss, loss2)


def test_many_rows_and_shapes():
    """More rows than the GPU holds blocks at once; leading dimensions; no rows."""
    x, t, g = draw(3000, 1003, torch.bfloat16, 9)
    r = L.token_logprobs(x.cuda().view(30, 100, 1003), t.cuda().view(30, 100), top=3)
    lp, lt, en, et = P.logprob(x, t, 1.0)
    assert r.logprob.shape == (30, 100) and r.top_id.shape == (30, 100, 3)
    near(r.logprob.view(-1), lp, lt)
    near(r.entropy.view(-1), en, et)
    assert torch.equal(r.top_id.view(-1, 3).cpu(), P.top(x, 3))
    up = torch.rand(3000, generator=g)
    ids, tlp = teacher(x, 5, 1.0, 4)
    a, at, b, bt = P.distill(x, ids, tlp, True, 1.0, up)
    loss, grad = L.distill_grad(x.cuda(), ids.cuda(), tlp.cuda(), up.cuda())
    near(loss, a, at)
    near(grad, b, bt, torch.bfloat16)
    none = L.token_logprobs(torch.empty(0, 10, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), top=2)
    assert none.logprob.shape == (0,) and none.top_id.shape == (0, 2)
    vec = L.token_logprobs(x[7].cuda(), t[7].cuda(), top=1)
    near(vec.logprob.view(1), lp[7:8], lt[7:8])


def test_other_stream_and_repeat():
    """The same call twice gives the same bits, on the default and on a side stream."""
    x, t, g = draw(65, 50257, torch.float16, 21)
    xc, tc = x.cuda(), t.cuda()
    up = torch.randn(65, generator=g).cuda()
    ids, tlp = (v.cuda() for v in teacher(x, 20, 1.0, 3))

    def both():
        r = L.token_logprobs(xc, tc, top=7)
        return (r.logprob, r.entropy, r.top_logprob, r.top_id, *L.distill_grad(xc, ids, tlp, up),
                L.token_logprobs_grad(xc, tc, up, up).grad)
    first = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = both()
    torch.cuda.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_gradient_in_the_logits_place_of_cut_rows():
    """Few rows, each cut into many segments whose blocks replace their logits: the listed and given
    entries of other segments must have been read before.  Equal to the gradient written elsewhere."""
    for rows, vocab in ((1, 131072), (2, 100003), (5, 200000)):
        x, t, g = draw(rows, vocab, torch.bfloat16, vocab)
        ids, tlp = (v.cuda() for v in teacher(x, 64, 1.0, 3))
        up = torch.randn(rows, generator=g).cuda()
        for _ in range(5):
            a, b = x.cuda(), x.cuda()
            loss, grad = L.distill_grad(a, ids, tlp, up)
            loss2, _ = L.distill_grad(b, ids, tlp, up, inplace=True)
            assert torch.equal(loss, loss2) and torch.equal(grad, b)
            b = x.cuda()
            r = L.token_logprobs_grad(a, t.cuda(), up, up)
            r2 = L.token_logprobs_grad(b, t.cuda(), up, up, inplace=True)
            assert torch.equal(r.logprob, r2.logprob) and torch.equal(r.entropy, r2.entropy)
            assert torch.equal(r.grad, b)


def test_gradient_beside_the_logits():
    """Rows of logits and of their gradient by turns in one buffer: no row touches another's."""
    for rows, vocab in ((3, 50257), (300, 9000)):
        x, t, g = draw(rows, vocab, torch.bfloat16, vocab)
        both = torch.zeros(rows, 2, vocab, dtype=torch.bfloat16, device="cuda")
        both[:, 0] = x.cuda()
        up = torch.randn(rows, generator=g).cuda()
        want = L.token_logprobs_grad(x.cuda(), t.cuda(), up, up).grad
        F.flashopt_logprob_grad(both[:, 0], t.cuda(), up, up, both[:, 1])
        assert torch.equal(both[:, 1], want) and torch.equal(both[:, 0].cpu(), x)
        with pytest.raises(F.FlashoptError):
            F.flashopt_logprob_grad(both[:, 0], t.cuda(), up, up, both.view(rows, -1)[:, 1:vocab + 1])


@pytest.mark.parametrize("rows,vocab", [(3, 90001), (3, 1000), (300, 9000)])
def test_rows_without_a_distribution_ignore_their_upstream(rows, vocab):
    """Cut rows, whole rows, rows in registers: nothing but -inf gives a gradient of 0, whatever
    the upstream gradients."""
    x = torch.randn(rows, vocab, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    x[1] = -math.inf
    t = torch.full((rows,), 5, device="cuda")
    up = torch.ones(rows, device="cuda")
    up[1] = math.nan
    xg = x.clone().requires_grad_()
    r = L.token_logprobs(xg, t)
    grads = [L.token_logprobs_grad(x, t, up, up).grad, L.token_logprobs_grad(x, t, up).grad,
             torch.autograd.grad((r.logprob, r.entropy), xg, (up, up))[0]]
    for tail in (False, True):
        grads.append(L.distill_grad(x, t.view(rows, 1), -up.view(rows, 1).nan_to_num(0.5), up, tail=tail)[1])
    for gr in grads:
        assert bool((gr[1] == 0).all()) and bool(torch.isfinite(gr).all())


def test_in_place_refuses_a_stale_backward():
    """torch's graph sees that the logits' values are gone."""
    x = torch.randn(4, 100, device="cuda", requires_grad=True)
    y = x * 1.0
    s = (y * y).sum()                                     # keeps y for its backward pass
    L.token_logprobs_grad(y, torch.zeros(4, dtype=torch.int64, device="cuda"), torch.ones(4, device="cuda"), inplace=True)
    with pytest.raises(RuntimeError):
        s.backward()


def test_captured_and_replayed():
    """The one-call forms in a HIP graph, replayed over new logits with eager work in between."""
    rows, vocab = 9, 33001
    x, t, _ = draw(rows, vocab, torch.bfloat16, 31)
    ids, tlp = teacher(x, 12, 1.0, 1)
    xs, ts, ids, tlp = x.cuda(), t.cuda(), ids.cuda(), tlp.cuda()
    up = torch.linspace(-1, 1, rows, device="cuda")

    def work():
        r = L.token_logprobs(xs, ts, top=9)
        return (r.logprob, r.top_id, *L.distill_grad(xs, ids, tlp, up), L.token_logprobs_grad(xs, ts, up).grad)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for k in range(3):
        xs.copy_(draw(rows, vocab, torch.bfloat16, 50 + k)[0])
        eager = [o.clone() for o in work()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, eager):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("words", [512, 1536, 2048, 3584, 4096, 8192])
def test_rows_at_the_borders_of_the_cut(dtype, words):
    """Rows that one block takes whole, in short and in long chunks, and the first that it does not."""
    for over in (0, 1):
        vocab = words * (4 if dtype == torch.float32 else 8) + over
        test_logprob_entropy_top(dtype, vocab)
        test_logprob_gradient(dtype, vocab)
        test_distill(dtype, vocab, over == 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,words", [(1, 1025), (1, 4096), (1, 4097), (3, 1024), (127, 4097), (128, 4097), (130, 8192), (130, 8193)])
def test_gradient_of_few_whole_rows(dtype, rows, words):
    """Just before and behind the borders of the rows that a block holds in registers; the gradient in
    the logits' place and elsewhere."""
    vocab = words * (4 if dtype == torch.float32 else 8) + 3
    x, t, g = draw(rows, vocab, dtype, rows + vocab, True)
    gl, gh = torch.randn(rows, generator=g), torch.randn(rows, generator=g)
    ref, tol = P.logprob_grad(x.cuda(), t.cuda(), gl.cuda(), gh.cuda(), 1.0)
    r = L.token_logprobs_grad(x.cuda(), t.cuda(), gl.cuda(), gh.cuda())
    near(r.grad, ref, tol, dtype)
    b = x.cuda()
    r2 = L.token_logprobs_grad(b, t.cuda(), gl.cuda(), gh.cuda(), inplace=True)
    assert torch.equal(b, r.grad) and torch.equal(r2.logprob, r.logprob) and torch.equal(r2.entropy, r.entropy)
