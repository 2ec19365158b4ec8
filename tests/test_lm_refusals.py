"""Host validation of the language-model operators (include/flashopt_lm.h):
every bad call is refused before anything is launched (no GPU call is made
here: each case fails validation first), and the Python layers refuse what
the C calls cannot see."""
import ctypes

import pytest
import torch

from compressed_adamw_state_amd import flashopt as F
from compressed_adamw_state_amd import int8 as I
from compressed_adamw_state_amd import losses as L

P = ctypes.c_void_p
A, ODD = P(0x10000), P(0x10001)                  # never dereferenced
BF16, FP32 = 0, 2


def logprob(logits=A, type=BF16, rows=4, vocab=100, stride=100, temp=1.0, targets=A, top=0, ws=A, wsb=1 << 20,
            lp=A, en=A, st=A, tl=None, ti=None):
    return F.lib().flashopt_logprob(logits, type, rows, vocab, stride, temp, targets, top, ws, wsb, lp, en, st, tl, ti, None)


def test_logprob_refusals():
    assert logprob(rows=0) == 0
    assert logprob(type=3) == -4 and logprob(type=-1) == -4
    assert logprob(rows=-1) == -2 and logprob(vocab=0) == -2 and logprob(vocab=524289, stride=524289) == -2
    assert logprob(stride=99) == -2 and logprob(rows=1 << 31) == -2 and logprob(stride=1 << 61) == -2
    assert logprob(rows=(1 << 23) + 1) == -2 and logprob(rows=1 << 22, vocab=524288, stride=524288, type=FP32) == -2
    for t in (0.0, -1.0, float("nan"), float("inf"), 1e-39, 1e39):
        assert logprob(temp=t) == -4
    assert logprob(logits=None) == -1 and logprob(logits=ODD) == -3 and logprob(logits=P(0x10002), type=FP32) == -3
    assert logprob(top=65) == -4 and logprob(top=-1) == -4 and logprob(vocab=3, top=4) == -4
    assert logprob(top=2) == -1 and logprob(top=2, tl=A) == -1
    assert logprob(targets=None) == -1 and logprob(targets=P(0x10004)) == -3
    assert logprob(st=P(0x10008)) == -3 and logprob(lp=P(0x10002)) == -3 and logprob(en=ODD) == -3
    assert logprob(top=1, tl=ODD, ti=A) == -3 and logprob(top=1, tl=A, ti=P(0x10004)) == -3
    big = dict(vocab=100000, stride=100000)
    need = F.lib().flashopt_logprob_workspace_bytes(BF16, 4, 100000, 0)
    assert need > 0 and logprob(wsb=need - 1, **big) == -6
    assert logprob(ws=P(0x10010), **big) == -6 and logprob(ws=None, **big) == -1
    assert F.lib().flashopt_logprob_workspace_bytes(9, 4, 100, 0) == 0
    assert F.lib().flashopt_logprob_workspace_bytes(BF16, 4, 100, 65) == 0
    assert F.lib().flashopt_logprob_workspace_bytes(BF16, -4, 100, 5) == 0
    assert F.lib().flashopt_logprob_workspace_bytes(BF16, 4, 100000, 5) >= need + 4 * 5 * 8


def test_logprob_gradient_refusals():
    def back(grad=A, gs=100, st=A, targets=A, gl=A, gh=None, rows=4):
        return F.lib().flashopt_logprob_backward(A, BF16, rows, 100, 100, 1.0, targets, st, gl, gh, grad, gs, None)
    assert back(rows=0) == 0 and back(grad=None) == -1 and back(st=None) == -1 and back(targets=None) == -1
    assert back(gs=99) == -2 and back(grad=ODD) == -3 and back(gl=P(0x10002)) == -3 and back(gh=ODD) == -3

    def both(grad=A, gs=100000, targets=A, gl=A, ws=A, wsb=1 << 20, lp=A):
        return F.lib().flashopt_logprob_grad(A, BF16, 4, 100000, 100000, 1.0, targets, gl, None, ws, wsb, lp, A, grad, gs, None)
    assert both(grad=None) == -1 and both(targets=None) == -1 and both(gl=P(0x10002)) == -3
    assert both(gs=99) == -2 and both(wsb=1) == -6 and both(ws=None) == -1 and both(lp=ODD) == -3


def test_distill_refusals():
    def fwd(rows=4, vocab=100000, ids=A, tlp=A, top=4, tail=1, ws=A, wsb=1 << 20, loss=A, st=A, temp=1.0):
        return F.lib().flashopt_distill(A, BF16, rows, vocab, vocab, temp, ids, tlp, top, tail, ws, wsb, loss, st, None)
    assert fwd(rows=0) == 0 and fwd(top=0) == -4 and fwd(top=65) == -4 and fwd(vocab=3) == -4 and fwd(tail=2) == -4
    assert fwd(ids=None) == -1 and fwd(tlp=None) == -1 and fwd(st=None) == -1 and fwd(ws=None) == -1
    assert fwd(ids=P(0x10004)) == -3 and fwd(tlp=ODD) == -3 and fwd(st=P(0x10008)) == -3 and fwd(wsb=1) == -6
    assert fwd(temp=0.0) == -4

    def back(ids=A, st=A, g=A, grad=A, gs=100, top=4):
        return F.lib().flashopt_distill_backward(A, BF16, 4, 100, 100, 1.0, ids, A, top, st, g, grad, gs, None)
    assert back(ids=None) == -1 and back(st=None) == -1 and back(g=None) == -1 and back(grad=None) == -1
    assert back(gs=1) == -2 and back(top=0) == -4 and back(grad=ODD) == -3 and back(g=ODD) == -3

    def both(g=A, grad=A, wsb=1 << 20, top=4, tail=0):
        return F.lib().flashopt_distill_grad(A, BF16, 4, 100000, 100000, 1.0, A, A, top, tail, g, A, wsb, A, grad,
                                             100000, None)
    assert both(g=None) == -1 and both(grad=None) == -1 and both(wsb=1) == -6 and both(top=0) == -4 and both(tail=-1) == -4


def test_int8_refusals():
    lib = F.lib()
    assert [lib.flashopt_int8_ld(k) for k in (1, 128, 129, 131072, 0, -5, 131073)] == [128, 128, 256, 131072, 0, 0, 0]

    def quant(x=A, type=BF16, rows=4, cols=100, stride=100, q=A, s=A):
        return lib.flashopt_quantize_rows(x, type, rows, cols, stride, q, s, None)
    assert quant(rows=0) == 0 and quant(type=5) == -4 and quant(rows=-1) == -2 and quant(cols=0) == -2
    assert quant(cols=131073, stride=131073) == -2 and quant(stride=99) == -2 and quant(rows=(1 << 24) + 1) == -2
    assert quant(x=None) == -1 and quant(q=None) == -1 and quant(s=None) == -1
    assert quant(x=ODD) == -3 and quant(q=P(0x10008)) == -3 and quant(s=P(0x10002)) == -3

    st = F.Tensor(100, A, A, A, None)

    def state(t=st, kind=0, cols=10, q=A, s=A):
        return lib.flashopt_tensor_quantize_rows(ctypes.byref(t) if t is not None else None, kind, cols, q, s, None)
    assert state(t=None) == -1 and state(kind=7) == -4 and state(cols=0) == -2 and state(cols=33) == -2
    assert state(q=None) == -1 and state(s=None) == -1 and state(q=ODD) == -3
    assert state(t=F.Tensor(100, A, None, A, None)) == -1 and state(t=F.Tensor(0, None, None, None, None)) == 0
    assert state(t=F.Tensor(100, A, P(0x10008), A, None)) == -3

    def prod(a=A, sa=A, b=A, sb=A, bias=None, m=4, n=5, k=100, out=A, type=BF16, os=5, ws=A, wsb=1 << 24):
        return lib.flashopt_int8_matmul(a, sa, b, sb, bias, m, n, k, out, type, os, ws, wsb, None)
    assert prod(m=0) == 0 and prod(n=0) == 0 and prod(m=-1) == -2 and prod(k=0) == -2 and prod(k=131073) == -2
    assert prod(m=1 << 24, n=1 << 24, os=1 << 24) == -2
    assert prod(os=4) == -2 and prod(type=3) == -4 and prod(n=(1 << 24) + 1, os=1 << 25) == -2
    assert prod(a=None) == -1 and prod(sa=None) == -1 and prod(b=None) == -1 and prod(sb=None) == -1
    assert prod(out=None) == -1 and prod(a=P(0x10008)) == -3 and prod(b=P(0x10004)) == -3
    assert prod(out=ODD) == -3 and prod(bias=ODD) == -3

    need = lib.flashopt_int8_matmul_workspace_bytes(100, 200, 14336)         # few tiles: cut along the row
    cut = dict(m=100, n=200, k=14336, os=200)
    assert need > 0 and prod(wsb=need - 1, **cut) == -6 and prod(ws=None, **cut) == -1 and prod(ws=P(0x10010), **cut) == -6
    assert lib.flashopt_int8_matmul_workspace_bytes(4, 5, 0) == 0 and lib.flashopt_int8_matmul_workspace_bytes(4, 5, 100) == 0

    def lin(x=A, type=BF16, m=9, k=100, xs=100, w=A, ws=A, bias=None, n=5, out=A, os=5, work=A, wb=1 << 24):
        return lib.flashopt_int8_linear(x, type, m, k, xs, w, ws, bias, n, out, os, work, wb, None)
    assert lin(m=0) == 0 and lin(n=0) == 0 and lin(x=None) == -1 and lin(work=None) == -1 and lin(w=None) == -1
    assert lin(xs=99) == -2 and lin(os=4) == -2 and lin(type=9) == -4 and lin(k=131073, xs=131073) == -2
    assert lin(x=ODD) == -3 and lin(wb=1) == -6 and lin(work=P(0x10010)) == -6
    assert lin(m=1, x=None) == -1 and lin(m=1, w=None) == -1 and lin(m=1, out=None) == -1 and lin(m=1, bias=ODD) == -3
    assert lin(m=1, w=P(0x10008)) == -3 and lin(m=1, ws=P(0x10002)) == -3 and lin(m=1, out=ODD) == -3
    assert lib.flashopt_int8_workspace_bytes(4, 5, 0) == 0 and lib.flashopt_int8_workspace_bytes(9, 5, 100) > 0


def test_overlapping_outputs_are_refused():
    """A gradient that overlaps its logits other than in their place, a layer's output that
    overlaps its input; rows that lie between each other's are no overlap (they then fail later
    validation here: nothing is launched)."""
    lib = F.lib()

    def grads(grad, gs, stride=300, rows=4, up=A):
        yield lib.flashopt_logprob_backward(A, BF16, rows, 100, stride, 1.0, A, A, up, None, grad, gs, None)
        yield lib.flashopt_logprob_grad(A, BF16, rows, 100, stride, 1.0, A, up, None, A, 1 << 20, A, A, grad, gs, None)
        yield lib.flashopt_distill_backward(A, BF16, rows, 100, stride, 1.0, A, A, 4, A, up, grad, gs, None)
        yield lib.flashopt_distill_grad(A, BF16, rows, 100, stride, 1.0, A, A, 4, 1, up, A, 1 << 20, A, grad, gs, None)

    for grad, gs in ((P(0x10000 + 198), 300), (P(0x10000 - 198), 300), (P(0x10000 + 402), 300), (A, 301), (A, 100),
                     (P(0x10000 + 600), 300), (P(0x10000 - 600), 300), (P(0x10000 + 1200), 400)):
        assert set(grads(grad, gs)) == {-4}
    assert set(grads(P(0x10000 + 2), 100, rows=1)) == {-4}

    def lin(out, os=500, m=9, k=100, xs=500, n=50, type=BF16):
        return lib.flashopt_int8_linear(A, type, m, k, xs, P(0x900000), P(0x800000), None, n, out, os,
                                        P(0xA00000), 1 << 24, None)
    for m in (1, 9):
        assert lin(A, m=m) == -4 and lin(P(0x10000 + 198), m=m) == -4 and lin(P(0x10000 - 98), m=m) == -4
        assert lin(P(0x10000 + 100), os=60, m=m) == -4 and lin(P(0x10000 + 396), m=m, type=FP32) == -4
    assert lin(P(0x10000 + 1000 - 98)) == -4


def test_a_frozen_layer_keeps_its_scales():
    layer = I.Int8Linear(I.Int8Weight(torch.zeros((4, 128), dtype=torch.int8), torch.full((4,), 1 / 3), 10), torch.ones(4))
    layer = torch.nn.Sequential(layer).to(torch.bfloat16).half()[0]
    assert torch.equal(layer.scale, torch.full((4,), 1 / 3)) and layer.bias.dtype == torch.float16
    assert layer.codes.dtype == torch.int8 and set(layer.state_dict()) == {"codes", "scale", "bias"}
    with pytest.raises(ValueError):                       # a bias that would want a gradient
        I.int8_linear(torch.zeros(2, 10), I.Int8Weight(layer.codes, layer.scale, 10), torch.zeros(4, requires_grad=True))


def test_python_refusals():
    x = torch.zeros(4, 10)
    t = torch.zeros(4, dtype=torch.int64)
    for bad in (lambda: L.token_logprobs(x, t),                                       # not on a GPU
                lambda: L.token_logprobs(x, t, top=11), lambda: L.token_logprobs(x, t, top=-1),
                lambda: L.token_logprobs(x, t, temperature=0.0), lambda: L.token_logprobs(x, t.int()),
                lambda: L.token_logprobs(x, t[:3]), lambda: L.token_logprobs_grad(x, t, torch.zeros(3)),
                lambda: L.token_logprobs_grad(x, t, torch.zeros(4).double()),
                lambda: L.distill_loss(x, t.view(4, 1), torch.zeros(4, 2)),
                lambda: L.distill_loss(x, torch.zeros(4, 11, dtype=torch.int64), torch.zeros(4, 11)),
                lambda: L.distill_loss(x, t.view(4, 1), torch.zeros(4, 1, requires_grad=True)),
                lambda: L.distill_loss(x, t, torch.zeros(4)),
                lambda: L.distill_grad(x, t.view(4, 1), torch.zeros(4, 1), torch.zeros(5)),
                lambda: F.row_stride(torch.zeros(1, 10).expand(4, 10)), lambda: F.row_stride(x.t()),
                lambda: F.row_stride(torch.zeros(10)), lambda: F.element_type(x.double()),
                lambda: I.Int8Weight(torch.zeros((4, 100), dtype=torch.int8), torch.zeros(4), 100),
                lambda: I.Int8Weight(torch.zeros((4, 128), dtype=torch.int8), torch.zeros(3), 100),
                lambda: I.Int8Weight.from_codes(torch.zeros(4, 8), torch.zeros(4)),
                lambda: I.Int8Weight.from_weight(torch.zeros(4, 8)),
                lambda: I.int8_linear(x, I.Int8Weight(torch.zeros((4, 128), dtype=torch.int8), torch.zeros(4), 11)),
                lambda: I.int8_linear(x, I.Int8Weight(torch.zeros((4, 128), dtype=torch.int8), torch.zeros(4), 10))):
        with pytest.raises(ValueError):
            bad()
