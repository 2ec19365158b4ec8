"""Forward-mode differentiation: the language-model operators have none, so a tensor that carries a
tangent is refused, with and without gradients enabled, and not taken as a plain one (whose results
would silently lack their tangent)."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

from compressed_adamw_state_amd import int8 as I
from compressed_adamw_state_amd import losses as L


def calls(x, up, t, w, device):
    """name, call of one dual tensor"""
    ids = torch.zeros(4, 1, dtype=torch.int64, device=device)
    tlp = torch.full((4, 1), -0.5, device=device)

    def dual(v):
        return fwd.make_dual(v, torch.ones_like(v))
    yield "logits", lambda: L.token_logprobs(dual(x), t)
    yield "logits", lambda: L.token_logprobs(dual(x).reshape(2, 2, -1), top=2)
    yield "logits", lambda: L.token_logprobs_grad(dual(x), t, up)
    yield "grad_logprob", lambda: L.token_logprobs_grad(x, t, dual(up))
    yield "grad_entropy", lambda: L.token_logprobs_grad(x, t, up, dual(up))
    yield "logits", lambda: L.distill_loss(dual(x), ids, tlp)
    yield "top_logprob", lambda: L.distill_loss(x, ids, dual(tlp))
    yield "logits", lambda: L.distill_grad(dual(x), ids, tlp, up)
    yield "grad_loss", lambda: L.distill_grad(x, ids, tlp, dual(up))
    yield "x", lambda: I.int8_linear(dual(x), w)
    yield "bias", lambda: I.int8_linear(x, w, dual(torch.zeros(3, device=device)))
    leaf = x.clone().requires_grad_()
    yield "logits", lambda: L.token_logprobs(dual(leaf), t)


def refused(device, w):
    x, up = torch.randn(4, 10, device=device), torch.ones(4, device=device)
    t = torch.zeros(4, dtype=torch.int64, device=device)
    with fwd.dual_level():
        for name, call in calls(x, up, t, w, device):
            for mode in (torch.enable_grad, torch.no_grad):
                with mode(), pytest.raises(ValueError, match=f"{name} has a forward-mode tangent"):
                    call()


def test_tangents_are_refused():
    refused("cpu", I.Int8Weight(torch.zeros((3, 128), dtype=torch.int8), torch.zeros(3), 10))


@pytest.mark.gpu
def test_tangents_are_refused_on_the_gpu():
    w = I.Int8Weight.from_weight(torch.randn(3, 10).cuda())
    refused("cuda", w)
    x = torch.randn(4, 10, device="cuda")
    with fwd.dual_level():                                 # a plain tensor is taken
        assert torch.equal(I.int8_linear(x, w), I.int8_linear(x.clone(), w))
        assert L.token_logprobs(x, top=1).top_id.shape == (4, 1)
