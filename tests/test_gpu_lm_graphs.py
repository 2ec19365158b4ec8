"""The language-model operators beside torch's automatic differentiation: a tensor that a call
overwrites counts as modified, one that a refused call left alone does not, and what the operators
cannot differentiate they refuse."""
import pytest
import torch

from compressed_adamw_state_amd import flashopt as F
from compressed_adamw_state_amd import int8 as I
from compressed_adamw_state_amd import losses as L

pytestmark = pytest.mark.gpu


def layer(n, k, device="cuda"):
    return I.Int8Weight.from_weight(torch.randn(n, k, generator=torch.Generator().manual_seed(1)).to(device))


@pytest.mark.parametrize("m", [1, 40])
def test_an_output_given_counts_as_modified(m):
    w, x = layer(32, 64), torch.randn(m, 64, device="cuda")
    y = torch.randn(m, 32, device="cuda", requires_grad=True) * 1.0
    s = (y * y).sum()                                      # keeps y for its backward pass
    with torch.no_grad():
        I.int8_linear(x, w, out=y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        s.backward()
    base = torch.randn(2, m, 32, device="cuda", requires_grad=True) * 1.0
    s = (base * base).sum()
    I.int8_linear(x, w, out=base.detach()[1])              # a view of the same storage
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        s.backward()


def test_an_output_with_a_gradient_is_refused():
    w, x = layer(32, 64), torch.randn(4, 64, device="cuda")
    y = torch.zeros(4, 32, device="cuda", requires_grad=True)
    with pytest.raises(ValueError, match="out requires a gradient"):
        I.int8_linear(x, w, out=y)
    with torch.no_grad():
        I.int8_linear(x, w, out=y)
    assert torch.equal(y.detach(), I.int8_linear(x, w))


def test_a_refused_output_stays_as_it_was():
    w = layer(100, 200)
    both = torch.randn(6, 400, device="cuda", requires_grad=True) * 1.0
    s = (both * both).sum()
    with pytest.raises(F.FlashoptError):                   # the output lies over the input
        I.int8_linear(both.detach()[:, :200], w, out=both.detach()[:, 150:250])
    s.backward()


def test_a_refused_gradient_in_place_leaves_the_logits_usable():
    """A vocabulary past the limit: the logits were not replaced, and what saved them still has them."""
    y = torch.randn(1, F.lib().flashopt_int8_ld(131072) * 4 + 1, device="cuda", requires_grad=True) * 1.0
    s = (y * y).sum()
    one, t = torch.ones(1, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    with pytest.raises(F.FlashoptError):
        L.token_logprobs_grad(y, t, one, inplace=True)
    with pytest.raises(F.FlashoptError):
        L.distill_grad(y, t.view(1, 1), -one.view(1, 1), one, inplace=True)
    s.backward()
