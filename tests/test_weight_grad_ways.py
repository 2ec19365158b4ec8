"""The sizes that the weight gradients are tested at take the ways that they are meant to (grad_ways.py)."""
import pytest

import grad_ways as W
from compressed_adamw_state_amd import flashopt as F

CASES = [(kind, way, *s) for kind, ways in W.SIZES.items() for way, sizes in ways.items() for s in sizes]


@pytest.mark.parametrize("kind,way,m,n,k", CASES)
def test_a_size_takes_its_way(kind, way, m, n, k):
    got, size = W.way_of(kind, m, n, k)
    assert got == way
    for type in ((2,) if kind == "32" else (0, 1)):                # what the rule says is what the library does
        assert F.lib().flashopt_held_weight_grad_workspace_bytes(type, m, n, k) == size


def test_every_way_has_a_size():
    for kind, cuts in (("16", ("whole", "cut", "mixed")), ("32", ("whole", "cut"))):
        want = {(way, cut) for way in ("teams", "small", "large") for cut in cuts if cut != "mixed" or way == "large"}
        assert set(W.SIZES[kind]) == want


def test_the_largest_products_are_mixed():
    assert W.way_of("16", 8192, 14336, 4096)[0] == ("large", "mixed")
