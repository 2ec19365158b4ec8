"""Outputs that overlap what a call reads are refused before anything is launched (include/flashopt_lm.h):
held arrays, weights, tables and ids, not only matrices of the same kind.  Every call here fails that check;
the addresses are never dereferenced."""
import ctypes

import pytest

from compressed_adamw_state_amd import flashopt as F

P = ctypes.c_void_p
A, B, C, D = 0x10000000, 0x20000000, 0x30000000, 0x40000000
BF16, FP32 = 0, 2
ARG = -4


def both_ends(start, size, step, own):
    """Addresses (multiples of step) of `own` bytes that reach into start .. start + size by one step at
    either end, and inside."""
    return [start - own + step, start + size - step, start + size // 2 // step * step]


# 4 rows of 100 BF16 values: 4 x 128 codes, 4 x 4 bytes of powers
@pytest.mark.parametrize("x", both_ends(B, 512, 2, 800) + [C - 798, C + 14])
def test_hold(x):
    assert F.lib().flashopt_hold(P(x), BF16, 4, 100, 100, P(B), P(C), None) == ARG


@pytest.mark.parametrize("out", both_ends(B, 512, 4, 1600) + [C - 1596, C + 12])
def test_held_values(out):
    assert F.lib().flashopt_held_values(P(B), P(C), 4, 100, P(out), FP32, 100, None) == ARG


# m = 9 tokens, n = 20, k = 30: 9 x 128 codes, 9 x 4 powers, 20 x 30 weights, 20 bias
@pytest.mark.parametrize("w", both_ends(B, 1152, 2, 1200) + [C - 1198, C + 34])
def test_weight_gradient(w):
    assert F.lib().flashopt_held_weight_grad(P(A), BF16, 9, 20, 20, P(B), P(C), 30, P(w), 30, None, None, 0, None) == ARG


@pytest.mark.parametrize("b", both_ends(B, 1152, 2, 40) + [C - 38, C + 34] + both_ends(A, 360, 2, 40) + both_ends(D, 1200, 2, 40))
def test_bias_gradient(b):
    assert F.lib().flashopt_held_weight_grad(P(A), BF16, 9, 20, 20, P(B), P(C), 30, P(D), 30, P(b), None, 0, None) == ARG


def test_rows_between_others_are_told_apart():
    """A wide matrix's rows with codes over one of them."""
    for row in range(4):
        assert F.lib().flashopt_hold(P(A), BF16, 4, 100, 1 << 20, P(A + row * (1 << 21) + 192), P(C), None) == ARG


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("over", [A, B, C])                        # gate, up, y
def test_gated_held_arrays(which, over):
    held = [D, D + 0x1000, D + 0x2000, D + 0x3000]
    for at in (over, over + 784):
        held[which] = at
        assert F.lib().flashopt_gated(P(A), P(B), BF16, 0, 4, 100, 100, 100, P(C), 100, *map(P, held), None) == ARG


@pytest.mark.parametrize("which", range(4))
def test_gated_held_arrays_without_an_output(which):
    held = [D, D + 0x1000, D + 0x2000, D + 0x3000]
    held[which] = A + 784
    assert F.lib().flashopt_gated(P(A), P(B), BF16, 0, 4, 100, 100, 100, None, 0, *map(P, held), None) == ARG


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("second", [False, True])
def test_gated_backward(which, second):
    held = [D, D + 0x1000, D + 0x2000, D + 0x3000]
    size = (512, 16)[which % 2]
    for out in (held[which] - 798, held[which] + size - 2):
        dg, du = (C, out) if second else (out, C)
        assert F.lib().flashopt_gated_backward(P(A), BF16, 1, 4, 100, 100, *map(P, held), P(dg), 100, P(du), 100, None) == ARG


# 5 ids, a table of 10 x 20: 10 x 128 codes, 10 scales, 5 x 20 outputs
@pytest.mark.parametrize("out", both_ends(A, 40, 2, 200) + both_ends(B, 1280, 2, 200) + both_ends(C, 40, 2, 200))
def test_embedding_int8(out):
    assert F.lib().flashopt_embedding_int8(P(A), 5, P(B), P(C), 10, 20, 1.0, P(out), BF16, 20, None) == ARG


@pytest.mark.parametrize("out", both_ends(A, 40, 2, 200))
def test_embedding_ids(out):
    assert F.lib().flashopt_embedding(P(A), 5, P(B), BF16, 10, 20, 20, 1.0, P(out), 20, None) == ARG


@pytest.mark.parametrize("grad", both_ends(A, 40, 2, 400))
def test_embedding_backward_ids(grad):
    need = F.lib().flashopt_embedding_workspace_bytes(5, 10, 20)
    assert F.lib().flashopt_embedding_backward(P(A), 5, P(B), BF16, 20, 10, 20, 1.0, P(C), need, P(grad), 20, None) == ARG
