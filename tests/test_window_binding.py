"""The binding's own arithmetic for windows and sinks."""

import pytest

from context_causal_attention_load_gb300 import cpattn


@pytest.mark.parametrize("n", [-1, -2 ** 31 - 1, -2 ** 32 + 5, -2 ** 32, -2 ** 40])
def test_counts_below_zero_stay_below_zero(n):
    """(a C int of their low 32 bits would be a window of 5, or no sinks)"""
    assert cpattn._count(n) == -1


@pytest.mark.parametrize("n,c", [(0, 0), (1, 1), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1)])
def test_counts(n, c):
    assert cpattn._count(n) == c
