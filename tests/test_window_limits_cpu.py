"""Sizes whose whole tiles no longer fit an int: refused on the host, before any CUDA call."""

import ctypes

import pytest

from tests._lib import built_lib

P = ctypes.c_void_p(0x1000)  # never dereferenced


@pytest.mark.parametrize("S,cp", [(1 << 24, 1 << 23), (1 << 25, 1 << 23), (3 << 23, 3 << 22)])
def test_many_short_chunks_are_refused(S, cp):
    lib = built_lib()
    n = ctypes.c_size_t(0)
    args = (1, 1, 1, S, 64, cp, 1, 4, 0)
    assert lib.cp_attn_fwd_window(*[P] * 5, *args, None) == -2 and b"chunks" in lib.cp_attn_last_error()
    assert lib.cp_attn_bwd_window(*[P] * 9, *args, P, 1 << 40, None) == -2
    assert lib.cp_attn_bwd_window_workspace(*args, ctypes.byref(n), None) == -2

