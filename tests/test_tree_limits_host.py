"""Limits of the tree attention's lengths, without a GPU."""
import ctypes

import pytest

from self_speculative_sparse_gb300 import binding as vb
from tests.test_tree_host import attn_call, dims, lib  # noqa: F401


@pytest.mark.parametrize("max_len", [2 ** 31 - 1, 2 ** 31 - 64, 2 ** 31 - 2048])
def test_lengths_that_31_bits_do_not_hold_are_refused(lib, max_len):  # noqa: F811
    """(Their scratch's size would not be a number of 32 bits.)"""
    d = dims(B=1, H_q=1, H_kv=1, max_len=max_len)
    assert attn_call(lib, d=d, n=16, stride=1 << 31) == vb.VG_ERR_UNSUPPORTED_SHAPE
    assert "max_len" in lib.vg_last_error().decode()
    assert lib.vg_tree_verify_workspace_size(ctypes.byref(d), 16) == 0 and "max_len" in lib.vg_last_error().decode()
