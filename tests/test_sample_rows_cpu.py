"""Sizes of sampling calls of very many rows, without a GPU."""
from __future__ import annotations

import ctypes

import pytest

import bit_weight_only_packed_amd as Q


@pytest.mark.parametrize("vocab", [16385, 65536])
def test_a_workgroup_takes_a_row_however_many_there_are(vocab):
    """From 256 rows on up to 65,536 tokens need no workspace to speak of; 256 times the rows may pass 2^31."""
    n = ctypes.c_size_t()
    for rows in (256, 1 << 22, (1 << 23) - 1, 1 << 23, 1 << 24, (1 << 31) - 1):
        assert Q.lib().qgs_sample_workspace(rows, vocab, ctypes.byref(n)) == Q.QG_OK
        assert n.value == 16, rows


def test_the_workspace_does_not_grow_past_a_launch():
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    for vocab in (65537, 131071, 1 << 20):
        Q.lib().qgs_sample_workspace(1 << 14, vocab, ctypes.byref(a))
        Q.lib().qgs_sample_workspace((1 << 31) - 1, vocab, ctypes.byref(b))
        assert a.value == b.value
