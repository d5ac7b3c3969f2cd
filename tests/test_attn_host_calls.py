"""Attention operators without a GPU: calls at the ends of what the arguments
allow, and what the sources keep to."""

import ctypes

import pytest

from test_attn_host import Args, sef  # noqa: F401


@pytest.mark.parametrize("prefix,status", [(0x7ff00000, 0), (0x7ff00000 + 16, 4), (0x7ffffff0, 4)])
def test_prefixes_end_where_positions_fit(sef, prefix, status):  # noqa: F811
    """A page may be named again and again, so a small cache can stand for a prefix
    of any length: one whose last tile would pass 2^31 - 1 is refused."""
    a = Args(sef, seq_start=None, n_rows=0, n_seqs=0, prefix=prefix, pt=13 * Args.BASE)
    assert a.decode() == status
    n = ctypes.c_size_t()
    assert sef.colibri_attention_decode_workspace(ctypes.byref(a.KV), ctypes.byref(a.SQ), 8, prefix,
                                                  ctypes.byref(n)) == status
