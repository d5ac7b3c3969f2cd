"""Attention operators without a GPU: calls at the ends of what the arguments
allow, and what the sources keep to."""

import ctypes
import os
import re

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


@pytest.mark.parametrize("bad,status", [(dict(), 0), (dict(kv_len=None), 0), (dict(kv_len=None, table_stride=0), 0),
                                        (dict(q=None), 1), (dict(page_size=0), 1), (dict(n_rows=-1), 1)])
def test_batches_without_sequences(sef, bad, status):  # noqa: F811
    """Rows of padding only: the sequences' arrays have no entries, and an empty
    tensor's address is NULL."""
    none = dict(n_seqs=0, kv_len=3 * Args.BASE + 64, page_table=None)
    a = Args(sef, **{**none, **bad})
    assert a.append() == status
    a = Args(sef, **{**none, **bad, "ws": None, "wsb": 0})
    assert a.prompt() == status
    n = ctypes.c_size_t(1)
    if "q" not in bad:
        assert sef.colibri_attention_prompt_workspace(ctypes.byref(a.KV), ctypes.byref(a.SQ), 8,
                                                      ctypes.byref(n)) == status
        assert status or n.value == 0
    assert Args(sef, **{**none, **bad, "scale": 0.0}).prompt() == 1
    single = dict(seq_start=None, n_rows=0, ws=None, wsb=0)
    assert Args(sef, **{**none, **single, **bad}).decode() == status
    # with a sequence they are needed, and packed keys are the call's rows
    for kw in (dict(page_table=None), dict(page_table=None, kv_len=None)):
        assert Args(sef, **kw).append() == 1 and Args(sef, **kw).prompt() == 1


@pytest.mark.parametrize("scale,status", [(2.3e38, 0), (2.4e38, 1), (3.4e38, 1), (1e-45, 0)])
def test_scales_whose_product_with_log2_e_is_finite(sef, scale, status):  # noqa: F811
    """The kernels multiply scores by scale * log2(e): an infinite one would make equal
    scores NaN."""
    assert Args(sef, n_seqs=0, scale=scale).prompt() == status
    assert Args(sef, seq_start=None, n_seqs=0, n_rows=0, scale=scale).decode() == status


def test_waits_are_set_and_the_environment_is_read_once(sef, monkeypatch):  # noqa: F811
    from sparse_expert_ffn_gb300 import attention as A
    assert sef.colibri_attention_waits(5, -1) == 1
    said = []
    monkeypatch.setattr(sef.library(), "colibri_attention_waits", lambda *a: said.append(a) or 0)
    A._pass_on_waits()
    assert said == []
    monkeypatch.setenv("COLIBRI_WAIT_LIMIT_NS", "123")
    A._pass_on_waits(), A._pass_on_waits()
    monkeypatch.setenv("COLIBRI_TEST_STALL_TMA", "2")
    A._pass_on_waits()
    monkeypatch.delenv("COLIBRI_WAIT_LIMIT_NS")
    monkeypatch.delenv("COLIBRI_TEST_STALL_TMA")
    A._pass_on_waits(), A._pass_on_waits()
    assert said == [(123, 0), (123, 2), (0, 0)]
    host = _source("attn_host.cu")
    once = host[host.index("    Waits() {"):]
    assert host.count("getenv") == once[:once.index("    }\n};")].count("getenv") == 2


B = Args.BASE


@pytest.mark.parametrize("o,ok", [(5 * B + 1024, True), (5 * B + 4096 - 1024, True), (5 * B - 1024, True),
                                  (9 * B, True), (5 * B + 512, False), (5 * B + 1008, False), (5 * B, False),
                                  (5 * B + 4096 - 512, False), (5 * B - 512, False), (5 * B + 4096 * 9 + 512, False),
                                  (5 * B + 4096 * 10, True), (2 * B + 64, False), (B - 9 * 4096 - 1024, True),
                                  (B - 16, False)])
def test_outputs_between_the_columns_of_q(sef, o, ok):  # noqa: F811
    """10 rows of q, 1024 bytes each, 4096 bytes apart, the cache at B and 2 B: o may
    lie between q's columns and nowhere in them or in the cache.  No sequences, so that
    an accepted call does nothing, and a workspace, so that only the overlap refuses."""
    kw = dict(q=5 * B, qs=2048, o=o, os=2048)
    assert Args(sef, n_seqs=0, **kw).prompt() == (0 if ok else 1)
    if not ok:
        assert Args(sef, **kw).prompt() == 1                       # (two sequences)
        assert Args(sef, seq_start=None, n_seqs=10, **kw).decode() == 1


@pytest.mark.parametrize("qo,stride,ok", [(5 * B + 2048, 2048, True), (5 * B + 2560, 2048, True), (5 * B, 2048, True),
                                          (9 * B, 512, True), (5 * B + 1024, 2048, False), (5 * B + 16, 2048, False),
                                          (5 * B + 1536, 2048, False), (5 * B + 2048 - 16, 2048, False),
                                          (5 * B + 3088, 2048, False), (5 * B + 2048, 512, False), (5 * B, 512, False),
                                          (B, 512, False), (2 * B + 4096, 512, False), (B - 512, 512, False)])
def test_append_outputs_between_the_columns_of_a_projection(sef, qo, stride, ok):  # noqa: F811
    """q, k and v side by side in rows of 4096 bytes of which they take 2048: q_out may
    be q, or lie in what is left."""
    def call(n_seqs):
        a = Args(sef, q=5 * B, qs=2048, ks=2048, vs=2048, qo=qo, qos=stride, n_seqs=n_seqs)
        a.at.update(k=5 * B + 1024, v=5 * B + 1536)
        return a.append()
    assert call(0) == (0 if ok else 1)
    if not ok:
        assert call(2) == 1


CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_expert_ffn_gb300", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_kernels_read_from_l2_before_they_wait():
    """A kernel that is launched before its predecessor is done is promised other
    grids' writes only once it has waited.  Kernels wait first, or read from L2 only
    (no read-only path, no plain loads of q) what was complete when they started."""
    for name in ("attn_tc.cu", "attn_simt.cu", "rope_append.cu"):
        kernels = re.findall(r"__global__[^{]*\{(.*?)\n\}", _source(name), re.S)
        assert kernels
        for body in kernels:
            before = body[:re.search(r"\n    pdl_enter\(\);", body).start()]
            reads = r"__ldg|attn_seq|attn_item|work_item|row_place|load\(|simt_tile" \
                r"|\ba\.(q|k|v|o|lse|seq_start|kv_len|table|freq|q_norm|k_norm|q_out|k_out|v_out|part_\w+|piece_\w+)\b"
            assert not re.search(reads, before), name
    for name in ("attn_decode.cu", "attn_join.cu"):
        text = _source(name)
        calls = re.findall(r"\b(?:attn_seq|attn_page|seq_steps|count_steps|ld_early)\b(<[^>]*>)?", text)
        assert calls and all(c.endswith("kEarly>") for c in calls) and "__ldg" not in text, name
    # the kernels of kEarly and not: who waits first may read through L1
    assert "if constexpr (kEarly) pdl_launch_dependents();\n    else pdl_enter();\n    decode_share<Rows, kEarly>" in \
        _source("attn_decode.cu")
    join = re.sub(r"\s+", " ", _source("attn_join.cu"))
    assert "if (!early) pdl_enter(); if (warp == 0) { const Place p = early ? row_parts<T, D, true>" in join
    assert ": row_parts<T, D, false>" in join and "} if (early) pdl_enter(); __syncthreads();" in join
    common = _source("attn_common.cuh")
    for name in ("AttnSeq attn_seq", "int attn_page"):
        body = common[common.index(name):]
        assert "ld_early<kEarly>" in body[:body.index("\n}")], name
    assert "return kEarly ? __ldcg(p) : __ldg(p);" in common
