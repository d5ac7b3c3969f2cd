"""The 8-bit cache without a GPU: the oracle's pins, the axis maps, and every refusal of
the C entry points (before any CUDA call)."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import attention as oa


@pytest.fixture(scope="module")
def sef():
    from sparse_expert_ffn_gb300 import build
    build.build()
    import sparse_expert_ffn_gb300
    return sparse_expert_ffn_gb300


def test_oracle_codes():
    """Against torch's conversions, all codes and the middles between them."""
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double().numpy()
    every = np.sort(every[np.isfinite(every)])
    assert np.array_equal(oa.nearest_code(every, "e4m3"), every)
    mid = (every[1:] + every[:-1]) / 2
    for y in (mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)):
        want = torch.from_numpy(y).float().to(torch.float8_e4m3fn).float().double().numpy()
        assert np.array_equal(oa.nearest_code(y, "e4m3"), want)
    assert oa.nearest_code([0.5, 1.5, -2.5, 126.6], "int8").tolist() == [0.0, 2.0, -2.0, 127.0]
    for code, most in oa.CODE_MOST.items():
        assert oa.fitting_scale(most, code) == 1.0 and oa.fitting_scale(most * 1.0001, code) == 2.0
        assert oa.fitting_scale(0.0, code) == 2.0 ** -100


def test_oracle_positions_per_pair():
    rng = np.random.default_rng(0)
    x, f = rng.standard_normal((4, 2, 16)), oa.rope_frequencies(16)[0]
    same = oa.norm_rotate(x, np.repeat(np.arange(4)[:, None], 8, 1), f)
    assert np.allclose(same, oa.norm_rotate(x, np.arange(4), f))
    pos = np.zeros((4, 8))
    pos[:, 3] = 5
    y = oa.norm_rotate(x, pos, f)
    still = [i for i in range(16) if i % 8 != 3]
    assert np.array_equal(y[..., still], x[..., still])
    z = (x[..., 3] + 1j * x[..., 11]) * np.exp(5j * f[3])
    assert np.allclose(y[..., 3], z.real) and np.allclose(y[..., 11], z.imag)


def test_rope_axes(sef):
    from sparse_expert_ffn_gb300 import attention as A
    assert A.rope_axes([2, 3, 1]).tolist() == [0, 0, 1, 1, 1, 2]
    assert A.rope_axes([2, 3, 1], interleaved=True).tolist() == [0, 1, 2, 0, 1, 1]
    assert A.rope_axes([4]).tolist() == [0] * 4 and A.rope_axes([0, 2]).tolist() == [1, 1]
    for bad in ([], [1] * 9, [3, -1]):
        with pytest.raises(ValueError):
            A.rope_axes(bad)


class Args:
    """Well-formed arguments over host memory (never dereferenced by a check)."""

    BASE = 1 << 20

    def __init__(self, sef, **bad):
        self.sef, P = sef, self.BASE
        self.kv = dict(k=P, v=2 * P, k_scale=13 * P, v_scale=14 * P, page_stride=4 * 32 * 64, head_stride=32 * 64,
                       row_stride=64, num_pages=8, page_size=32, n_kv_heads=4, head_dim=64, code=0, block=16)
        self.sq = dict(seq_start=3 * P, kv_len=3 * P + 64, page_table=3 * P + 128, n_seqs=2, n_rows=10, table_stride=4)
        self.rope = dict(freq=4 * P, rot_dim=64, style=0, mscale=1.0)
        self.ps = dict(at=4 * P + 4096, axis=4 * P + 8192, axis_stride=10, n_axes=3)
        self.a = dict(hq=8, q=5 * P, qs=512, kr=6 * P, ks=256, vr=7 * P, vs=256, qn=8 * P, kn=8 * P + 256, eps=1e-6,
                      qo=9 * P, qos=512, scale=0.125, o=11 * P, os=512, lse=12 * P, ws=32 * P, wsb=1 << 40, prefix=0,
                      pt=None, pages=15 * P, n_pages=3, ko=20 * P, vo=24 * P, dtype=1)
        for name, v in bad.items():
            next(d for d in (self.kv, self.sq, self.rope, self.ps, self.a) if name in d)[name] = v
        self.C = sef.ColibriKVPages8(**self.kv)
        self.SQ, self.RP, self.PS = sef.ColibriSeqs(**self.sq), sef.ColibriRope(**self.rope), sef.ColibriPositions(**self.ps)

    def append(self, cache=True, rope=True, positions=True):
        a, r = self.a, ctypes.byref
        return self.sef.colibri_append_qkv8(r(self.C) if cache else None, r(self.SQ), r(self.RP) if rope else None,
                                            r(self.PS) if positions else None, a["hq"], a["q"], a["qs"], a["kr"], a["ks"],
                                            a["vr"], a["vs"], a["qn"], a["kn"], a["eps"], a["qo"], a["qos"], None)

    def append16(self):
        a, r = self.a, ctypes.byref
        kv = self.sef.ColibriKVPages(self.BASE, 2 * self.BASE, 4 * 32 * 64, 32 * 64, 64, 8, 32, 4, 64, a["dtype"])
        return self.sef.colibri_append_qkv_at(r(kv), r(self.SQ), r(self.RP), r(self.PS), a["hq"], a["q"], a["qs"], a["kr"],
                                              a["ks"], a["vr"], a["vs"], a["qn"], a["kn"], a["eps"], a["qo"], a["qos"], None)

    def rotate(self, rope=True):
        a, r = self.a, ctypes.byref
        return self.sef.colibri_qk_norm_rope_at(r(self.SQ), r(self.RP) if rope else None, r(self.PS), a["hq"], 4, 64, 1,
                                                a["q"], a["qs"], a["kr"], a["ks"], a["qn"], a["kn"], a["eps"], a["qo"],
                                                a["qos"], a["ko"], 256, None)

    def values(self):
        a = self.a
        return self.sef.colibri_values8(ctypes.byref(self.C), a["pages"], a["n_pages"], a["ko"], a["vo"], None)

    def prompt(self):
        a, r = self.a, ctypes.byref
        return self.sef.colibri_attention_prompt8(r(self.C), r(self.SQ), a["hq"], a["q"], a["qs"], a["scale"], 1, a["o"],
                                                  a["os"], a["lse"], a["ws"], a["wsb"], None)

    def decode(self):
        a, r = self.a, ctypes.byref
        return self.sef.colibri_attention_decode8(r(self.C), r(self.SQ), a["hq"], a["q"], a["qs"], a["scale"], a["prefix"],
                                                  a["pt"], a["o"], a["os"], a["lse"], a["ws"], a["wsb"], None)


B = Args.BASE
KV_BAD = [(dict(k=None), 1), (dict(v=8), 1), (dict(k_scale=None), 1), (dict(v_scale=14 * B + 2), 1), (dict(row_stride=72), 1),
          (dict(row_stride=48), 1), (dict(head_stride=8), 1), (dict(page_stride=-64), 1), (dict(num_pages=0), 1),
          (dict(page_size=0), 1), (dict(page_size=8), 4), (dict(page_size=48), 4), (dict(page_size=1 << 17), 4),
          (dict(head_dim=96), 4), (dict(n_kv_heads=0), 1), (dict(code=2), 1), (dict(code=-1), 1), (dict(block=0), 1),
          (dict(block=8), 4), (dict(block=64), 4), (dict(block=24), 4)]
SQ_BAD = [(dict(n_seqs=-1), 1), (dict(n_rows=-1), 1), (dict(kv_len=None), 1), (dict(table_stride=0), 1),
          (dict(n_rows=1 << 29), 1), (dict(hq=0), 1), (dict(hq=6), 1), (dict(page_table=None), 1)]


@pytest.mark.parametrize("bad,status", KV_BAD + SQ_BAD + [
    (dict(q=None), 1), (dict(q=8), 1), (dict(qs=504), 1), (dict(ks=128), 1), (dict(vs=260), 1), (dict(qn=2), 1),
    (dict(eps=-1.0), 1), (dict(qo=None), 1), (dict(qo=6 * B), 1), (dict(qo=B), 1), (dict(q=13 * B), 1), (dict(qo=14 * B), 1),
    (dict(vr=14 * B - 256), 1), (dict(v_scale=13 * B), 1), (dict(k_scale=2 * B + 1024), 1), (dict(rot_dim=72), 1), (dict(freq=None), 1), (dict(at=None), 1), (dict(at=4 * B + 2), 1),
    (dict(n_axes=0), 1), (dict(n_axes=9), 1), (dict(axis_stride=-1), 1), (dict(n_rows=0), 0), (dict(n_seqs=0), 0)])
def test_append8_refusals(sef, bad, status):
    a = Args(sef, **bad)
    assert a.append() == status
    if status and not set(bad) & {*a.ps, "qn"}:
        assert a.append(positions=False) == status
    assert Args(sef).append(cache=False) == 1 and Args(sef).append(rope=False) == 1


@pytest.mark.parametrize("bad,status", [
    (dict(at=None), 1), (dict(at=4 * B + 2), 1), (dict(n_axes=0), 1), (dict(n_axes=9), 1), (dict(axis_stride=1 << 40), 1),
    (dict(axis_stride=-1), 1), (dict(rot_dim=8), 1), (dict(n_rows=0), 0), (dict(n_seqs=0), 0)])
def test_positions_refusals(sef, bad, status):
    assert Args(sef, **bad).append16() == status and Args(sef, **bad).rotate() == status
    assert Args(sef).rotate(rope=False) == 1


@pytest.mark.parametrize("bad,status", KV_BAD + [
    (dict(n_pages=-1), 1), (dict(pages=15 * B + 1), 1), (dict(pages=None, n_pages=9), 1), (dict(ko=None), 1), (dict(vo=8), 1),
    (dict(ko=20 * B, vo=20 * B + 4096), 1), (dict(ko=B), 1), (dict(vo=2 * B + 4096), 1), (dict(ko=13 * B), 1),
    (dict(n_pages=1 << 30), 4), (dict(n_pages=0), 0), (dict(n_pages=0, ko=None, vo=None), 0)])
def test_values8_refusals(sef, bad, status):
    assert Args(sef, **bad).values() == status


ATTN_BAD = [(dict(q=None), 1), (dict(q=8), 1), (dict(qs=504), 1), (dict(os=500), 1), (dict(o=None), 1), (dict(o=5 * B), 1),
            (dict(o=B + 256), 1), (dict(o=13 * B), 1), (dict(o=14 * B), 1), (dict(lse=2), 1), (dict(scale=0.0), 1),
            (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(hq=4 * 129, qs=1 << 16, os=1 << 16), 4)]


@pytest.mark.parametrize("bad,status", KV_BAD + SQ_BAD + ATTN_BAD + [
    (dict(seq_start=None), 1), (dict(n_rows=0), 0), (dict(n_seqs=0), 0)])
def test_prompt8_refusals(sef, bad, status):
    assert Args(sef, **bad).prompt() == status


@pytest.mark.parametrize("bad,status", KV_BAD + SQ_BAD + ATTN_BAD + [
    (dict(seq_start=3 * B), 1), (dict(n_rows=9), 1), (dict(prefix=-32), 1), (dict(prefix=48, pt=16 * B), 1),
    (dict(prefix=32, pt=None), 1), (dict(prefix=0, pt=16 * B), 1), (dict(prefix=32, pt=16 * B + 2), 1),
    (dict(n_rows=0, n_seqs=0), 0)])
def test_decode8_refusals(sef, bad, status):
    assert Args(sef, **{**dict(seq_start=None, n_seqs=10), **bad}).decode() == status


def test_workspace8_is_checked(sef):
    a, n = Args(sef, seq_start=None, n_seqs=2, n_rows=2, table_stride=2048), ctypes.c_size_t()
    r = ctypes.byref
    assert sef.colibri_attention_decode8_workspace(r(a.C), r(a.SQ), 8, 0, r(n)) == 0 and n.value > 0
    kw = dict(seq_start=None, n_seqs=2, n_rows=2, table_stride=2048)
    assert Args(sef, **kw, ws=None).decode() == 1
    assert Args(sef, **kw, wsb=n.value - 1).decode() == 1
    assert Args(sef, **kw, ws=32 * B + 128).decode() == 1
    a = Args(sef, table_stride=2048)
    assert sef.colibri_attention_prompt8_workspace(r(a.C), r(a.SQ), 8, r(n)) == 0
    if n.value:
        assert Args(sef, table_stride=2048, ws=None).prompt() == 1
        assert Args(sef, table_stride=2048, wsb=n.value - 1).prompt() == 1
    for name, args in (("prompt8", ()), ("decode8", (0,))):
        assert getattr(sef, f"colibri_attention_{name}_workspace")(r(a.C), r(a.SQ), 8, *args, None) == 1


def test_the_frame_of_single_rows_reads_from_l2_before_it_waits():
    """What tests/test_attn_host_calls.py asks of the kernels for single rows, of the
    headers that they are made of."""
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_expert_ffn_gb300", "csrc")
    for name in ("attn_share.cuh", "attn_rows8.cuh"):
        with open(os.path.join(csrc, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        calls = re.findall(r"\b(?:attn_seq|attn_page|seq_steps|seq_tiles|seq_items|count_steps|ld_early)\b(<[^>]*>)", text)
        assert calls and all(c.endswith("kEarly>") for c in calls) and "__ldg" not in text, name
    with open(os.path.join(csrc, "append8.cu")) as f:
        for body in re.findall(r"__global__[^{]*\{(.*?)\n\}", f.read(), re.S):
            assert not re.search(r"__ldg|find_span|\ba\.(q|k|v|table|kv_len)\b", body[:body.index("pdl_enter();")])


@pytest.mark.parametrize("dtype", range(-20, 0))
def test_no_number_stands_for_codes_in_calls_of_16_bits(sef, dtype):
    r, n = ctypes.byref, ctypes.c_size_t()
    a = Args(sef, dtype=dtype)
    kv = sef.ColibriKVPages(B, 2 * B, 4 * 32 * 64, 32 * 64, 64, 8, 32, 4, 64, dtype)
    single = sef.ColibriSeqs(None, 3 * B + 64, 3 * B + 128, 10, 10, 4)
    assert a.append16() == 1
    assert sef.colibri_attention_prompt_workspace(r(kv), r(a.SQ), 8, r(n)) == 1
    assert sef.colibri_attention_decode_workspace(r(kv), r(single), 8, 0, r(n)) == 1
    args = (8, 5 * B, 512, 0.125)
    assert sef.colibri_attention_prompt(r(kv), r(a.SQ), *args, 1, 11 * B, 512, None, 32 * B, 1 << 40, None) == 1
    assert sef.colibri_attention_decode(r(kv), r(single), *args, 0, None, 11 * B, 512, None, 32 * B, 1 << 40, None) == 1
