"""Attention operators without a GPU: the oracle's pins, the frequencies, and
every refusal of the C entry points (before any CUDA call)."""

import ctypes
import math

import numpy as np
import pytest

from oracle import attention as oa


@pytest.fixture(scope="module")
def sef():
    from sparse_expert_ffn_gb300 import build
    build.build()
    import sparse_expert_ffn_gb300
    return sparse_expert_ffn_gb300


# ------------------------------------------------------------ oracle pins

def test_oracle_attention_closed_forms():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    o, lse, _ = oa.attend(np.zeros((3, 4, 8)), k, v, [9, 4, 0], 0.3)
    assert np.allclose(o[0, 1], v[:, 0].mean(0)) and np.allclose(o[1, 2], v[:4, 1].mean(0))
    assert np.allclose(lse[0], math.log(9)) and (o[2] == 0).all() and np.isneginf(lse[2]).all()
    q = rng.standard_normal((1, 2, 8))
    o1, lse1, _ = oa.attend(q, k, v, [1], 0.5)
    assert np.allclose(o1[0], v[0]) and np.allclose(lse1[0], 0.5 * (q[0] * k[0]).sum(-1))
    # two key ranges joined by their log-sums
    qa = rng.standard_normal((2, 2, 8))
    full = oa.attend(qa, k, v, [9, 9], 0.7)
    a, b = oa.attend(qa, k[:5], v[:5], [5, 5], 0.7), oa.attend(qa, k[5:], v[5:], [4, 4], 0.7)
    w = 1 / (1 + np.exp(b[1] - a[1]))
    assert np.allclose(w[..., None] * a[0] + (1 - w)[..., None] * b[0], full[0])


@pytest.mark.parametrize("style", ["half", "interleaved"])
def test_oracle_rotation_properties(style):
    rng = np.random.default_rng(1)
    f, _ = oa.rope_frequencies(16, 100.0)
    q, k = rng.standard_normal((1, 1, 24)), rng.standard_normal((1, 1, 24))
    r = [oa.norm_rotate(x, [t], f, style) for x, t in ((q, 11), (k, 4))]
    s = [oa.norm_rotate(x, [t], f, style) for x, t in ((q, 1007), (k, 1000))]
    assert np.allclose((r[0] * r[1]).sum(), (s[0] * s[1]).sum())       # only the distance counts
    assert np.allclose(np.linalg.norm(r[0]), np.linalg.norm(q))
    assert np.array_equal(r[0][..., 16:], q[..., 16:])
    assert np.array_equal(oa.norm_rotate(q, [0], f, style), q)
    # by hand, position 1, first pair: angle f_0 = 1
    a, b = (q[0, 0, 0], q[0, 0, 8]) if style == "half" else (q[0, 0, 0], q[0, 0, 1])
    y = oa.norm_rotate(q, [1], f, style)[0, 0]
    assert np.isclose(y[0], a * math.cos(1) - b * math.sin(1))
    assert np.isclose(y[8 if style == "half" else 1], b * math.cos(1) + a * math.sin(1))
    n = oa.norm_rotate(q, [3], None, style, weight=np.full(24, 2.0), eps=0.0)
    assert np.isclose((n ** 2).mean(), 4.0)


# ------------------------------------------------------------ frequencies

@pytest.mark.parametrize("rot", [16, 48, 128])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0),
                                            ("yarn", 1.0)])
def test_rope_frequencies_match_the_formula(sef, rot, scaling, factor):
    from sparse_expert_ffn_gb300 import attention as A
    got, ms = A.rope_frequencies(rot, 10000.0, scaling, factor, trained=2048)
    want, wms = oa.rope_frequencies(rot, 10000.0, scaling, factor, trained=2048)
    # powers and logarithms are good to a few units of 2^-52
    assert np.allclose(got.numpy(), want, rtol=2.0 ** -46, atol=0) and abs(ms - wms) <= 2.0 ** -24 * wms
    if scaling == "yarn":
        plain, _ = oa.rope_frequencies(rot)
        assert np.isclose(got[0].item(), plain[0]) and got[-1].item() <= plain[-1] / factor * (1 + 1e-12)


def test_rope_frequencies_refusals(sef):
    f, m = (ctypes.c_double * 64)(), ctypes.c_float()
    call = lambda *a: sef.colibri_rope_frequencies(*a, ctypes.cast(f, ctypes.c_void_p), ctypes.byref(m))  # noqa: E731
    assert call(64, 1e4, 0, 1.0, 4096, 32.0, 1.0) == 0
    for bad in [(0, 1e4, 0, 1.0, 4096, 32.0, 1.0), (24, 1e4, 0, 1.0, 4096, 32.0, 1.0), (64, 1.0, 0, 1.0, 4096, 32.0, 1.0),
                (64, float("nan"), 0, 1.0, 4096, 32.0, 1.0), (64, 1e4, 4, 1.0, 4096, 32.0, 1.0),
                (64, 1e4, 1, 0.5, 4096, 32.0, 1.0), (64, 1e4, 2, float("inf"), 4096, 32.0, 1.0),
                (64, 1e4, 3, 2.0, 0, 32.0, 1.0), (64, 1e4, 3, 2.0, 4096, 1.0, 1.0), (64, 1e4, 3, 2.0, 4096, 32.0, 0.0)]:
        assert call(*bad) == 1, bad
    assert sef.colibri_rope_frequencies(64, 1e4, 0, 1.0, 4096, 32.0, 1.0, None, ctypes.byref(m)) == 1
    assert sef.colibri_rope_frequencies(64, 1e4, 0, 1.0, 4096, 32.0, 1.0, ctypes.cast(f, ctypes.c_void_p), None) == 1


# --------------------------------------------------------------- refusals

class Args:
    """Well-formed arguments over host memory (never dereferenced by a check);
    `bad` replaces fields before a call."""

    BASE = 1 << 20

    def __init__(self, sef, **bad):
        self.sef, P = sef, self.BASE
        self.kv = dict(k=P, v=2 * P, page_stride=4 * 16 * 64, head_stride=16 * 64, row_stride=64, num_pages=8,
                       page_size=16, n_kv_heads=4, head_dim=64, dtype=sef.DTYPE_BF16)
        self.sq = dict(seq_start=3 * P, kv_len=3 * P + 64, page_table=3 * P + 128, n_seqs=2, n_rows=10, table_stride=4)
        self.rope = dict(freq=4 * P, rot_dim=64, style=0, mscale=1.0)
        self.at = dict(hq=8, q=5 * P, qs=512, k=6 * P, ks=256, v=7 * P, vs=256, qn=8 * P, kn=8 * P + 256, eps=1e-6,
                       qo=9 * P, qos=512, ko=10 * P, kos=256, scale=0.125, causal=1, o=11 * P, os=512, lse=12 * P,
                       ws=16 * P, wsb=1 << 30, prefix=0, pt=None)
        for name, v in bad.items():                 # (k and v: the cache's)
            next(d for d in (self.kv, self.sq, self.rope, self.at) if name in d)[name] = v
        self.KV = sef.ColibriKVPages(**self.kv)
        self.SQ = sef.ColibriSeqs(**self.sq)
        self.RP = sef.ColibriRope(**self.rope)

    def append(self, cache=True, rope=True):
        a, r = self.at, ctypes.byref
        return self.sef.colibri_append_qkv(r(self.KV) if cache else None, r(self.SQ), r(self.RP) if rope else None,
                                           a["hq"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["qn"], a["kn"],
                                           a["eps"], a["qo"], a["qos"], None)

    def rotate(self):
        a, r = self.at, ctypes.byref
        return self.sef.colibri_qk_norm_rope(r(self.SQ), r(self.RP), a["hq"], self.kv["n_kv_heads"], self.kv["head_dim"],
                                             self.kv["dtype"], a["q"], a["qs"], a["k"], a["ks"], a["qn"], a["kn"],
                                             a["eps"], a["qo"], a["qos"], a["ko"], a["kos"], None)

    def prompt(self):
        a, r = self.at, ctypes.byref
        return self.sef.colibri_attention_prompt(r(self.KV), r(self.SQ), a["hq"], a["q"], a["qs"], a["scale"],
                                                 a["causal"], a["o"], a["os"], a["lse"], a["ws"], a["wsb"], None)

    def decode(self):
        a, r = self.at, ctypes.byref
        return self.sef.colibri_attention_decode(r(self.KV), r(self.SQ), a["hq"], a["q"], a["qs"], a["scale"],
                                                 a["prefix"], a["pt"], a["o"], a["os"], a["lse"], a["ws"], a["wsb"],
                                                 None)


KV_BAD = [(dict(k=None), 1), (dict(v=None), 1), (dict(k=8), 1), (dict(v=24), 1), (dict(row_stride=60), 1),
          (dict(row_stride=0), 1), (dict(row_stride=68), 1), (dict(head_stride=4), 1), (dict(page_stride=12), 1),
          (dict(page_stride=-64), 1), (dict(num_pages=0), 1), (dict(page_size=0), 1), (dict(page_size=12), 4),
          (dict(page_size=4), 4), (dict(page_size=1 << 17), 4), (dict(head_dim=96), 4), (dict(head_dim=0), 1),
          (dict(n_kv_heads=0), 1), (dict(n_kv_heads=3), 1), (dict(dtype=7), 1), (dict(hq=0), 1), (dict(hq=-8), 1),
          (dict(hq=4 * 129, qs=1 << 16, qos=1 << 16, os=1 << 16), 4)]
SQ_BAD = [(dict(n_seqs=-1), 1), (dict(n_rows=-1), 1), (dict(kv_len=None), 1), (dict(table_stride=0), 1),
          (dict(table_stride=-1), 1), (dict(kv_len=3 * Args.BASE + 2), 1), (dict(n_rows=1 << 29), 1)]


@pytest.mark.parametrize("bad,status", KV_BAD + SQ_BAD + [
    (dict(page_table=None), 1), (dict(q=None), 1), (dict(q=8), 1), (dict(qs=511), 1), (dict(qs=504), 1),
    (dict(ks=128), 1), (dict(vs=260), 1), (dict(qn=2), 1), (dict(kn=8), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(qo=None), 1), (dict(qos=520, qo=5 * Args.BASE), 1), (dict(rot_dim=0), 1),
    (dict(rot_dim=72), 1), (dict(rot_dim=80), 1), (dict(freq=None), 1), (dict(freq=4), 1), (dict(style=2), 1),
    (dict(mscale=float("inf")), 1), (dict(seq_start=None), 1), (dict(n_rows=0), 0), (dict(n_seqs=0), 0)])
def test_append_refusals(sef, bad, status):
    assert Args(sef, **bad).append() == status
    if status and not set(bad) & set(Args(sef).rope):
        assert Args(sef, **bad).append(rope=False) == status
    assert Args(sef).append(cache=False) == 1


@pytest.mark.parametrize("bad,status", [
    (dict(hq=0), 1), (dict(head_dim=80), 4), (dict(dtype=3), 1), (dict(n_rows=-2), 1), (dict(q=None), 1),
    (dict(qo=4), 1), (dict(ko=None), 1), (dict(kos=250), 1), (dict(ko=10 * Args.BASE + 8), 1), (dict(rot_dim=8), 1),
    (dict(n_rows=0), 0)])
def test_qk_norm_rope_refusals(sef, bad, status):
    assert Args(sef, **bad).rotate() == status


ATTN_BAD = [(dict(q=None), 1), (dict(q=8), 1), (dict(qs=504), 1), (dict(os=500), 1), (dict(o=None), 1),
            (dict(o=5 * Args.BASE), 1), (dict(o=Args.BASE + 256), 1), (dict(o=2 * Args.BASE - 512), 1),
            (dict(lse=2), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
            (dict(scale=float("inf")), 1)]


@pytest.mark.parametrize("bad,status", KV_BAD + SQ_BAD + ATTN_BAD + [
    (dict(seq_start=None), 1), (dict(page_table=None), 1), (dict(page_table=None, kv_len=None), 1), (dict(n_rows=0), 0),
    (dict(n_seqs=0), 0)])
def test_prompt_refusals(sef, bad, status):
    assert Args(sef, **bad).prompt() == status
    n = ctypes.c_size_t()
    a = Args(sef, **bad)
    if not set(bad) & set(a.at) or "hq" in bad:
        assert sef.colibri_attention_prompt_workspace(ctypes.byref(a.KV), ctypes.byref(a.SQ), a.at["hq"],
                                                      ctypes.byref(n)) == status
    assert sef.colibri_attention_prompt_workspace(ctypes.byref(a.KV), ctypes.byref(a.SQ), 8, None) == 1


@pytest.mark.parametrize("bad,status", KV_BAD + SQ_BAD + ATTN_BAD + [
    (dict(page_table=None), 1), (dict(seq_start=3 * Args.BASE), 1), (dict(n_rows=9), 1), (dict(prefix=-16), 1),
    (dict(prefix=24, pt=13 * Args.BASE), 1), (dict(prefix=32, pt=None), 1), (dict(prefix=0, pt=13 * Args.BASE), 1),
    (dict(prefix=32, pt=13 * Args.BASE + 2), 1), (dict(n_rows=0, n_seqs=0), 0)])
def test_decode_refusals(sef, bad, status):
    base = dict(seq_start=None, n_seqs=10)
    assert Args(sef, **{**base, **bad}).decode() == status


def test_overlaps_are_refused_and_column_ranges_are_not(sef):
    B = Args.BASE
    row = 1024                                          # q 512, k 256, v 256 elements of one projection
    fused = dict(q=5 * B, qs=row, ks=row, vs=row)
    ok = dict(n_rows=0)                                 # nothing runs
    def at(**kw):
        a = Args(sef, **kw)
        a.at.update(k=5 * B + 1024, v=5 * B + 1536)
        return a
    assert at(**fused, **ok, qo=5 * B, qos=row).append() == 0
    for kw, status in [(dict(qo=5 * B + 1024, qos=row), 1), (dict(qo=5 * B + 16, qos=row), 1),
                       (dict(qo=5 * B + 2048, qos=512), 1), (dict(qo=B), 1)]:
        assert at(**fused, **kw).append() == status, kw
    # o between the columns of q's tensor (checked before the workspace is)
    wide = dict(qs=2048, os=2048, q=5 * B, table_stride=4096, ws=None)
    assert Args(sef, **{**wide, "o": 5 * B + 512}).prompt() == 1
    assert Args(sef, **{**wide, "o": 5 * B + 1024, "n_rows": 0, "ws": 16 * B}).prompt() == 0
    for kw in (dict(ko=5 * B), dict(qo=6 * B), dict(qo=9 * B, ko=9 * B), dict(ko=6 * B + 16)):
        a = Args(sef)
        a.at.update(kw)
        assert a.rotate() == 1, kw


def test_workspace_is_checked(sef):
    # few rows over a long table: the keys are split, so a workspace is needed
    kw = dict(seq_start=None, n_seqs=2, n_rows=2, table_stride=4096)
    a, n = Args(sef, **kw), ctypes.c_size_t()
    assert sef.colibri_attention_decode_workspace(ctypes.byref(a.KV), ctypes.byref(a.SQ), 8, 0, ctypes.byref(n)) == 0
    assert n.value > 0
    assert Args(sef, **kw, ws=None).decode() == 1
    assert Args(sef, **kw, wsb=n.value - 1).decode() == 1
    assert Args(sef, **kw, ws=16 * Args.BASE + 128).decode() == 1
    kw = dict(table_stride=4096)
    assert Args(sef, **kw, ws=None).prompt() == 1
