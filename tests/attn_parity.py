"""Helpers of the attention tests: seeded problems and the error bounds.

Bounds, per element (u = 2^-24, half a float32 step; r = half a step of the
output type, 2^-8 for bf16):

* Norm and rotation: the sum of up to 128 squares over 8 sequential additions
  and at most 4 butterfly ones, its division, root, reciprocal and two
  products stay within 24 u; sine and cosine of a float32 half turn are good
  to 4 u of 1 and the turn itself, rounded to 24 bits, to pi 2^-25 < 2 u of an
  angle; two products and a sum add 2 u.  Together less than
  C = 32 u (|a| + |b|) mscale for the pair (a, b) after the norm, and one
  rounding r of the result.
* A score: float32 sum of d products, at most (d + 2) u scale |q| |k| off, and
  the product with scale * log2 e and the difference to the maximum 3 u of the
  larger of the two: E_s.  2^x is good to 2^-22.  Weights are then off by at
  most e = expm1(E_s) + 2^-22 each and their sums, however they are added up,
  by (keys + 8) * 2^-23 (half steps of products and sums in any order, twice
  that for the tensor cores, which may cut instead of round).  o = sum w v /
  sum w is off by at most 2 (e + (keys + 8) 2^-23) sum w |v|.
* bf16 rounds each weight to bf16 for the product with v: r sum w |v| more.
* A kernel that joins key ranges rounds as the sums do; it is inside the count.
* ln sum: E_s + e + (keys + 8) 2^-23, and 4 u of its own size.
"""

from __future__ import annotations

import numpy as np
import torch

import oracle
from oracle import attention as oa

U = 2.0 ** -24
HALF = {torch.float32: torch.finfo(torch.float32).eps / 2, torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2}
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return oracle.to_f64(t.detach().cpu().contiguous())


class Problem:
    """Sequences of (rows, keys) with a shuffled paged cache (page > 0) or
    packed keys, all from one seed."""

    def __init__(self, lens, hq, hkv, d, dtype="bf16", page=16, layout="heads", prefix=0, spare=0, seed=0,
                 q_scale=1.5, fill=None, device="cuda:0", wide=0):
        self.lens, self.hq, self.hkv, self.d, self.page, self.prefix = lens, hq, hkv, d, page, prefix
        self.dt, dev = DT[dtype], torch.device(device)
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.rows = sum(n for n, _ in lens) + spare

        def normal(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g) * scale).to(self.dt).to(dev)

        self.start = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
        self.kv = np.array([t for _, t in lens], dtype=np.int32)
        self.q = normal(self.rows, hq, d, scale=q_scale)
        self.seq_start = torch.from_numpy(self.start).to(dev)
        self.kv_len = torch.from_numpy(self.kv).to(dev)
        if not page:
            self.k, self.v = normal(self.rows, hkv, d), normal(self.rows, hkv, d)
            return
        shared = prefix // page
        need = [max(0, -(-max(t, 0) // page) - shared) for t in self.kv]
        count = shared + sum(need) + 3
        ids = rng.permutation(count).astype(np.int32)
        self.prefix_ids = ids[:shared]
        width = shared + max(max(need, default=0), 1) + wide
        # entries that no key lies under name pages that do not exist
        self.table_np = np.full((len(lens), width), count + 7, dtype=np.int32)
        at = shared
        for b, n in enumerate(need):
            self.table_np[b, shared:shared + n] = ids[at:at + n]
            at += n
        self.table = torch.from_numpy(self.table_np).to(dev)
        self.prefix_table = torch.from_numpy(self.prefix_ids.copy()).to(dev)
        shape = (count, page, hkv, d) if layout == "rows" else (count, hkv, page, d)
        self.kp, self.vp = normal(*shape), normal(*shape)
        if layout == "rows":
            self.kp, self.vp = self.kp.transpose(1, 2), self.vp.transpose(1, 2)
        if fill is not None:
            # every place that holds no key of any sequence
            used = torch.zeros(count, page, dtype=torch.bool)
            for b in range(len(lens)):
                for j in range(max(int(self.kv[b]), 0)):
                    used[self.page_of(b, j), j % page] = True
            hole = (~used)[:, None, :, None].expand(count, hkv, page, d).to(dev)
            self.kp.masked_fill_(hole, fill)
            self.vp.masked_fill_(hole, fill)

    def page_of(self, b, j):
        return int(self.prefix_ids[j // self.page]) if j < self.prefix else int(self.table_np[b, j // self.page])

    def keys(self, b):
        """float64 keys and values of sequence b."""
        if not self.page:
            s = slice(int(self.start[b]), int(self.start[b + 1]))
            return f64(self.k)[s], f64(self.v)[s]
        L = max(int(self.kv[b]), 0)
        j = np.arange(L)
        pid = np.array([self.page_of(b, int(x)) for x in j], dtype=np.int64)
        return [f64(x)[pid, :, j % self.page] if L else np.zeros((0, self.hkv, self.d)) for x in (self.kp, self.vp)]

    def limits(self, b, causal):
        n = int(self.start[b + 1] - self.start[b])
        kv = int(self.kv[b]) if self.page else n
        return kv - n + np.arange(n) + 1 if causal else np.full(n, kv)

    def check(self, out, lse, causal, scale=None, rows=None):
        """Every row against the oracle (rows: a subset of row numbers)."""
        scale = self.d ** -0.5 if scale is None else scale
        q, got, glse = f64(self.q), f64(out), None if lse is None else lse.double().cpu().numpy()
        r = HALF[self.dt]
        for b in range(len(self.lens)):
            k, v = self.keys(b)
            lim = self.limits(b, causal)
            at = np.arange(self.start[b], self.start[b + 1])
            if rows is not None:
                pick = np.isin(at, rows)
                at, lim = at[pick], lim[pick]
            if not len(at):
                continue
            o, ls, spread = oa.attend(q[at], k, v, lim, scale)
            keys = max(len(k), 1)
            qk = np.linalg.norm(q[at], axis=-1) * (np.linalg.norm(k, axis=-1).max() if len(k) else 0.0) * scale
            es = ((self.d + 2) + 6) * U * qk                        # [n, hq]
            e = np.expm1(es) + 2.0 ** -22
            tol = 2 * (e + (keys + 8) * 2.0 ** -23)[..., None] * spread + r * np.abs(o)
            if self.dt == torch.bfloat16:
                tol = tol + r * spread * (1 + r)
            bad = ~(np.abs(got[at] - o) <= tol)
            assert not bad.any(), (b, self.lens[b], "o", int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                                   float(np.nanmax(np.abs(got[at] - o) / np.maximum(tol, 1e-30))))
            if glse is not None:
                fine = np.isfinite(ls)
                assert np.array_equal(np.isneginf(glse[at]), ~fine), (b, "lse of empty rows")
                lt = es + e + (keys + 8) * 2.0 ** -23 + 4 * U * np.abs(np.where(fine, ls, 0))
                d = np.abs(np.where(fine, glse[at] - np.where(fine, ls, 0), 0))
                assert (d <= lt).all(), (b, "lse", float(d.max()), float((d / lt).max()))


def seqs(sef_attention, p, paged=True, decode=False):
    return sef_attention.Sequences(None if decode else p.seq_start, p.kv_len if paged else None,
                                   p.table if paged else None)
