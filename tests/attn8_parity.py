"""Helpers of the 8-bit cache's tests: problems over codes and scales.

The bounds are those of attn_parity.  Codes and their products with a bf16 query
are exact in the kernels' operands; a score takes one product more (the block's
scale times scale * log2 e, 1 u) and a weight one more (the block's scale of v, 1 u
before the rounding to bf16 that is counted).  Both are inside the six units that
the bound of a score adds to its d + 2.

Single rows hold a weight times its value scale in f16 (half a step 2^-11, less than
bf16's 2^-8 that is counted), on a reference that puts the largest of a piece of a row
at 2^6 or above.  Below 2^-14 f16's half step is 2^-25, so each key may be off by
2^-25 / 2^6 = 2^-31 of the row's largest w_j scale_j, times its code: together by at
most keys * 2^-31 * sum_j w_j scale_j * (largest code).
"""

from __future__ import annotations

import numpy as np
import torch

from attn_parity import HALF, U, Problem, f64
from oracle import attention as oa

CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def decoded(codes):
    """Codes as float64 numpy."""
    return codes.detach().cpu().contiguous().float().double().numpy()


def random_codes(shape, code, g, nan=False):
    if code == "int8":
        return torch.randint(-127, 128, shape, generator=g, dtype=torch.int16).to(torch.int8)
    return (torch.randn(shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)


def same(a, b):
    """Equal bits of code tensors."""
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


class Problem8(Problem):
    """Sequences over a paged cache of codes.  Places that hold no key have the code
    0x7f (e4m3: NaN), blocks without keys the scale NaN; `pow2`: scales are powers of
    two, as the append leaves them."""

    def __init__(self, lens, hq, hkv, d, code="e4m3", block=16, page=16, layout="heads", prefix=0, spare=0, seed=0,
                 wide=0, pow2=False, size=1.0, device="cuda:0"):
        super().__init__(lens, hq, hkv, d, "bf16", page, layout, prefix, spare, seed, wide=wide, device=device)
        self.code, self.block = code, block
        dev = self.q.device
        g = torch.Generator().manual_seed(seed + 1)
        count, per = self.kp.shape[0], page // block
        used = np.zeros((count, page), dtype=bool)
        for b in range(len(lens)):
            for j in range(max(int(self.kv[b]), 0)):
                used[self.page_of(b, j), j % page] = True
        hole = torch.from_numpy(~used).to(dev)
        empty = hole.view(count, per, block).all(-1)
        top = 127.0 if code == "int8" else 200.0
        store = []
        for x in range(2):
            shape = (count, page, hkv, d) if layout == "rows" else (count, hkv, page, d)
            c = random_codes(shape, code, g).to(dev)
            c = c.transpose(1, 2) if layout == "rows" else c
            raw = c.view(torch.uint8)
            raw.copy_(torch.where(hole[:, None, :, None], torch.full_like(raw, 0x7f), raw))
            s = torch.exp(torch.randn(count, hkv, per, generator=g)) * (3.0 * size / top)
            if pow2:
                s = torch.exp2(torch.floor(torch.log2(s)))
            s = s.to(dev)
            s.masked_fill_(empty[:, None, :], float("nan"))
            store += [c, s]
        self.kc, self.ks, self.vc, self.vs = store

    def cache(self, A):
        return A.PagedKVCache8(self.kc, self.vc, self.ks, self.vs)

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
            largest = oa.attend(q[at], k, np.broadcast_to(self.value_scale(b)[..., None], v.shape), lim, scale)[2]
            keys = max(len(k), 1)
            qk = np.linalg.norm(q[at], axis=-1) * (np.linalg.norm(k, axis=-1).max() if len(k) else 0.0) * scale
            es = ((self.d + 2) + 6) * U * qk                        # [n, hq]
            e = np.expm1(es) + 2.0 ** -22
            tol = 2 * (e + (keys + 8) * 2.0 ** -23)[..., None] * spread + r * np.abs(o) + r * spread * (1 + r)
            tol = tol + keys * 2.0 ** -31 * largest * oa.CODE_MOST[self.code] * (1 + r)
            bad = ~(np.abs(got[at] - o) <= tol)
            assert not bad.any(), (b, self.lens[b], "o", int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                                   float(np.nanmax(np.abs(got[at] - o) / np.maximum(tol, 1e-30))))
            if glse is not None:
                fine = np.isfinite(ls)
                assert np.array_equal(np.isneginf(glse[at]), ~fine), (b, "lse of empty rows")
                # (the reference that the sum is taken on may be off the largest score by the
                # value scales' log2, 64 at most)
                lt = es + e + (keys + 8) * 2.0 ** -23 + 4 * U * (np.abs(np.where(fine, ls, 0)) + 64)
                d = np.abs(np.where(fine, glse[at] - np.where(fine, ls, 0), 0))
                assert (d <= lt).all(), (b, "lse", float(d.max()), float((d / lt).max()))

    def value_scale(self, b):
        """float64 scales of v of sequence b's keys, [L, hkv]."""
        j = np.arange(max(int(self.kv[b]), 0))
        pid = np.array([self.page_of(b, int(x)) for x in j], dtype=np.int64)
        return np.abs(f64(self.vs)[pid, :, j % self.page // self.block]) if len(j) else np.zeros((0, self.hkv))

    def keys(self, b):
        L = max(int(self.kv[b]), 0)
        j = np.arange(L)
        pid = np.array([self.page_of(b, int(x)) for x in j], dtype=np.int64)
        off = j % self.page
        out = []
        for c, s in ((self.kc, self.ks), (self.vc, self.vs)):
            at = torch.from_numpy(pid).to(c.device), torch.from_numpy(off).to(c.device)
            v = decoded(c.view(torch.uint8)[at[0], :, at[1]].view(c.dtype)) if L else np.zeros((0, self.hkv, self.d))
            out.append(v * f64(s)[pid, :, off // self.block][..., None])
        return out
