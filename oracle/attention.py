"""Plain float64 CPU oracle of the attention operators (test infrastructure only).

Definitions, one sequence or one head at a time:

* ``rope_frequencies``: theta^(-2 i / rot), stretched for long contexts
  (linear, ntk: theta raised; yarn: by parts, Peng et al., 2023);
* ``norm_rotate``: RMSNorm of each head, then the rotation of its pairs, the
  pair (a, b) taken as the complex number a + i b times e^(i t f);
* ``attend``: softmax(scale q k^T) v over the first ``limit`` keys of each row,
  zeros and a log-sum of -inf for a row without keys.
"""

from __future__ import annotations

import math

import numpy as np


def rope_frequencies(rot, theta=10000.0, scaling="none", factor=1.0, trained=4096, beta_fast=32.0,
                     beta_slow=1.0):
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = theta ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        # pair i turns trained * f_i / 2 pi times in the trained context
        def pair(turns):
            return rot * math.log(trained / (2 * math.pi * turns)) / (2 * math.log(theta))
        lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), rot - 1)
        stretch = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        return f / factor * stretch + f * (1 - stretch), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def norm_rotate(x, pos, freq=None, style="half", mscale=1.0, weight=None, eps=0.0):
    """x [n, heads, d] at positions pos [n]."""
    x = np.array(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * weight
    if freq is None:
        return x
    half = len(freq)
    turn = mscale * np.exp(1j * np.asarray(pos, dtype=np.float64)[:, None] * freq)[:, None, :]
    a, b = (x[..., :half], x[..., half:2 * half]) if style == "half" else \
        (x[..., 0:2 * half:2], x[..., 1:2 * half:2])
    z = (a + 1j * b) * turn
    if style == "half":
        x[..., :half], x[..., half:2 * half] = z.real, z.imag
    else:
        x[..., 0:2 * half:2], x[..., 1:2 * half:2] = z.real, z.imag
    return x


def attend(q, k, v, limit, scale):
    """q [n, hq, d]; k, v [L, hkv, d]; limit [n] keys each row sees.
    Returns o [n, hq, d], lse [n, hq], spread [n, hq, d] = sum_j w_j |v_j|."""
    n, hq, d = q.shape
    L, hkv = k.shape[0], k.shape[1]
    o, lse, spread = np.zeros((n, hq, d)), np.full((n, hq), -np.inf), np.zeros((n, hq, d))
    for h in range(hq):
        kh, vh = k[:, h // (hq // hkv)], v[:, h // (hq // hkv)]
        for i in range(n):
            c = int(min(max(limit[i], 0), L))
            if c == 0:
                continue
            s = scale * (kh[:c] @ q[i, h])
            m = s.max()
            w = np.exp(s - m)
            lse[i, h] = m + math.log(w.sum())
            w /= w.sum()
            o[i, h] = w @ vh[:c]
            spread[i, h] = w @ np.abs(vh[:c])
    return o, lse, spread
