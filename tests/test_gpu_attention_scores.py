"""Scores that move the reference of the softmax, or have it stay where it is:
every kernel forms weights on a reference that stands as long as they fit
(tensor cores: 2^24 above, 2^-64 below while a row has none; single rows: 2^8), so
rows are given scores far below it, far above it, and rising past it in every
step of 128 keys, over at least five steps.  Against the oracle, at attn_parity's
bounds, which grow with the size of the scores."""

import numpy as np
import pytest
import torch

from attn_parity import Problem, seqs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A(lib):
    from sparse_expert_ffn_gb300 import attention
    return attention


# log2 of the weight of key j, before noise
PATTERNS = {
    "low": lambda j: np.full(len(j), -200.0),
    "low then 0": lambda j: np.where(j < 128, -200.0, 0.0),
    "low then high": lambda j: np.where(j < 128, -200.0, 100.0),
    "rising": lambda j: 30.0 * (j // 128),
    "falling": lambda j: -30.0 * (j // 128),
    "low tail": lambda j: np.where(j % 128 < 96, -200.0, 20.0),     # the last 32 keys of each step
    "jumps": lambda j: 150.0 * np.sin(j // 12 * 2.0),
}


def _set_scores(p, pattern):
    """Column 0 of the queries and keys gives the pattern (rows in turn at full size,
    a sixteenth of it, and reversed), the other columns noise of a few units."""
    p.q.mul_(0.1)
    size = torch.tensor([8.0, 0.5, -8.0])[torch.arange(p.rows) % 3].to(p.q)
    p.q[..., 0] = size[:, None]

    def column(j):
        return torch.from_numpy(PATTERNS[pattern](j) * np.log(2.0) / 8.0).to(p.q.device).to(p.dt)

    for b, (n, total) in enumerate(p.lens):
        j = np.arange(n if not p.page else total)
        if not len(j):
            continue
        if not p.page:
            p.k[int(p.start[b]):int(p.start[b + 1]), :, 0] = column(j)[:, None]
        else:
            pid = torch.from_numpy(np.array([p.page_of(b, int(x)) for x in j], dtype=np.int64)).to(p.q.device)
            p.kp[pid, :, torch.from_numpy(j % p.page).to(p.q.device), 0] = column(j)[:, None]


def _pick(p):
    """Some rows of every sequence, the first and last among them."""
    r = np.random.default_rng(4)
    out = [s for s in (p.start[:-1], p.start[1:] - 1)]
    return np.unique(np.concatenate(out + [r.integers(0, p.rows, 60)]))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pattern", list(PATTERNS))
@pytest.mark.parametrize("d,hq,hkv", [(64, 2, 1), (128, 3, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_packed_prompts(A, d, hq, hkv, causal, pattern, dtype):
    p = Problem([(777, 777), (140, 140), (640, 640)], hq, hkv, d, dtype, 0, seed=d)
    _set_scores(p, pattern)
    out, lse = torch.empty_like(p.q), torch.empty(p.rows, hq, device=p.q.device)
    A.attention_prompt(seqs(A, p, paged=False), p.q, p.k, p.v, scale=1.0, causal=causal, out=out, lse=lse)
    p.check(out, lse, causal, scale=1.0, rows=_pick(p))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pattern", list(PATTERNS))
@pytest.mark.parametrize("d,hq,hkv,page", [(64, 16, 16, 16), (128, 16, 8, 64)])
def test_paged_prompts(A, d, hq, hkv, page, pattern, dtype):
    """Many key heads, so that the keys of a tile stay in one or two ranges."""
    p = Problem([(130, 900), (70, 800), (300, 1100), (520, 700)], hq, hkv, d, dtype, page, seed=d, fill=float("nan"))
    _set_scores(p, pattern)
    out, lse = torch.empty_like(p.q), torch.empty(p.rows, hq, device=p.q.device)
    A.attention_prompt_paged(A.PagedKVCache(p.kp, p.vp), seqs(A, p), p.q, scale=1.0, out=out, lse=lse)
    p.check(out, lse, True, scale=1.0, rows=_pick(p))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pattern", list(PATTERNS))
@pytest.mark.parametrize("d,hq,hkv,page", [(64, 16, 16, 64), (128, 32, 16, 128)])
def test_prefixes(A, d, hq, hkv, page, pattern, dtype):
    """9 ranges of five steps each over the prefix, own keys that go on in the pattern
    or end inside the prefix."""
    prefix = 9 * 5 * 128
    p = Problem([(1, prefix + 200), (1, prefix), (1, prefix + 7), (1, 1000), (1, 130), (1, 0)], hq, hkv, d, dtype, page,
                prefix=prefix, seed=d, fill=float("nan"))
    _set_scores(p, pattern)
    out, lse = torch.empty_like(p.q), torch.empty(p.rows, hq, device=p.q.device)
    A.attention_decode(A.PagedKVCache(p.kp, p.vp), seqs(A, p, decode=True), p.q, prefix_len=prefix,
                       prefix_table=p.prefix_table, scale=1.0, out=out, lse=lse)
    p.check(out, lse, False, scale=1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pattern", list(PATTERNS))
@pytest.mark.parametrize("d,hq,hkv,page", [(64, 2, 2, 8), (128, 4, 1, 32), (64, 20, 1, 64), (128, 33, 1, 16)])
def test_single_rows(A, d, hq, hkv, page, pattern, dtype):
    """Lengths that stay in one share and ones that are cut."""
    p = Problem([(1, 5000), (1, 60), (1, 700), (1, 1), (1, 131)], hq, hkv, d, dtype, page, seed=d, fill=float("nan"))
    _set_scores(p, pattern)
    out, lse = torch.empty_like(p.q), torch.empty(p.rows, hq, device=p.q.device)
    A.attention_decode(A.PagedKVCache(p.kp, p.vp), seqs(A, p, decode=True), p.q, scale=1.0, out=out, lse=lse)
    p.check(out, lse, False, scale=1.0)


@pytest.mark.parametrize("d", [64, 128])
def test_longest_shares_of_single_rows(A, d):
    """Enough keys that a share has many steps, the reference of which moves again and
    again (bf16: more than 2^8 after the first step)."""
    p = Problem([(1, 60000), (1, 60000)], 4, 1, d, "bf16", 64, seed=d)
    _set_scores(p, "jumps")
    out, lse = torch.empty_like(p.q), torch.empty(p.rows, 4, device=p.q.device)
    A.attention_decode(A.PagedKVCache(p.kp, p.vp), seqs(A, p, decode=True), p.q, scale=1.0, out=out, lse=lse)
    p.check(out, lse, False, scale=1.0)
