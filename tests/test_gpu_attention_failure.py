"""Attention operators where something is wrong, without faulting the GPU: a
producer that copies nothing (every wait of the tensor-core kernel is bounded;
rows whose wait gave up are NaN and the context stays usable), and scores that
are not numbers."""

import pytest
import torch

from attn_parity import Problem, seqs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A(lib):
    from sparse_expert_ffn_gb300 import attention
    return attention


@pytest.mark.parametrize("d", [64, 128])
def test_stalled_copies_give_nan_rows(A, monkeypatch, d):
    p = Problem([(200, 200), (9, 9)], 4, 2, d, "bf16", 0, spare=3, seed=1)
    sq = seqs(A, p, paged=False)
    ref = A.attention_prompt(sq, p.q, p.k, p.v)
    dec = Problem([(1, 1300 + i) for i in range(5)], 8, 2, d, "bf16", 16, prefix=1024, seed=2)
    cache, dsq = A.PagedKVCache(dec.kp, dec.vp), seqs(A, dec, decode=True)
    dref = A.attention_decode(cache, dsq, dec.q, prefix_len=1024, prefix_table=dec.prefix_table)
    torch.cuda.synchronize()
    monkeypatch.setenv("COLIBRI_WAIT_LIMIT_NS", "20000000")
    monkeypatch.setenv("COLIBRI_TEST_STALL_TMA", "1")
    out, lse = torch.zeros_like(p.q), torch.zeros(p.rows, 4, device="cuda:0")
    A.attention_prompt(sq, p.q, p.k, p.v, out=out, lse=lse)
    dout = A.attention_decode(cache, dsq, dec.q, prefix_len=1024, prefix_table=dec.prefix_table)
    torch.cuda.synchronize()
    monkeypatch.delenv("COLIBRI_WAIT_LIMIT_NS")
    monkeypatch.delenv("COLIBRI_TEST_STALL_TMA")
    assert out[:209].isnan().all() and lse[:209].isnan().all()
    assert (out[209:] == 0).all() and (lse[209:] == 0).all()
    assert dout.isnan().all()
    assert torch.equal(A.attention_prompt(sq, p.q, p.k, p.v)[:209], ref[:209])
    again = A.attention_decode(cache, dsq, dec.q, prefix_len=1024, prefix_table=dec.prefix_table)
    assert torch.equal(again, dref)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scores_that_are_not_numbers(A, dtype):
    """A NaN or infinite query makes its own rows NaN and no other; a NaN key
    the rows that see it."""
    p = Problem([(1, 700), (1, 40), (1, 700), (1, 1300)], 4, 1, 64, dtype, 16, seed=3)
    cache, sq = A.PagedKVCache(p.kp, p.vp), seqs(A, p, decode=True)
    ref = A.attention_decode(cache, sq, p.q)
    q = p.q.clone()
    q[0, 1] = float("nan")
    q[2, 3, 5] = float("inf")
    lse = torch.empty(4, 4, device="cuda:0")
    got = A.attention_decode(cache, sq, q, lse=lse)
    hit = torch.zeros(4, 4, dtype=torch.bool, device="cuda:0")
    hit[0, 1] = hit[2, 3] = True
    assert got[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(got[~hit], ref[~hit])
    pr = Problem([(300, 300)], 4, 1, 64, dtype, 0, seed=4)
    psq = seqs(A, pr, paged=False)
    ref = A.attention_prompt(psq, pr.q, pr.k, pr.v)
    pr.k[170] = float("nan")
    got = A.attention_prompt(psq, pr.q, pr.k, pr.v)
    assert torch.equal(got[:170], ref[:170]) and got[170:].isnan().all()
