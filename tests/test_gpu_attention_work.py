"""How the attention operators hand out their work: more work items than the
GPU takes at once (CTAs that take over others' items, also inside a replayed
graph), orders over many sequences, keys cut into more than a thousand pieces,
CTAs that give up in the middle of their work, and arrays that hold anything."""

import threading

import numpy as np
import pytest
import torch

from attn_parity import Problem, seqs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A(lib):
    from sparse_expert_ffn_gb300 import attention
    return attention


def _uneven(count, top, seed):
    r = np.random.default_rng(seed)
    return [(int(n), int(n)) for n in r.integers(1, top, count)]


@pytest.mark.parametrize("count,top,hq,hkv,d,causal", [(30, 500, 16, 8, 64, True), (12, 900, 32, 8, 128, True),
                                                       (150, 60, 8, 8, 64, True), (40, 300, 16, 8, 128, False)])
def test_more_items_than_sms(A, count, top, hq, hkv, d, causal):
    """Every item is done once, eagerly and in a graph whose lengths change
    between replays; sampled rows against the oracle."""
    p = Problem(_uneven(count, top, d + count), hq, hkv, d, "bf16", 0, seed=count)
    sq = seqs(A, p, paged=False)
    out, lse = torch.full_like(p.q, 9.0), torch.full((p.rows, hq), 9.0, device="cuda:0")
    A.attention_prompt(sq, p.q, p.k, p.v, causal=causal, out=out, lse=lse)
    torch.cuda.synchronize()
    pick = np.unique(np.concatenate([p.start[:-1], p.start[1:] - 1, np.random.default_rng(1).integers(0, p.rows, 30)]))
    p.check(out, lse, causal, rows=pick[:: max(1, len(pick) // 60)])
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    again = A.attention_prompt(sq, p.q, p.k, p.v, causal=causal)
    assert torch.equal(again, out)
    g = torch.cuda.CUDAGraph()
    gout = torch.empty_like(out)
    with torch.cuda.graph(g):
        A.attention_prompt(sq, p.q, p.k, p.v, causal=causal, out=gout)
    start = p.seq_start.clone()
    for t in range(3):
        p.seq_start.copy_(start)
        p.seq_start[1:-1] -= t                        # other lengths of the same rows
        p.seq_start.clamp_(min=0)
        gout.fill_(5.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(gout, A.attention_prompt(sq, p.q, p.k, p.v, causal=causal, out=torch.full_like(gout, 5.0)))


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (5, 1, 128), (20, 1, 64)])
def test_one_sequence_in_many_pieces(A, hq, hkv, d):
    """40000 keys of one head over all warps of the GPU; equal scores and
    one-hot values give the exact count of the keys."""
    keys = 40000 + 37
    p = Problem([(1, keys)], hq, hkv, d, "bf16", 64, seed=2)
    p.q.zero_()
    pid = torch.from_numpy(p.table_np[0].astype(np.int64)).cuda()
    j = torch.arange(keys, device="cuda:0")
    p.vp.zero_()
    p.vp[pid[j // 64], 0, j % 64, j % d] = 1.0
    lse = torch.empty(1, hq, device="cuda:0")
    out = A.attention_decode(A.PagedKVCache(p.kp, p.vp), seqs(A, p, decode=True), p.q, lse=lse)
    want = torch.bincount(j % d, minlength=d).double() / keys
    # weights 1 and exact sums per piece; their joining and the rounding to bf16:
    # a few units of 2^-23 and half a step
    assert ((out.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -18) * want).all()
    assert (lse.double() - np.log(keys)).abs().max() <= 2.0 ** -19 * np.log(keys)


def test_rows_of_a_cta_that_gives_up_in_the_middle(A, monkeypatch):
    """Copies stop at the second item that a CTA takes over: each row is what it
    would have been, or NaN, and nothing else is written."""
    p = Problem(_uneven(30, 400, 3), 16, 8, 128, "bf16", 0, spare=4, seed=5)
    sq = seqs(A, p, paged=False)
    ref = A.attention_prompt(sq, p.q, p.k, p.v, out=torch.zeros_like(p.q))
    torch.cuda.synchronize()
    monkeypatch.setenv("COLIBRI_WAIT_LIMIT_NS", "20000000")
    monkeypatch.setenv("COLIBRI_TEST_STALL_TMA", "2")
    out, lse = torch.zeros_like(p.q), torch.zeros(p.rows, 16, device="cuda:0")
    A.attention_prompt(sq, p.q, p.k, p.v, out=out, lse=lse)
    torch.cuda.synchronize()
    monkeypatch.delenv("COLIBRI_WAIT_LIMIT_NS")
    monkeypatch.delenv("COLIBRI_TEST_STALL_TMA")
    n = int(p.start[-1])
    gone = out.isnan().all(-1)
    assert gone[:n].any() and not gone[:n].all()
    assert torch.equal(out[~gone], ref[~gone]) and torch.equal(lse[:n].isnan(), gone[:n])
    assert (out[n:] == 0).all()
    assert torch.equal(A.attention_prompt(sq, p.q, p.k, p.v, out=torch.zeros_like(p.q)), ref)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_arrays_that_hold_anything(A, dtype):
    """Whatever seq_start, kv_len and the tables hold, nothing outside the
    outputs and the cache is written, and the next calls are right."""
    r = np.random.default_rng(6)
    p = Problem([(50, 90), (70, 70), (30, 200)], 8, 2, 64, dtype, 16, spare=10, seed=7, wide=3)
    cache, sq = A.PagedKVCache(p.kp, p.vp), seqs(A, p)
    ref = A.attention_prompt_paged(cache, sq, p.q, out=torch.zeros_like(p.q))
    guard = torch.full((p.rows + 64, 8, 64), 3.0, dtype=p.dt, device="cuda:0")
    out = guard[32:-32]
    edge = np.array([-2 ** 31, -1, 0, 1, 49, 120, 160, 2 ** 30, 2 ** 31 - 1], dtype=np.int64)
    k, v = (torch.randn(p.rows, 2, 64, device="cuda:0").to(p.dt) for _ in range(2))
    f, _ = A.rope_frequencies(64)
    rope = A.Rope(f.cuda())
    one = torch.zeros(3, 8, 64, dtype=p.dt, device="cuda:0")
    for trial in range(40):
        junk = A.Sequences(*(torch.from_numpy(r.choice(edge, s).astype(np.int32)).cuda()
                             for s in ((4,), (3,), (3, p.table.shape[1]))))
        store = A.PagedKVCache(p.kp.clone(), p.vp.clone())
        A.append_qkv(store, junk, p.q, k, v, rope=rope, q_out=out)
        A.qk_norm_rope(A.Sequences(junk.seq_start, junk.kv_len), p.q, k, rope=rope, q_out=out)
        A.attention_prompt_paged(store, junk, p.q, causal=bool(trial & 1), out=out)
        A.attention_prompt(A.Sequences(junk.seq_start), p.q, k, v, causal=bool(trial & 1), out=out)
        A.attention_decode(store, A.Sequences(None, junk.kv_len, junk.page_table), one, prefix_len=32,
                           prefix_table=junk.page_table[0, :2].contiguous())
        torch.cuda.synchronize()
        assert (guard[:32] == 3.0).all() and (guard[-32:] == 3.0).all()
    assert torch.equal(A.attention_prompt_paged(cache, sq, p.q, out=torch.zeros_like(p.q)), ref)


def test_two_threads_with_the_same_objects(A):
    """One cache, one Sequences and one Rope used by two threads, with different
    numbers of rows, on streams of their own."""
    p = Problem([(60, 60), (40, 90)], 8, 2, 64, "bf16", 16, spare=20, seed=8)
    cache, sq = A.PagedKVCache(p.kp, p.vp), seqs(A, p)
    n = int(p.start[-1])
    ref = A.attention_prompt_paged(cache, sq, p.q[:n])
    torch.cuda.synchronize()
    good = []

    def work(rows):
        s = torch.cuda.Stream()
        for _ in range(50):
            out = A.attention_prompt_paged(cache, sq, p.q[:rows], stream=s)
            s.synchronize()
            good.append(torch.equal(out[:n], ref))

    threads = [threading.Thread(target=work, args=(rows,)) for rows in (n, n + 20)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert len(good) == 100 and all(good)


# ------------------------------------------------------------ float32 single tokens

@pytest.mark.parametrize("page,prefix", [(8, 0), (64, 0), (32, 96)])
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (2, 1, 128), (6, 2, 64), (4, 1, 128), (5, 1, 64), (8, 8, 128),
                                     (11, 1, 128), (32, 1, 64), (33, 1, 64)])
def test_float32_tokens_around_a_step(A, hq, hkv, d, page, prefix):
    """Lengths around the 8 and 16 keys of a step, none, and long ones that are cut
    into pieces; places that hold no key are NaN."""
    own = [0, 1, 7, 8, 9, 15, 16, 17, 31, 33, 64, 20011, 0, 5003]
    p = Problem([(1, prefix + t) for t in own], hq, hkv, d, "fp32", page, prefix=prefix, seed=hq + d, fill=float("nan"))
    lse = torch.full((p.rows, hq), 9.0, device=p.q.device)
    out = A.attention_decode(A.PagedKVCache(p.kp, p.vp), seqs(A, p, decode=True), p.q, prefix_len=prefix,
                             prefix_table=p.prefix_table if prefix else None, out=torch.full_like(p.q, 9.0), lse=lse)
    p.check(out, lse, False)


@pytest.mark.parametrize("hq,d", [(1, 64), (3, 128), (4, 64), (20, 128)])
def test_one_float32_sequence_in_many_pieces(A, hq, d):
    """Equal scores and one-hot values give the exact count of the keys."""
    keys = 40000 + 37
    p = Problem([(1, keys)], hq, 1, d, "fp32", 64, seed=3)
    p.q.zero_()
    pid = torch.from_numpy(p.table_np[0].astype(np.int64)).cuda()
    j = torch.arange(keys, device="cuda:0")
    p.vp.zero_()
    p.vp[pid[j // 64], 0, j % 64, j % d] = 1.0
    lse = torch.empty(1, hq, device="cuda:0")
    out = A.attention_decode(A.PagedKVCache(p.kp, p.vp), seqs(A, p, decode=True), p.q, lse=lse)
    want = torch.bincount(j % d, minlength=d).double() / keys
    # weights 1 and exact sums per piece; a piece's division, and the joining of up to
    # 1216 pieces by their log2-sums (each to a few 2^-24 of at most 16): 2^-18
    assert ((out.double() - want).abs() <= 2.0 ** -18 * want).all()
    assert ((lse.double() - np.log(keys)).abs() <= 2.0 ** -18 * np.log(keys)).all()


def test_float32_tokens_large_equal_and_nan_scores(A):
    """Scores that move the reference again and again, a sequence of equal scores,
    and one NaN key, which makes its sequence's rows NaN and no other's."""
    p = Problem([(1, 700), (1, 300), (1, 90), (1, 1)], 4, 1, 64, "fp32", 16, seed=5, q_scale=40.0)
    for j in range(300):
        p.kp[int(p.table_np[1, j // 16]), 0, j % 16, :] = 0
    cache = A.PagedKVCache(p.kp, p.vp)
    lse = torch.empty(4, 4, device="cuda:0")
    out = A.attention_decode(cache, seqs(A, p, decode=True), p.q, lse=lse)
    p.check(out, lse, False)
    p.kp[int(p.table_np[2, 40 // 16]), 0, 40 % 16, 3] = float("nan")
    again = A.attention_decode(cache, seqs(A, p, decode=True), p.q)
    assert torch.isnan(again[2]).all() and torch.equal(again[[0, 1, 3]], out[[0, 1, 3]])


# ------------------------------------------------------------ workspaces

def _cut(seed, lens, dtype="bf16"):
    """Sequences whose keys are cut into pieces, so that a call needs its workspace."""
    return Problem([(1, t) for t in lens], 8, 2, 64, dtype, 16, seed=seed)


def test_calls_of_two_threads_on_one_stream(A):
    """Each call's pieces stay its own although the calls of the threads interleave."""
    p = [_cut(1, [9000, 5, 3000]), _cut(2, [40, 12000])]
    cache = [A.PagedKVCache(x.kp, x.vp) for x in p]
    sq = [seqs(A, x, decode=True) for x in p]
    want = [A.attention_decode(cache[i], sq[i], p[i].q).clone() for i in range(2)]
    p[0].check(want[0], None, False)
    p[1].check(want[1], None, False)
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        got[i] = [A.attention_decode(cache[i], sq[i], p[i].q) for _ in range(200)]

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 200 and all(torch.equal(g, want[i]) for g in got[i])


def test_graphs_and_eager_calls_share_no_workspace(A):
    """Two graphs captured after eager calls, replayed beside each other and beside
    eager calls on a third stream."""
    p = [_cut(3, [20000, 700]), _cut(4, [300, 15000]), _cut(5, [8000, 8000])]
    cache = [A.PagedKVCache(x.kp, x.vp) for x in p]
    sq = [seqs(A, x, decode=True) for x in p]
    want = [A.attention_decode(cache[i], sq[i], p[i].q).clone() for i in range(3)]
    for x, w in zip(p, want):
        x.check(w, None, False)
    graphs, outs = [], []
    for i in range(2):
        g, out = torch.cuda.CUDAGraph(), torch.empty_like(want[i])
        with torch.cuda.graph(g):
            A.attention_decode(cache[i], sq[i], p[i].q, out=out)
        graphs.append(g), outs.append(out)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        [o.fill_(7.0) for o in outs]
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = [A.attention_decode(cache[2], sq[2], p[2].q) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
        assert all(torch.equal(e, want[2]) for e in eager)


def test_workspaces_of_growing_and_alternating_calls(A):
    """Small, large and small again, on streams in turn without waiting between."""
    p = [_cut(6, [700]), _cut(7, [9000] * 8, "fp32"), _cut(8, [2000, 60])]
    cache = [A.PagedKVCache(x.kp, x.vp) for x in p]
    sq = [seqs(A, x, decode=True) for x in p]
    want = [A.attention_decode(cache[i], sq[i], p[i].q).clone() for i in range(3)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for n in range(60):
        with torch.cuda.stream(streams[n // 2 % 2]):
            got.append((n % 3, A.attention_decode(cache[n % 3], sq[n % 3], p[n % 3].q)))
        got.append(((n + 1) % 3, A.attention_decode(cache[(n + 1) % 3], sq[(n + 1) % 3], p[(n + 1) % 3].q,
                                                    stream=streams[n % 2])))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i]) for i, g in got)
    for x, w in zip(p, want):
        x.check(w, None, False)
