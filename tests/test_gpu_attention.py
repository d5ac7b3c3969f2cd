"""Attention operators on the GPU against the float64 oracle, element by element
within the bounds that attn_parity derives: append (norm, rotation, placement),
prompt, decode with a shared prefix, and a run of all of them around MoE
layers."""

import numpy as np
import pytest
import torch

import oracle
import synth
from attn_parity import DT, HALF, U, Problem, f64, seqs
from oracle import attention as oa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A(lib):
    from sparse_expert_ffn_gb300 import attention
    return attention


# ----------------------------------------------------------------- append

def _close(got, x, pos, freq, style, mscale, w, eps, dt):
    """Rows of a head tensor against the oracle's, within the derived bound."""
    y = oa.norm_rotate(x, pos, None, weight=w, eps=eps)
    want = oa.norm_rotate(x, pos, freq, style, mscale, w, eps)
    mag = np.abs(y)
    if freq is not None:
        half = len(freq)
        if style == "half":
            s = (mag[..., :half] + mag[..., half:2 * half]) * abs(mscale)
            mag[..., :half], mag[..., half:2 * half] = s, s
        else:
            s = (mag[..., 0:2 * half:2] + mag[..., 1:2 * half:2]) * abs(mscale)
            mag[..., 0:2 * half:2], mag[..., 1:2 * half:2] = s, s
    r = HALF[dt]
    tol = r * np.abs(want) + (1 + r) * 32 * U * mag
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           float((np.abs(got - want) / np.maximum(tol, 1e-30)).max()))


def _positions(p):
    return np.concatenate([np.arange(t - n, t) for n, t in p.lens]) if p.lens else np.zeros(0)


APPEND = [
    # lens, hq, hkv, d, dtype, page, layout, style, rot, scaling, norm, spare
    ([(1, 1)], 4, 1, 64, "bf16", 8, "heads", "half", 64, "none", True, 0),
    ([(1, 17), (1, 1), (1, 300)], 32, 8, 128, "bf16", 16, "heads", "half", 128, "none", False, 3),
    ([(5, 5), (0, 9), (31, 40), (1, 8)], 6, 2, 128, "bf16", 8, "rows", "interleaved", 128, "linear", True, 0),
    ([(40, 1000040), (3, 2000000003 - 1999990000)], 5, 5, 64, "fp32", 65536, "rows", "half", 48, "yarn", True, 0),
    ([(130, 131), (257, 257)], 8, 4, 128, "fp32", 64, "heads", "interleaved", 32, "ntk", False, 2),
    ([(200, 777)], 16, 16, 128, "bf16", 32, "rows", "half", 16, "yarn", True, 0),
    ([(170, 170), (9, 1033)], 7, 7, 64, "bf16", 256, "heads", "interleaved", 16, "none", True, 1),
    ([(160, 200)], 64, 1, 128, "bf16", 16, "heads", "half", 96, "none", True, 0),
    ([(33, 64)], 4, 2, 64, "fp32", 16, "heads", None, 0, "none", True, 0),
    ([(33, 64)], 4, 2, 64, "bf16", 16, "heads", None, 0, "none", False, 0),
]


@pytest.mark.parametrize("lens,hq,hkv,d,dtype,page,layout,style,rot,scaling,norm,spare", APPEND)
def test_append_places_rows(A, lens, hq, hkv, d, dtype, page, layout, style, rot, scaling, norm, spare):
    p = Problem(lens, hq, hkv, d, dtype, page, layout, spare=spare, seed=5)
    dev, dt = p.q.device, p.dt
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn(p.rows, hkv, d, generator=g).to(dt).to(dev) for _ in range(2))
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(dt).to(dev) if norm else None for _ in range(2)]
    freq, ms, rope = None, 1.0, None
    if style:
        f, ms = A.rope_frequencies(rot, 10000.0, scaling, 1.0 if scaling == "none" else 8.0)
        rope, freq = A.Rope(f.to(dev), style, ms), f.numpy()
    cache = A.PagedKVCache(p.kp, p.vp)
    before = [p.kp.clone(), p.vp.clone()]
    out = torch.full((p.rows, hq, d), 7.0, dtype=dt, device=dev)
    r = A.append_qkv(cache, seqs(A, p), p.q, k, v, rope=rope, q_norm=w[0], k_norm=w[1], eps=1e-5, q_out=out)
    torch.cuda.synchronize()
    assert r is out
    n, pos = int(p.start[-1]), _positions(p)
    _close(f64(out)[:n], f64(p.q)[:n], pos, freq, style, ms, None if not norm else f64(w[0]), 1e-5, dt)
    assert (out[n:] == 7.0).all()                             # rows behind the last sequence
    seq = np.repeat(np.arange(len(lens)), [x[0] for x in lens])
    pid = np.array([p.table_np[b, int(t) // page] for b, t in zip(seq, pos)], dtype=np.int64)
    off = pos.astype(np.int64) % page
    _close(f64(p.kp)[pid, :, off], f64(k)[:n], pos, freq, style, ms, None if not norm else f64(w[1]), 1e-5, dt)
    at = torch.from_numpy(pid).to(dev), torch.from_numpy(off).to(dev)
    assert torch.equal(p.vp[at[0], :, at[1]], v[:n])          # v's bits
    for now, was in zip((p.kp, p.vp), before):                # nothing else is written
        now = now.clone()
        now[at[0], :, at[1]] = was[at[0], :, at[1]]
        assert torch.equal(now, was)
    # no cache: the same rows
    q2, k2 = A.qk_norm_rope(A.Sequences(p.seq_start, p.kv_len), p.q, k, rope=rope, q_norm=w[0], k_norm=w[1], eps=1e-5,
                            q_out=torch.full_like(out, 7.0), k_out=torch.full_like(k, 3.0))
    assert torch.equal(q2, out) and torch.equal(k2[:n], p.kp[at[0], :, at[1]]) and (k2[n:] == 3.0).all()


def test_append_in_place_from_one_projection(A):
    """q, k, v as column ranges of one tensor, q rotated in place, one norm."""
    p = Problem([(20, 21), (3, 3)], 4, 2, 64, "bf16", 16, seed=3)
    x = torch.randn(23, 9 * 64, device="cuda:0").to(torch.bfloat16)
    q, k, v = (t.unflatten(1, (-1, 64)) for t in x.split([256, 128, 192], 1))
    v = v[:, :2]
    was = x.clone()
    f, ms = A.rope_frequencies(64)
    rope = A.Rope(f.cuda(), "half", ms)
    w = torch.full((64,), 0.5, dtype=torch.bfloat16, device="cuda:0")
    A.append_qkv(A.PagedKVCache(p.kp, p.vp), seqs(A, p), q, k, v, rope=rope, k_norm=w, q_out=q)
    pos = _positions(p)
    _close(f64(q), f64(was)[:, :256].reshape(23, 4, 64), pos, f.numpy(), "half", 1.0, None, 0, torch.bfloat16)
    assert torch.equal(x[:, 256:], was[:, 256:])
    pid = np.concatenate([p.table_np[0, (np.arange(1, 21)) // 16], p.table_np[1, [0, 0, 0]]])
    _close(f64(p.kp)[pid, :, pos % 16], f64(was)[:, 256:384].reshape(23, 2, 64), pos, f.numpy(), "half", 1.0,
           np.full(64, 0.5), 1e-6, torch.bfloat16)


def test_append_leaves_out_rows_without_a_place(A):
    """Positions before 0, pages that do not exist and lengths beyond the table
    store nothing; the queries are written all the same."""
    p = Problem([(6, 2), (4, 40), (4, 100)], 2, 2, 64, "bf16", 16, seed=4)
    p.table[1, 2] = -5                                         # positions 36 .. 39
    table = p.table[:, :5].contiguous()                        # 80 positions: 96 .. 99 are beyond
    k, v = (torch.randn(14, 2, 64, device="cuda:0").to(torch.bfloat16) for _ in range(2))
    before = p.kp.clone(), p.vp.clone()
    out = A.append_qkv(A.PagedKVCache(p.kp, p.vp), A.Sequences(p.seq_start, p.kv_len, table), p.q, k, v)
    assert torch.equal(out, p.q)
    page = int(p.table_np[0, 0])
    for now, was, new in zip((p.kp, p.vp), before, (k, v)):
        was[page, :, 0], was[page, :, 1] = new[4], new[5]      # positions 0 and 1 of sequence 0
        assert torch.equal(now, was)


# ----------------------------------------------------------------- prompt

PACKED = [
    ([(1, 1)], 1, 1, 64), ([(128, 128)], 4, 4, 128), ([(129, 129), (1, 1), (0, 0), (127, 127)], 2, 1, 64),
    ([(300, 300), (37, 37)], 6, 2, 128), ([(65, 65), (200, 200)], 7, 1, 128), ([(520, 520)], 8, 8, 64),
    ([(31, 31), (32, 32), (33, 33), (64, 64)], 32, 8, 128), ([(257, 257)], 5, 1, 64), ([(40, 40)], 64, 1, 64),
    ([(20, 20)], 128, 1, 64), ([(700, 700)], 3, 1, 128),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,hq,hkv,d", PACKED)
def test_prompt_packed(A, lens, hq, hkv, d, causal, dtype):
    p = Problem(lens, hq, hkv, d, dtype, 0, spare=2, seed=len(lens) + d)
    n = int(p.start[-1])
    p.k[n:], p.v[n:] = float("nan"), float("inf")              # rows of no sequence
    out = torch.full_like(p.q, 9.0)
    lse = torch.full((p.rows, hq), 9.0, device=p.q.device)
    A.attention_prompt(seqs(A, p, paged=False), p.q, p.k, p.v, causal=causal, out=out, lse=lse)
    torch.cuda.synchronize()
    p.check(out, lse, causal)
    assert (out[n:] == 9.0).all() and (lse[n:] == 9.0).all()


PAGED = [
    # lens, hq, hkv, d, page, layout
    ([(1, 1)], 4, 2, 128, 8, "heads"), ([(10, 210), (130, 130)], 8, 2, 128, 16, "heads"),
    ([(64, 300), (3, 517), (0, 40), (5, 5)], 4, 1, 64, 32, "rows"), ([(100, 1000)], 6, 3, 128, 64, "rows"),
    ([(129, 400), (1, 128), (2, 129)], 16, 16, 64, 128, "heads"), ([(33, 600)], 7, 1, 128, 256, "heads"),
    ([(50, 2000), (700, 700)], 2, 2, 64, 8, "rows"),
    ([(40, 25), (4, 0), (3, 2)], 4, 2, 64, 16, "heads"),       # fewer keys than rows: the first rows see none
    ([(16, 5000)], 8, 1, 128, 16, "heads"),                    # few rows far into a context
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,hq,hkv,d,page,layout", PAGED)
def test_prompt_paged(A, lens, hq, hkv, d, page, layout, causal, dtype):
    """Places of the cache that hold no key are NaN, entries behind a
    sequence's pages name pages that do not exist."""
    p = Problem(lens, hq, hkv, d, dtype, page, layout, seed=page + d, fill=float("nan"), spare=1)
    lse = torch.full((p.rows, hq), 9.0, device=p.q.device)
    out = A.attention_prompt_paged(A.PagedKVCache(p.kp, p.vp), seqs(A, p), p.q, causal=causal,
                                   out=torch.full_like(p.q, 9.0), lse=lse)
    torch.cuda.synchronize()
    p.check(out, lse, causal)
    assert (out[-1] == 9.0).all() and (lse[-1] == 9.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d,group,page", [(64, 1, 0), (128, 4, 0), (128, 7, 16), (64, 16, 64)])
def test_prompt_reads_every_key_once(A, d, group, page, dtype):
    """Equal scores and one-hot values: column c is the exact count of the seen
    keys that stand at c modulo d, over their number.  Weights are exactly 1 and
    sums exact, so only 1 / sum, the product and the output rounding are off."""
    lens = [(611, 611 if not page else 900), (130, 130)]
    p = Problem(lens, group, 1, d, dtype, page, seed=1)
    p.q.zero_()
    hot = torch.eye(d, device=p.q.device, dtype=p.dt)
    for b, (n, total) in enumerate(lens):
        for j in range(total):
            if page:
                p.vp[p.page_of(b, j), :, j % page] = hot[j % d]
            else:
                p.v[p.start[b] + j] = hot[j % d]
    lse = torch.empty(p.rows, group, device=p.q.device)
    if page:
        out = A.attention_prompt_paged(A.PagedKVCache(p.kp, p.vp), seqs(A, p), p.q, lse=lse)
    else:
        out = A.attention_prompt(seqs(A, p, paged=False), p.q, p.k, p.v, lse=lse)
    got, c = f64(out), np.arange(d)
    for b, (n, total) in enumerate(lens):
        for i in range(n):
            lim = total - n + i + 1
            want = ((lim - c + d - 1) // d) / lim
            row = p.start[b] + i
            assert (np.abs(got[row] - want) <= (HALF[p.dt] * (1 + 8 * U) + 8 * U) * want).all(), (b, i)
            assert (np.abs(lse[row].double().cpu().numpy() - np.log(lim)) <= 2.0 ** -22 * (1 + np.log(lim))).all()


def test_prompt_large_scores_and_rising_maxima(A):
    """Scores that rise along the keys (every tile has a new maximum), and ones
    whose weights underflow: against the oracle at the bound of their size."""
    p = Problem([(384, 384)], 2, 1, 64, "bf16", 0, seed=8)
    p.q[:] = 0
    p.q[..., 0] = 8.0
    p.k[:] = 0
    p.k[:, 0, 0] = (torch.arange(384, device="cuda:0") // 2).to(torch.bfloat16)
    out = torch.empty_like(p.q)
    lse = torch.empty(384, 2, device="cuda:0")
    A.attention_prompt(seqs(A, p, paged=False), p.q, p.k, p.v, scale=1.0, out=out, lse=lse)
    p.check(out, lse, True, scale=1.0)
    p.k[:, 0, 0] = -p.k[:, 0, 0]                               # falling: only the first keys count
    A.attention_prompt(seqs(A, p, paged=False), p.q, p.k, p.v, scale=1.0, out=out, lse=lse)
    p.check(out, lse, True, scale=1.0)


# ----------------------------------------------------------------- decode

DECODE = [
    # kv_len, hq, hkv, d, page, layout, prefix
    ([1], 1, 1, 64, 8, "heads", 0), ([0, 5, 16, 17], 8, 2, 128, 16, "heads", 0),
    ([1000, 1, 333], 32, 8, 128, 64, "rows", 0), ([4097], 7, 1, 128, 32, "heads", 0),
    ([200, 300, 1, 0, 129], 16, 16, 64, 128, "heads", 0), ([515] * 3, 24, 1, 64, 16, "rows", 0),
    ([777, 64], 64, 1, 128, 8, "heads", 0), ([90, 4000], 128, 1, 64, 256, "heads", 0),
    ([140, 129, 200, 128], 8, 2, 128, 16, "heads", 128), ([64, 300, 10, 0, 65], 4, 4, 64, 32, "rows", 64),
    ([2100 + i for i in range(40)], 8, 2, 128, 16, "heads", 2048), ([1030] * 5, 7, 1, 64, 8, "rows", 1024),
    ([700 + 3 * i for i in range(9)], 32, 1, 128, 64, "heads", 640), ([512, 512], 6, 2, 128, 256, "heads", 512),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kv,hq,hkv,d,page,layout,prefix", DECODE)
def test_decode(A, kv, hq, hkv, d, page, layout, prefix, dtype):
    p = Problem([(1, t) for t in kv], hq, hkv, d, dtype, page, layout, prefix=prefix, seed=prefix + d,
                fill=float("nan"), wide=5)
    lse = torch.full((p.rows, hq), 9.0, device=p.q.device)
    out = A.attention_decode(A.PagedKVCache(p.kp, p.vp), seqs(A, p, decode=True), p.q, prefix_len=prefix,
                             prefix_table=p.prefix_table if prefix else None, out=torch.full_like(p.q, 9.0), lse=lse)
    torch.cuda.synchronize()
    p.check(out, lse, False)
    # the prompt form of the same rows
    if not prefix:
        again = A.attention_prompt_paged(A.PagedKVCache(p.kp, p.vp), seqs(A, p), p.q)
        p.check(again, None, True)


def test_decode_prefix_equals_pages_named_by_every_sequence(A):
    """A shared prefix gives what the same pages in every row of the page table
    give, up to the order of the sums."""
    p = Problem([(1, 1500 + 7 * i) for i in range(12)], 16, 4, 128, "bf16", 32, prefix=1280, seed=2)
    cache, table = A.PagedKVCache(p.kp, p.vp), p.table.clone()
    table[:, :40] = p.prefix_table
    a = A.attention_decode(cache, seqs(A, p, decode=True), p.q, prefix_len=1280, prefix_table=p.prefix_table)
    b = A.attention_decode(cache, A.Sequences(None, p.kv_len, table), p.q)
    p.check(a, None, False)
    p.check(b, None, False)


# ------------------------------------------- strides, streams, graphs, sizes

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_inside_wider_tensors(A, dtype):
    p = Problem([(70, 70), (20, 20)], 4, 2, 64, dtype, 0, seed=6)
    qkv = torch.cat([p.q.flatten(1), p.k.flatten(1), p.v.flatten(1)], 1)
    q, k, v = (t.unflatten(1, (-1, 64)) for t in qkv.split([256, 128, 128], 1))
    wide = torch.full((90, 400), 5.0, dtype=p.dt, device=p.q.device)
    out = wide[:, 64:320].unflatten(1, (4, 64))
    A.attention_prompt(seqs(A, p, paged=False), q, k, v, out=out)
    p.check(out, None, True)
    assert (wide[:, :64] == 5.0).all() and (wide[:, 320:] == 5.0).all()


def test_page_id_out_of_range_reads_zeros(A):
    p = Problem([(1, 40), (1, 40)], 4, 2, 64, "bf16", 16, seed=7)
    ref = p.table.clone()
    p.table[0, 1], p.table[1, 1] = -1, 1 << 30
    cache = A.PagedKVCache(p.kp, p.vp)
    got = A.attention_decode(cache, seqs(A, p, decode=True), p.q)
    for b in range(2):
        p.kp[ref[b, 1].item()], p.vp[ref[b, 1].item()] = 0, 0
    want = A.attention_decode(cache, A.Sequences(None, p.kv_len, ref), p.q)
    assert torch.equal(got, want)
    one = A.attention_prompt_paged(cache, seqs(A, p), p.q)
    two = A.attention_prompt_paged(cache, A.Sequences(p.seq_start, p.kv_len, ref), p.q)
    assert torch.equal(one, two)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_offsets_beyond_32_bits(A, dtype):
    """Pages more than 2^31 elements into the cache, and a table that names them."""
    d, hkv, page, count = 128, 4, 64, 80000                    # 2.6e9 elements
    kp = torch.zeros(count, hkv, page, d, dtype=DT[dtype], device="cuda:0")
    vp = torch.zeros_like(kp)
    p = Problem([(1, 130), (150, 150)], 8, hkv, d, dtype, page, seed=9)
    far = count - 1 - torch.arange(p.kp.shape[0], device="cuda:0")
    kp[far], vp[far] = p.kp, p.vp
    table = torch.where(p.table < p.kp.shape[0], count - 1 - p.table, p.table)
    cache = A.PagedKVCache(kp, vp)
    sq = A.Sequences(p.seq_start, p.kv_len, table.int())
    p.check(A.attention_prompt_paged(cache, sq, p.q), None, True)
    one = A.Sequences(None, p.kv_len[:1].clone(), table[:1].int().contiguous())
    got = A.attention_decode(cache, one, p.q[:1])
    p.check(torch.cat([got, p.q[1:]]), None, True, rows=[0])
    k, v = (torch.randn(151, hkv, d, device="cuda:0").to(DT[dtype]) for _ in range(2))
    A.append_qkv(cache, sq, p.q, k, v)
    last = int(table[1, 149 // page])
    assert last * hkv * page * d > 1 << 31
    assert torch.equal(kp[last, :, 149 % page], k[150]) and torch.equal(vp[last, :, 149 % page], v[150])
    del kp, vp, cache
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_graph_replays_with_new_contents(A, dtype):
    """A decode step (append, attention over a shared prefix) and a prompt,
    captured once each and replayed with other lengths, tables and rows, in two
    graphs that share nothing but their inputs; the eager calls' bits."""
    p = Problem([(1, 300 + 50 * i) for i in range(6)], 8, 2, 128, dtype, 16, prefix=256, seed=11, wide=8)
    cache = A.PagedKVCache(p.kp, p.vp)
    f, ms = A.rope_frequencies(128)
    rope = A.Rope(f.cuda(), "half", ms)
    k, v = (torch.randn(6, 2, 128, device="cuda:0").to(p.dt) for _ in range(2))
    sq = seqs(A, p, decode=True)
    packed = Problem([(100, 100), (61, 61)], 8, 2, 128, dtype, 0, seed=12)
    psq = seqs(A, packed, paged=False)

    def step(out, lse):
        q = A.append_qkv(cache, sq, p.q, k, v, rope=rope)
        return A.attention_decode(cache, sq, q, prefix_len=256, prefix_table=p.prefix_table, out=out, lse=lse)

    def prompt(out):
        return A.attention_prompt(psq, packed.q, packed.k, packed.v, out=out)

    out, lse, pout = torch.empty_like(p.q), torch.empty(6, 8, device="cuda:0"), torch.empty_like(packed.q)
    step(out, lse), prompt(pout)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        step(out, lse)
    with torch.cuda.graph(g2):
        prompt(pout)
    for t in range(3):
        p.kv_len += torch.tensor([1, 0, 2, 1, 3, 1], dtype=torch.int32, device="cuda:0") * t
        p.q.copy_(torch.randn(p.q.shape, device="cuda:0"))
        packed.seq_start[1] = 100 - 17 * t
        out.fill_(1), pout.fill_(1)
        s2 = torch.cuda.Stream()
        s2.wait_stream(torch.cuda.current_stream())
        g1.replay()
        with torch.cuda.stream(s2):                            # both at once
            g2.replay()
        torch.cuda.current_stream().wait_stream(s2)
        torch.cuda.synchronize()
        a, b, c = out.clone(), lse.clone(), pout.clone()
        want, wl = torch.empty_like(out), torch.empty_like(lse)
        step(want, wl)
        assert torch.equal(a, want) and torch.equal(b, wl)
        assert torch.equal(c, prompt(torch.empty_like(pout)))


def test_two_streams_and_repeats_give_the_same_bits(A):
    p = Problem([(1, 3000 + 100 * i) for i in range(8)], 16, 4, 128, "bf16", 16, prefix=1024, seed=13)
    cache, sq = A.PagedKVCache(p.kp, p.vp), seqs(A, p, decode=True)
    packed = Problem([(300, 300), (500, 500)], 16, 4, 128, "bf16", 0, seed=14)
    psq = seqs(A, packed, paged=False)
    call = [lambda **kw: A.attention_decode(cache, sq, p.q, prefix_len=1024, prefix_table=p.prefix_table, **kw),
            lambda **kw: A.attention_prompt(psq, packed.q, packed.k, packed.v, **kw)]
    ref = [c() for c in call]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for s in streams:
            for i, c in enumerate(call):
                got.append((i, c(stream=s)))
    torch.cuda.synchronize()
    for i, t in got:
        assert torch.equal(t, ref[i])


def test_arguments_are_checked(A):
    p = Problem([(4, 4)], 4, 2, 64, "bf16", 16, seed=1)
    cache, sq = A.PagedKVCache(p.kp, p.vp), seqs(A, p)
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda:0")
    bad = [lambda: A.append_qkv(cache, sq, p.q.float(), k, k), lambda: A.append_qkv(cache, sq, p.q, k[:3], k),
           lambda: A.append_qkv(cache, sq, p.q, k, k.cpu()), lambda: A.append_qkv(cache, sq, p.q, k, k, q_norm=k[0, 0, :32]),
           lambda: A.attention_prompt_paged(cache, sq, p.q[:, :, :32]), lambda: A.attention_prompt(sq, p.q, k, k),
           lambda: A.attention_prompt(A.Sequences(p.seq_start), p.q, k, k[:, :1]),
           lambda: A.attention_decode(cache, sq, p.q), lambda: A.Sequences(p.seq_start.long()),
           lambda: A.Sequences(p.seq_start, p.kv_len, p.table[:, :1].expand(2, 1)), lambda: A.Sequences(),
           lambda: A.attention_decode(cache, A.Sequences(None, p.kv_len, p.table), p.q),
           lambda: A.attention_prompt_paged(cache, sq, p.q, lse=torch.zeros(4, 4, device="cuda:0").half()),
           lambda: A.PagedKVCache(p.kp, p.vp.transpose(1, 2)), lambda: A.Rope(torch.zeros(32, device="cuda:0")),
           lambda: A.attention_decode(cache, A.Sequences(None, p.kv_len, p.table), p.q[:1], prefix_len=32,
                                      prefix_table=p.table[0, :1].contiguous())]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(str(i))
    import sparse_expert_ffn_gb300 as sef
    with pytest.raises(sef.ColibriError):
        A.attention_prompt_paged(cache, sq, p.q, scale=0.0)
    assert A.attention_prompt_paged(cache, sq, p.q[:0]).shape == (0, 4, 64)


# ------------------------------------------------------------ all together

def test_decoder_block_prompt_then_tokens(lib, A):
    """Two pre-norm blocks, attention and MoE: two prompts of different lengths
    fill the cache, then five single-token steps.  Every append and every
    attention is compared with the oracle on the GPU's own inputs, and a prompt
    of the whole text gives the last token the same hidden state as the
    steps did, within bf16 rounding of two blocks."""
    sef = lib
    dev, d, hq, hkv, D, page, steps = torch.device("cuda:0"), 256, 4, 2, 64, 16, 5
    shape = synth.LayerShape("attn_block", d, 256, 4, 4, "bf16")   # every expert: no routing to flip
    g = torch.Generator().manual_seed(21)
    mat = lambda a, b: (torch.randn(a, b, generator=g) * a ** -0.5).to(torch.bfloat16).to(dev)  # noqa: E731
    blocks = []
    for layer in range(2):
        moe = sef.MoELayer(synth.router_weight(shape, 5, layer, dev), *synth.expert_weights(shape, 5, layer, dev),
                           shape.top_k, max_tokens=256)
        blocks.append((mat(d, (hq + 2 * hkv) * D), mat(hq * D, d), moe,
                       [(1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).to(dev) for _ in range(2)]))
    gamma = torch.ones(d, dtype=torch.bfloat16, device=dev)
    f, ms = A.rope_frequencies(D, 10000.0, "yarn", 4.0, trained=64)
    rope = A.Rope(f.to(dev), "half", ms)
    lens = [45, 70]
    text = [torch.randn(n + steps, d, generator=g).to(torch.bfloat16).to(dev) for n in lens]
    width = 6

    def model(hidden, caches, sq, single, record=None):
        for (wqkv, wo, moe, (qn, kn)), cache in zip(blocks, caches):
            x = hidden.float()
            u = (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)
            q, k, v = (t.unflatten(1, (-1, D)) for t in (u @ wqkv).split([hq * D, hkv * D, hkv * D], 1))
            qr = A.append_qkv(cache, sq, q, k, v, rope=rope, q_norm=qn, k_norm=kn)
            o = A.attention_decode(cache, sq, qr) if single else A.attention_prompt_paged(cache, sq, qr)
            if record is not None:
                record.append((q.clone(), k.clone(), qr, o, cache, qn, kn))
            hidden = (hidden.float() + (o.flatten(1) @ wo).float()).to(torch.bfloat16)
            moe.forward_stack_layer(hidden, gamma, 1e-6)
        return hidden

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    def new_caches():
        return [A.PagedKVCache.empty(2 * width, page, hkv, D, device=dev) for _ in range(2)]

    ids = np.random.default_rng(3).permutation(2 * width).reshape(2, width)
    table = ints(ids.tolist())

    def verify(record, pos, kv, seq):
        for q, k, qr, o, cache, qn, kn in record:
            _close(f64(qr), f64(q), pos, f.numpy(), "half", ms, f64(qn), 1e-6, torch.bfloat16)
            pid = ids[seq, pos // page]
            _close(f64(cache.k)[pid, :, pos % page], f64(k), pos, f.numpy(), "half", ms, f64(kn), 1e-6, torch.bfloat16)
            chk = Problem([(int((seq == b).sum()), kv[b]) for b in range(2)], hq, hkv, D, "bf16", page)
            chk.q, chk.kp, chk.vp, chk.table_np = qr, cache.k, cache.v, ids
            chk.check(o, None, True)

    caches = new_caches()
    start, kv = ints([0, lens[0], sum(lens)]), ints(lens)
    rec = []
    model(torch.cat([t[:n] for t, n in zip(text, lens)]), caches, A.Sequences(start, kv, table), False, rec)
    verify(rec, np.concatenate([np.arange(n) for n in lens]), lens, np.repeat([0, 1], lens))
    one = A.Sequences(None, kv, table)
    for s in range(steps):
        kv += 1                                                # the same tensor: read at every call
        rec = []
        h = model(torch.stack([t[n + s] for t, n in zip(text, lens)]), caches, one, True, rec)
        verify(rec, np.array([n + s for n in lens]), [n + s + 1 for n in lens], np.array([0, 1]))
    full = [n + steps for n in lens]
    again = model(torch.cat(text), new_caches(), A.Sequences(ints([0, full[0], sum(full)]), ints(full), table), False)
    last = again[[full[0] - 1, sum(full) - 1]]
    # the same mathematics through other kernels: both sides round hidden states
    # to bf16 (2^-8) four times, and every such difference passes the later
    # products
    diff = (last.float() - h.float()).norm(dim=1) / h.float().norm(dim=1)
    assert (diff <= 16 * 2.0 ** -8).all(), diff.tolist()
    for b in blocks:
        assert b[2].check() == sef.OK
        b[2].close()
