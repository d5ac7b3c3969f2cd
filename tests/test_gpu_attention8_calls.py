"""Calls of the 8-bit cache at the ends of what is allowed (arrays that hold anything,
offsets past 32 bits, idle batches, threads, streams, waits that give up), and rotary
positions of several axes in 16 and 32 bits."""

import threading

import numpy as np
import pytest
import torch

from attn8_parity import CODE, Problem8, decoded, same
from attn_parity import DT, HALF, U, Problem, f64, seqs
from oracle import attention as oa

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def A(lib):
    from sparse_expert_ffn_gb300 import attention
    return attention


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------- axes

AXES = [
    # sections, interleaved, style, rot, d, dtype, page, norm
    ([16, 24, 24], False, "half", 128, 128, "bf16", 16, True), ([16, 24, 24], True, "interleaved", 128, 128, "bf16", 0, False),
    ([4, 2, 1, 1], True, "half", 16, 64, "fp32", 8, False), ([32], False, "half", 64, 64, "bf16", 64, True),
    ([10, 0, 14], False, "interleaved", 48, 64, "fp32", 0, True), ([3] * 8, True, "half", 48, 128, "bf16", 32, False),
]


@pytest.mark.parametrize("sections,interleaved,style,rot,d,dtype,page,norm", AXES)
def test_positions_of_several_axes(A, sections, interleaved, style, rot, d, dtype, page, norm):
    lens, hq, hkv = [(37, 60), (1, 9), (0, 3), (70, 70)], 6, 3
    p = Problem(lens, hq, hkv, d, dtype, page or 16, spare=2, seed=3)
    dev, n, axes = p.q.device, 108, len(sections)
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(p.rows, hkv, d, generator=g).to(p.dt).to(dev) for _ in range(2))
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(p.dt).to(dev) if norm else None for _ in range(2)]
    which = A.rope_axes(sections, interleaved)
    f, ms = A.rope_frequencies(rot, 10000.0, "yarn", 4.0)
    # far ones, negative ones, and axes that are rows of a wider tensor
    store = torch.randint(-2 ** 31, 2 ** 31 - 1, (axes, p.rows + 5), generator=g, dtype=torch.int64).to(torch.int32)
    store[:, ::2] %= 4000
    positions = store.to(dev)[:, 2:2 + p.rows]
    at = store[:, 2:2 + n].numpy()[which.long().numpy()].T
    rope = A.Rope(f.to(dev), style, ms, axes=which.to(dev))
    out = torch.full_like(p.q, 7.0)
    sq = seqs(A, p)
    before = p.kp.clone()
    args = dict(rope=rope, positions=positions, q_norm=w[0], k_norm=w[1], eps=1e-5, q_out=out)
    if page:
        A.append_qkv(A.PagedKVCache(p.kp, p.vp), sq, p.q, k, v, **args)
        seq = np.repeat(np.arange(4), [x[0] for x in lens])
        place = np.concatenate([np.arange(t - m, t) for m, t in lens])
        pid = np.array([p.table_np[b, t // page] for b, t in zip(seq, place)], dtype=np.int64)
        got_k = f64(p.kp)[pid, :, place % page]
        there = torch.zeros(p.kp.shape[0], page, dtype=torch.bool)
        there[pid, place % page] = True
        untouched = ~there[:, None, :, None].to(dev).expand_as(p.kp)
        assert torch.equal(p.kp[untouched], before[untouched])
    else:
        k_out = torch.full_like(k, 3.0)
        A.qk_norm_rope(A.Sequences(p.seq_start, p.kv_len), p.q, k, k_out=k_out, **args)
        got_k = f64(k_out)[:n]
        assert (k_out[n:] == 3.0).all()
    assert (out[n:] == 7.0).all()
    r, half = HALF[p.dt], rot // 2
    # the angle: 2^-32 turn and t (f 2^-55 + 2^-64) turns off before it is rounded
    slack = 2 * np.pi * (2.0 ** -32 + np.abs(at) * (f.numpy() * 2.0 ** -55 + 2.0 ** -64)) * ms
    for got, x, wx in ((f64(out)[:n], f64(p.q)[:n], w[0]), (got_k, f64(k)[:n], w[1])):
        wx = None if wx is None else f64(wx)
        y = oa.norm_rotate(x, at, None, weight=wx, eps=1e-5)
        # (positions in longdouble: at 2^31 a float64 angle is off by as much)
        two_pi = np.longdouble("6.28318530717958647692528676655900577")
        angle = (at.astype(np.longdouble) * f.numpy().astype(np.longdouble)) % two_pi
        want = oa.norm_rotate(x, (angle / f.numpy()).astype(np.float64), f.numpy(), style, ms, wx, 1e-5)
        mag, off = np.abs(y), np.zeros_like(y)
        sl = (slice(0, half), slice(half, 2 * half)) if style == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
        both = mag[..., sl[0]] + mag[..., sl[1]]
        mag[..., sl[0]], mag[..., sl[1]] = both * ms, both * ms
        off[..., sl[0]], off[..., sl[1]] = both * slack[:, None], both * slack[:, None]
        tol = r * np.abs(want) + (1 + r) * (32 * U * mag + off)
        assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / np.maximum(tol, 1e-30)).max())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_axes_that_agree_are_plain_positions(A, dtype):
    """The positions that follow from the lengths, given on every axis: the same bits; so
    are axis numbers past the last axis, and one axis without a map."""
    p = Problem([(33, 80), (5, 5)], 4, 2, 64, dtype, 16, seed=6)
    k = torch.randn(38, 2, 64, device="cuda").to(p.dt)
    f = A.rope_frequencies(64)[0].cuda()
    at = torch.cat([torch.arange(47, 80), torch.arange(5)]).to(torch.int32).cuda()
    sq = A.Sequences(p.seq_start, p.kv_len)
    ref = A.qk_norm_rope(sq, p.q, k, rope=A.Rope(f))
    for axes, pos in ((A.rope_axes([10, 12, 10]).cuda(), at.repeat(3, 1)), (None, at), (None, at.repeat(2, 1)),
                      (A.rope_axes([10, 12, 10]).cuda(), at.expand(3, -1)),
                      (torch.full((32,), 255, dtype=torch.uint8, device="cuda"), torch.stack([at + 9, at]))):
        got = A.qk_norm_rope(sq, p.q, k, rope=A.Rope(f, axes=axes), positions=pos)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


# ------------------------------------------------------------------ 8 bits

def test_arrays_that_hold_anything(A):
    """Whatever seq_start, kv_len, the tables, scales and codes hold, nothing outside the
    outputs and the cache is written, and the next calls are right."""
    r = np.random.default_rng(6)
    p = Problem8([(50, 90), (70, 70), (30, 200)], 8, 2, 64, "e4m3", 16, 32, spare=10, seed=7, wide=3)
    ref = A.attention_prompt_paged(p.cache(A), seqs(A, p), p.q, out=torch.zeros_like(p.q))
    guard = torch.full((p.rows + 64, 8, 64), 3.0, dtype=p.dt, device="cuda:0")
    out = guard[32:-32]
    edge = np.array([-2 ** 31, -1, 0, 1, 49, 120, 160, 2 ** 30, 2 ** 31 - 1], dtype=np.int64)
    k, v = (torch.randn(p.rows, 2, 64, device="cuda:0").to(p.dt) for _ in range(2))
    one = torch.zeros(3, 8, 64, dtype=p.dt, device="cuda:0")
    pages = p.kc.shape[0]
    # codes and scales inside larger tensors, whose rest must stay as it is
    big = [torch.full((pages + 2, 2, 32, 64), 0x33, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scl = [torch.full((pages + 2, 2, 2), 5.0, device="cuda") for _ in range(2)]
    for trial in range(30):
        junk = A.Sequences(*(torch.from_numpy(r.choice(edge, s).astype(np.int32)).cuda()
                             for s in ((4,), (3,), (3, p.table.shape[1]))))
        for b, s in zip(big, scl):
            b[1:-1] = torch.randint(0, 256, b[1:-1].shape, dtype=torch.uint8, device="cuda")
            s[1:-1] = torch.randn(pages, 2, 2, device="cuda") * 1e30
        store = A.PagedKVCache8(*(b[1:-1].view(CODE["e4m3" if trial % 3 else "int8"]) for b in big), *(s[1:-1] for s in scl))
        rope = A.Rope(A.rope_frequencies(64)[0].cuda())
        positions = torch.from_numpy(r.choice(edge, (2, p.rows)).astype(np.int32)).cuda()
        A.append_qkv(store, junk, p.q, k, v, rope=rope, q_out=out, positions=positions if trial & 2 else None)
        A.attention_prompt_paged(store, junk, p.q, causal=bool(trial & 1), out=out)
        few = A.Sequences((junk.seq_start.clamp(max=5)), junk.kv_len, junk.page_table)
        A.attention_prompt_paged(store, few, p.q[:6], causal=bool(trial & 1), out=out[:6])
        A.attention_decode(store, A.Sequences(None, junk.kv_len, junk.page_table), one, prefix_len=32,
                           prefix_table=junk.page_table[0, :1].contiguous())
        store.values(junk.page_table.flatten())
        torch.cuda.synchronize()
        assert (guard[:32] == 3.0).all() and (guard[-32:] == 3.0).all()
        for b, s in zip(big, scl):
            assert (b[0] == 0x33).all() and (b[-1] == 0x33).all() and (s[0] == 5).all() and (s[-1] == 5).all()
    assert torch.equal(A.attention_prompt_paged(p.cache(A), seqs(A, p), p.q, out=torch.zeros_like(p.q)), ref)
    assert A.check() == 0


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_offsets_beyond_32_bits(A, code):
    """Pages more than 2^32 bytes into the cache, and a table that names them."""
    d, hkv, page, count = 128, 4, 64, 140000                   # 4.6e9 bytes each
    p = Problem8([(1, 130), (150, 150)], 8, hkv, d, code, 16, page, seed=9)
    raw = [torch.zeros(count, hkv, page, d, dtype=torch.uint8, device="cuda:0") for _ in range(2)]
    scale = [torch.zeros(count, hkv, page // 16, device="cuda:0") for _ in range(2)]
    far = count - 1 - torch.arange(p.kc.shape[0], device="cuda:0")
    for x, s, c, cs in zip(raw, scale, (p.kc, p.vc), (p.ks, p.vs)):
        x[far], s[far] = c.view(torch.uint8), cs
    table = torch.where(p.table < p.kc.shape[0], count - 1 - p.table, p.table).int()
    cache = A.PagedKVCache8(raw[0].view(CODE[code]), raw[1].view(CODE[code]), *scale)
    sq = A.Sequences(p.seq_start, p.kv_len, table)
    p.check(A.attention_prompt_paged(cache, sq, p.q), None, True)
    one = A.Sequences(None, p.kv_len[:1].clone(), table[:1].contiguous())
    p.check(torch.cat([A.attention_decode(cache, one, p.q[:1]), p.q[1:]]), None, True, rows=[0])
    few = A.Sequences(ints(0, 3), p.kv_len[:1].clone(), table[:1].contiguous())
    got = A.attention_prompt_paged(cache, few, p.q[:1].expand(3, -1, -1).contiguous())
    p.check(torch.cat([got[2:], p.q[1:]]), None, True, rows=[0])
    k, v = (torch.randn(151, hkv, d, device="cuda:0").to(BF) for _ in range(2))
    A.append_qkv(cache, sq, p.q, k, v)
    last = int(table[1, 149 // page])
    assert last * hkv * page * d > 1 << 32
    for x, s, new in ((raw[0], scale[0], k), (raw[1], scale[1], v)):
        want = oa.nearest_code(f64(new)[150] / f64(s)[last, :, 149 % page // 16, None], code)
        assert np.array_equal(decoded(x[last, :, 149 % page].view(CODE[code])), want)
    kv, _ = cache.values(ints(last))
    assert torch.equal(kv[0, :, 149 % page].float(), raw[0][last, :, 149 % page].view(CODE[code]).float() *
                       scale[0][last, :, 149 % page // 16, None])
    del raw, scale, cache
    torch.cuda.empty_cache()


@pytest.mark.parametrize("d", [64, 128])
def test_stalled_copies_give_nan_rows(A, monkeypatch, d):
    p = Problem8([(200, 300), (9, 90)], 4, 2, d, "e4m3", 16, 32, spare=3, seed=1)
    cache, sq = p.cache(A), seqs(A, p)
    ref = A.attention_prompt_paged(cache, sq, p.q)
    dec = Problem8([(1, 1300 + i) for i in range(5)], 8, 2, d, "int8", 16, 16, prefix=1024, seed=2)
    dcache, dsq = dec.cache(A), seqs(A, dec, decode=True)
    args = dict(prefix_len=1024, prefix_table=dec.prefix_table)
    dref = A.attention_decode(dcache, dsq, dec.q, **args)
    torch.cuda.synchronize()
    assert A.check() == 0
    monkeypatch.setenv("COLIBRI_WAIT_LIMIT_NS", "20000000")
    monkeypatch.setenv("COLIBRI_TEST_STALL_TMA", "1")
    out, lse = torch.zeros_like(p.q), torch.zeros(p.rows, 4, device="cuda:0")
    A.attention_prompt_paged(cache, sq, p.q, out=out, lse=lse)
    dout = A.attention_decode(dcache, dsq, dec.q, **args)
    torch.cuda.synchronize()
    monkeypatch.delenv("COLIBRI_WAIT_LIMIT_NS")
    monkeypatch.delenv("COLIBRI_TEST_STALL_TMA")
    assert out[:209].isnan().all() and lse[:209].isnan().all()
    assert (out[209:] == 0).all() and (lse[209:] == 0).all()
    assert dout.isnan().all() and A.check() != 0 and A.check() == 0
    assert torch.equal(A.attention_prompt_paged(cache, sq, p.q)[:209], ref[:209])
    assert torch.equal(A.attention_decode(dcache, dsq, dec.q, **args), dref)


def test_rows_of_a_cta_that_gives_up_in_the_middle(A, monkeypatch):
    """Copies that stop at a CTA's second item: its rows are NaN or right, none is left."""
    p = Problem8([(600, 700)] * 6, 32, 8, 128, "int8", 32, 64, seed=3)
    cache, sq = p.cache(A), seqs(A, p)
    ref = A.attention_prompt_paged(cache, sq, p.q)
    monkeypatch.setenv("COLIBRI_WAIT_LIMIT_NS", "20000000")
    monkeypatch.setenv("COLIBRI_TEST_STALL_TMA", "2")
    out = A.attention_prompt_paged(cache, sq, p.q, out=torch.full_like(p.q, 77.0))
    torch.cuda.synchronize()
    monkeypatch.delenv("COLIBRI_WAIT_LIMIT_NS")
    monkeypatch.delenv("COLIBRI_TEST_STALL_TMA")
    gone = out.isnan().all(-1)
    assert gone.any() and A.check() != 0
    assert torch.equal(out[~gone], ref[~gone])
    assert torch.equal(A.attention_prompt_paged(cache, sq, p.q), ref)


def test_scores_that_are_not_numbers(A):
    """A NaN or infinite query makes its own rows NaN and no other; a block whose scale of
    keys is NaN, the rows that see it."""
    p = Problem8([(1, 700), (1, 40), (1, 700), (1, 1300)], 4, 1, 64, "e4m3", 16, 16, seed=3)
    cache, sq = p.cache(A), seqs(A, p, decode=True)
    ref = A.attention_decode(cache, sq, p.q)
    q = p.q.clone()
    q[0, 1] = float("nan")
    q[2, 3, 5] = float("inf")
    lse = torch.empty(4, 4, device="cuda:0")
    got = A.attention_decode(cache, sq, q, lse=lse)
    hit = torch.zeros(4, 4, dtype=torch.bool, device="cuda:0")
    hit[0, 1] = hit[2, 3] = True
    assert got[hit].isnan().all() and lse[hit].isnan().all() and torch.equal(got[~hit], ref[~hit])
    for lens, n in (([(300, 300)], 176), ([(20, 300)], 0), ([(200, 400)], 0)):
        pr = Problem8(lens, 4, 1, 64, "int8", 16, 16, seed=4)
        psq = seqs(A, pr)
        ref = A.attention_prompt_paged(pr.cache(A), psq, pr.q)
        pr.ks[pr.page_of(0, 176)] = float("nan")               # keys 176 .. 191
        got = A.attention_prompt_paged(pr.cache(A), psq, pr.q)
        assert torch.equal(got[:n], ref[:n]) and got[n:].isnan().all()


def test_large_equal_and_rising_scores(A):
    """Scores that rise along the keys (every step moves the reference), fall, and are all
    equal, and value scales far apart."""
    for single in (True, False):
        lens = [(1, 900)] if single else [(150, 900)]
        for kind in ("rising", "falling", "equal", "scales"):
            p = Problem8(lens, 2, 1, 64, "int8", 16, 16, seed=8, pow2=True)
            p.q[:] = 0
            p.q[..., 0] = 8.0
            for j in range(0, 900, 16):
                pid = p.page_of(0, j)
                p.kc[pid, 0, :, 0] = 3 if kind == "equal" else j // 16
                p.ks[pid] = 0.5
                if kind == "scales":
                    p.vs[pid] = 2.0 ** (j // 16 % 40 - 20)
            if kind == "falling":
                p.kc[:, :, :, 0] = -p.kc[:, :, :, 0]
            lse = torch.empty(p.rows, 2, device="cuda")
            if single:
                p.check(A.attention_decode(p.cache(A), seqs(A, p, decode=True), p.q, scale=1.0, lse=lse), lse, False, 1.0)
            p.check(A.attention_prompt_paged(p.cache(A), seqs(A, p), p.q, scale=1.0, lse=lse), lse, True, 1.0)


def test_batches_of_padding_and_of_nothing(A):
    p = Problem8([(4, 20), (3, 9)], 4, 2, 64, "e4m3", 16, 16, seed=1)
    cache = p.cache(A)
    olds = [x.clone() for x in (p.kc, p.ks, p.vc, p.vs)]
    empty = A.Sequences(ints(0), ints(), torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    k = torch.randn(7, 2, 64, device="cuda").to(BF)
    out = torch.full_like(p.q, 9.0)
    A.append_qkv(cache, empty, p.q, k, k, q_out=out)
    A.attention_prompt_paged(cache, empty, p.q, out=out)
    for b in (0, 1):                                           # no rows at all
        sq = A.Sequences(ints(0, 0, 0), p.kv_len, p.table)
        A.append_qkv(cache, sq, p.q, k, k, q_out=out)
        A.attention_prompt_paged(cache, sq, p.q[:7 * b], out=out[:7 * b])
    none = A.Sequences(None, ints(), torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert A.attention_decode(cache, none, p.q[:0]).shape == (0, 4, 64)
    assert cache.values(ints())[0].shape == (0, 2, 16, 64)
    torch.cuda.synchronize()
    assert (out == 9.0).all()
    for now, was in zip((p.kc, p.ks, p.vc, p.vs), olds):
        assert same(now, was) if now.element_size() == 1 else torch.equal(now.nan_to_num(2.0), was.nan_to_num(2.0))


@pytest.mark.parametrize("count,rows", [(130, 1), (300, 0), (300, 1), (40, 3), (33, 7)])
def test_batches_of_many_sequences(A, count, rows):
    """Work lists past 32 and 128 sequences: single tokens (rows 0), and drafts whose rows
    run in equal shares (up to 32 rows times heads of a group each, 1024 in all) or not."""
    r = np.random.default_rng(count)
    kv = r.integers(1, 90, count)
    kv[r.integers(0, count, 5)] = 0
    kv[7] = 3000
    p = Problem8([(max(rows, 1), int(t)) for t in kv], 3 if rows != 7 else 8, 1, 64, "e4m3" if count % 2 else "int8", 16, 16,
                 spare=2 if rows else 0, seed=count)
    lse = torch.full((p.rows, p.hq), 9.0, device="cuda")
    out = torch.full_like(p.q, 9.0)
    if rows:
        A.attention_prompt_paged(p.cache(A), seqs(A, p), p.q, out=out, lse=lse)
        assert (out[-2:] == 9.0).all() and (lse[-2:] == 9.0).all()
    else:
        A.attention_decode(p.cache(A), seqs(A, p, decode=True), p.q, out=out, lse=lse)
    p.check(out, lse, bool(rows))


def test_threads_streams_and_repeats_give_the_same_bits(A):
    p = Problem8([(1, 300 + 17 * i) for i in range(30)], 16, 4, 128, "e4m3", 32, 32, seed=5)
    few = Problem8([(4, 500 + 31 * i) for i in range(9)], 8, 2, 64, "int8", 16, 16, seed=6)
    long = Problem8([(170, 900), (90, 90)], 8, 2, 128, "int8", 64, 64, seed=7)

    def calls():
        return (A.attention_decode(p.cache(A), seqs(A, p, decode=True), p.q),
                A.attention_prompt_paged(few.cache(A), seqs(A, few), few.q),
                A.attention_prompt_paged(long.cache(A), seqs(A, long), long.q))

    ref = calls()
    torch.cuda.synchronize()
    bad = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = calls()
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(x, y) for x, y in zip(got, ref)):
                    bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    s = torch.cuda.Stream()
    got = A.attention_prompt_paged(few.cache(A), seqs(A, few), few.q, stream=s)
    s.synchronize()
    assert torch.equal(got, ref[1])


def test_steps_behind_each_other_see_what_was_just_written(A):
    """100 steps of append and attention without a wait, eagerly and in a graph, over a
    shared prefix: the bits of steps that are waited for."""
    hq, hkv, d, page = 8, 2, 128, 16
    g = torch.Generator().manual_seed(3)
    prefix = Problem8([(1, 256)], hq, hkv, d, "e4m3", 16, page, seed=1, pow2=True)
    n = prefix.kc.shape[0]

    def fresh():
        c = A.PagedKVCache8.empty(n + 40, page, hkv, d, 16)
        for t, o in ((c.k, prefix.kc), (c.v, prefix.vc)):
            t.view(torch.uint8).zero_()
            t.view(torch.uint8)[:n] = o.view(torch.uint8)
        for t, o in ((c.k_scale, prefix.ks), (c.v_scale, prefix.vs)):
            t.zero_()
            t[:n] = o
        return c

    own = torch.arange(n, n + 40, device="cuda").to(torch.int32).view(4, 10)
    table = torch.cat([torch.zeros(4, 16, dtype=torch.int32, device="cuda"), own], 1).contiguous()
    rows = [[torch.randn(4, h, d, generator=g).cuda().to(BF) for h in (hq, hkv, hkv)] for _ in range(100)]
    kv, begin = torch.empty(4, dtype=torch.int32, device="cuda"), ints(256, 260, 270, 300)
    sq = A.Sequences(None, kv, table)
    where = torch.from_numpy(prefix.table_np[0, :16].copy()).cuda()

    def steps(c, wait):
        kv.copy_(begin)
        outs = []
        for q, k, v in rows:
            kv.add_(1)
            outs.append(A.attention_decode(c, sq, A.append_qkv(c, sq, q, k, v), prefix_len=256, prefix_table=where))
            if wait:
                torch.cuda.synchronize()
        return outs

    ref_cache, c = fresh(), fresh()
    ref, got = steps(ref_cache, True), steps(c, False)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, got)) and same(c.k, ref_cache.k)
    assert torch.equal(c.v_scale.nan_to_num(3.0), ref_cache.v_scale.nan_to_num(3.0))
    c = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = steps(c, False)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, got))
