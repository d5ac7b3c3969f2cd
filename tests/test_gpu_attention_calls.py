"""Attention operators in calls at the ends of what their documentation allows."""

import ctypes
import os

import numpy as np
import pytest
import torch

import synth
from attn_parity import HALF, U, Problem, f64, seqs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A(lib):
    from sparse_expert_ffn_gb300 import attention
    return attention


def _bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d,rot,style", [(64, 32, "half"), (64, 48, "interleaved"), (128, 16, "half"),
                                         (128, 112, "interleaved"), (64, 0, None), (128, 0, None)])
def test_elements_that_are_not_rotated_are_copied(A, d, rot, style, dtype):
    """Elements from rot_dim on, and all of them without a rope: the input's bits,
    whatever stands beside them (infinities, zeros with a sign)."""
    p = Problem([(37, 50), (9, 9)], 6, 3, d, dtype, 16, seed=d + rot)
    dev, g = p.q.device, torch.Generator().manual_seed(5)
    k, v = (torch.randn(p.rows, 3, d, generator=g).to(p.dt).to(dev) for _ in range(2))
    rope = A.Rope(A.rope_frequencies(rot)[0].to(dev), style, 1.0) if style else None
    plain = [x.clone() for x in (p.q, k)]
    for x in (p.q, k):
        special = torch.tensor([float("inf"), -float("inf"), 0.0, -0.0, 3.0], dtype=p.dt)
        at = torch.randint(0, 5, (p.rows, x.shape[1], d - rot), generator=g)
        hit = torch.rand(at.shape, generator=g).to(dev) < 0.4
        x[..., rot:] = torch.where(hit, special[at].to(dev), x[..., rot:])
    sq = A.Sequences(p.seq_start, p.kv_len)
    want = A.qk_norm_rope(sq, *plain, rope=rope)                   # the rotated part knows no other elements
    got = A.qk_norm_rope(sq, p.q, k, rope=rope)
    cache = A.PagedKVCache(p.kp, p.vp)
    got_q = A.append_qkv(cache, seqs(A, p), p.q, k, v, rope=rope)
    for x, y, z in zip(got, (p.q, k), want):
        assert torch.equal(_bits(x[..., rot:]), _bits(y[..., rot:]))
        assert torch.equal(_bits(x[..., :rot]), _bits(z[..., :rot]))
    assert torch.equal(_bits(got_q), _bits(got[0]))
    for b, (n, total) in enumerate(p.lens):
        for i in (0, n // 2, n - 1):
            t = total - n + i
            assert torch.equal(_bits(cache.k[p.page_of(b, t), :, t % 16]), _bits(got[1][int(p.start[b]) + i]))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_batch_of_padding(A, dtype):
    """No sequence and a few padded rows: nothing is written anywhere."""
    p = Problem([(5, 5)], 4, 2, 64, dtype, 16, seed=1)
    dev = p.q.device
    ints = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=dev)  # noqa: E731
    cache, sq = A.PagedKVCache(p.kp, p.vp), A.Sequences(ints(1), ints(0), ints(0, 7))
    before = p.kp.clone(), p.vp.clone()
    k, out = p.q[:, :2].contiguous(), torch.full_like(p.q, 3.0)
    lse = torch.full((5, 4), 3.0, device=dev)
    assert A.append_qkv(cache, sq, p.q, k, k, q_out=out) is out
    assert A.attention_prompt_paged(cache, sq, p.q, out=out, lse=lse) is out
    A.attention_prompt(A.Sequences(ints(1)), p.q, k, k, out=out, lse=lse)
    A.qk_norm_rope(sq, p.q, k, q_out=out, k_out=torch.full_like(k, 3.0))
    empty = A.Sequences(None, ints(0), ints(0, 7))
    assert A.attention_decode(cache, empty, p.q[:0]).shape == (0, 4, 64)
    assert (out == 3.0).all() and (lse == 3.0).all()
    assert torch.equal(p.kp, before[0]) and torch.equal(p.vp, before[1])


def test_errors_of_other_calls_are_not_reported(lib, A):
    """An init that asks for more memory than there is (550 GB of expert weights)
    returns OOM, once: calls after it, of other handles and without one, are fine."""
    sef = lib
    shape = synth.LayerShape("small", 128, 128, 4, 2, "bf16")
    moe = sef.MoELayer(synth.router_weight(shape, 1, 0, "cuda:0"), *synth.expert_weights(shape, 1, 0, "cuda:0"), 2,
                       max_tokens=16)
    x = torch.randn(16, 128, device="cuda:0").to(torch.bfloat16)
    want = moe.forward(x).clone()
    p = Problem([(40, 40)], 4, 2, 64, "bf16", 0, seed=2)
    sq = seqs(A, p, paged=False)
    ref = A.attention_prompt(sq, p.q, p.k, p.v)
    torch.cuda.synchronize()
    cfg = sef.ColibriConfig(d_model=16384, d_ff=32768, n_experts=256, top_k=2, max_tokens=16, dtype=sef.DTYPE_BF16,
                            device=0)
    h, there = ctypes.c_void_p(), ctypes.c_void_p(x.data_ptr())
    assert sef.colibri_init(ctypes.byref(cfg), there, None, there, there, there, 1, ctypes.byref(h)) == 2
    assert torch.equal(A.attention_prompt(sq, p.q, p.k, p.v), ref)
    assert sef.colibri_init(ctypes.byref(cfg), there, None, there, there, there, 1, ctypes.byref(h)) == 2
    assert torch.equal(moe.forward(x), want)
    assert moe.check() == sef.OK
    moe.close()


def test_the_environment_is_not_read_by_calls(lib, A):
    """A variable that another thread's setenv puts into the process's environment
    (not into os.environ, which the binding looks at) changes nothing."""
    p = Problem([(200, 200), (9, 9)], 4, 2, 64, "bf16", 0, seed=1)
    sq = seqs(A, p, paged=False)
    ref = A.attention_prompt(sq, p.q, p.k, p.v)
    os.putenv("COLIBRI_WAIT_LIMIT_NS", "20000000")
    os.putenv("COLIBRI_TEST_STALL_TMA", "1")
    try:
        got = A.attention_prompt(sq, p.q, p.k, p.v)
        torch.cuda.synchronize()
    finally:
        os.unsetenv("COLIBRI_WAIT_LIMIT_NS")
        os.unsetenv("COLIBRI_TEST_STALL_TMA")
    assert torch.equal(got, ref)


@pytest.mark.parametrize("decode", [False, True])
def test_waits_that_gave_up_are_reported(lib, A, monkeypatch, decode):
    """Rows of NaN from a wait that gave up come with a status, which is reported
    once; NaN that was in the inputs does not."""
    sef = lib
    p = Problem([(1, 1300 + i) for i in range(5)], 8, 2, 64, "bf16", 16, prefix=1024, seed=2)
    cache = A.PagedKVCache(p.kp, p.vp)
    sq = seqs(A, p, decode=True)
    packed = Problem([(150, 150)], 8, 2, 64, "bf16", 0, seed=3)
    psq = seqs(A, packed, paged=False)

    def call():
        if decode:
            return A.attention_decode(cache, sq, p.q, prefix_len=1024, prefix_table=p.prefix_table)
        return A.attention_prompt(psq, packed.q, packed.k, packed.v)

    A.check()                                                      # (what an earlier test left)
    ref = call()
    assert A.check() == sef.OK
    monkeypatch.setenv("COLIBRI_WAIT_LIMIT_NS", "20000000")
    monkeypatch.setenv("COLIBRI_TEST_STALL_TMA", "1")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bad = call()
    assert A.check(stream=side) == sef.ERR_TIMEOUT and bad.isnan().all()
    monkeypatch.delenv("COLIBRI_WAIT_LIMIT_NS")
    monkeypatch.delenv("COLIBRI_TEST_STALL_TMA")
    assert A.check() == sef.OK and A.check(device="cuda") == sef.OK
    assert torch.equal(call(), ref) and A.check() == sef.OK
    p.q.fill_(float("nan")), packed.q.fill_(float("nan"))
    assert call().isnan().all() and A.check() == sef.OK


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_results_between_the_columns_of_the_inputs(A, dtype):
    """q, k, v and the output as column ranges of one tensor's rows."""
    p = Problem([(150, 150), (40, 40)], 4, 2, 64, dtype, 0, seed=6)
    wide = torch.full((190, 896), 5.0, dtype=p.dt, device=p.q.device)
    q, o, k, v = (wide[:, a:b].unflatten(1, (-1, 64)) for a, b in ((0, 256), (256, 512), (576, 704), (768, 896)))
    q.copy_(p.q), k.copy_(p.k), v.copy_(p.v)
    was = wide.clone()
    A.attention_prompt(seqs(A, p, paged=False), q, k, v, out=o)
    p.check(o, None, True)
    wide[:, 256:512] = was[:, 256:512]
    assert torch.equal(wide, was)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("style", ["half", "interleaved"])
def test_angles_of_far_positions(A, style, dtype):
    """Up to the last int32 position.  Beside attn_parity's 32 u for the pair, the
    angle is off by 2^-32 turn and t (f 2^-55 + 2^-64) turns: the double f / 2 pi is off
    by 2^-53 of itself for the product and 2^-53.8 for the constant, together less than
    f 2^-55, its fraction ends at 2^-64, and the position multiplies both.  The
    oracle's angles are taken in 200 bits (a double product of 2^31 f is off by 2^-22)."""
    mp = pytest.importorskip("mpmath")
    d, kv = 128, [2 ** 31 - 1, 2 ** 28 + 5, 2 ** 24 + 1, 70]
    p = Problem([(3, t) for t in kv], 2, 1, d, dtype, 0, seed=12)
    freq = A.rope_frequencies(d, 10000.0)[0]
    sq = A.Sequences(p.seq_start, p.kv_len)
    got, _ = A.qk_norm_rope(sq, p.q, p.k, rope=A.Rope(freq.cuda(), style))
    pos = np.concatenate([np.arange(t - 3, t) for t in kv])
    with mp.workprec(200):
        angle = [[mp.fmod(mp.mpf(int(t)) * mp.mpf(f.item()), 2 * mp.pi) for f in freq] for t in pos]
        cos, sin = (np.array([[float(fn(a)) for a in row] for row in angle])[:, None] for fn in (mp.cos, mp.sin))
    x, y, f = f64(p.q), f64(got), freq.numpy()
    first, second = (slice(0, 64), slice(64, 128)) if style == "half" else (slice(0, 128, 2), slice(1, 128, 2))
    a, b = x[..., first], x[..., second]
    off = 2 * np.pi * (2.0 ** -32 + pos[:, None] * (f * 2.0 ** -55 + 2.0 ** -64))[:, None]
    for z, want in ((y[..., first], a * cos - b * sin), (y[..., second], b * cos + a * sin)):
        r = HALF[p.dt]
        tol = r * np.abs(want) + (1 + r) * (32 * U + off) * (np.abs(a) + np.abs(b))
        assert (np.abs(z - want) <= tol).all(), float((np.abs(z - want) / tol).max())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("count,prefix", [(128, 0), (129, 0), (129, 64), (300, 0), (300, 64)])
def test_batches_of_many_sequences(A, count, prefix, dtype):
    """Around and above the count of sequences from which the join waits before it
    looks at their lengths; some cut into pieces, some empty."""
    r = np.random.default_rng(count)
    own = r.integers(0, 60, count)
    own[[3, count // 2, count - 1]] = [6000, 3001, 900]
    p = Problem([(1, prefix + int(t)) for t in own], 2, 1, 64, dtype, 16, prefix=prefix, seed=count, fill=float("nan"))
    lse = torch.full((p.rows, 2), 9.0, device=p.q.device)
    out = A.attention_decode(A.PagedKVCache(p.kp, p.vp), seqs(A, p, decode=True), p.q, prefix_len=prefix,
                             prefix_table=p.prefix_table if prefix else None, lse=lse)
    p.check(out, lse, False)


@pytest.mark.parametrize("count", [100, 140])
def test_ranges_of_many_short_prompts(A, count):
    """float32 prompts of one or two rows far into a context: key ranges and a join."""
    r = np.random.default_rng(count)
    p = Problem([(int(n), 300 + int(t)) for n, t in zip(r.integers(1, 3, count), r.integers(0, 500, count))], 2, 1, 64,
                "fp32", 16, seed=count, spare=2, fill=float("nan"))
    lse = torch.full((p.rows, 2), 9.0, device=p.q.device)
    out = A.attention_prompt_paged(A.PagedKVCache(p.kp, p.vp), seqs(A, p), p.q, out=torch.full_like(p.q, 9.0), lse=lse)
    p.check(out, lse, True)
    assert (out[-2:] == 9.0).all() and (lse[-2:] == 9.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
@pytest.mark.parametrize("hq,hkv,d,page,prefix,kv", [
    (8, 2, 64, 16, 1040, [0, 0, 0]), (8, 2, 128, 16, 1040, [5, 0, 700, 129]), (4, 4, 128, 64, 4096, [128, 128, 64]),
    (16, 1, 64, 128, 2048, [0] * 19 + [1300]), (33, 1, 64, 16, 512, [1, 511, 300]), (3, 3, 64, 8, 64, [63] * 200 + [0])])
def test_prefixes_that_no_sequence_reaches_the_end_of(A, hq, hkv, d, page, prefix, kv, fill, dtype):
    """Keys and values of the prefix behind every sequence's length may hold anything."""
    p = Problem([(1, t) for t in kv], hq, hkv, d, dtype, page, prefix=prefix, seed=prefix, fill=fill)
    lse = torch.full((p.rows, hq), 9.0, device=p.q.device)
    out = A.attention_decode(A.PagedKVCache(p.kp, p.vp), seqs(A, p, decode=True), p.q, prefix_len=prefix,
                             prefix_table=p.prefix_table, out=torch.full_like(p.q, 9.0), lse=lse)
    p.check(out, lse, False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("paged", [False, True])
def test_rows_before_the_first_sequence(A, paged, dtype):
    """seq_start may begin behind row 0: the rows before it belong to no sequence."""
    p = Problem([(150, 150), (0, 0), (70, 200 if paged else 70)], 4, 2, 64, dtype, 16 if paged else 0, seed=3)
    pad = lambda t, x: torch.cat([torch.full_like(t[:9], x), t])  # noqa: E731
    sq = A.Sequences(p.seq_start + 9, p.kv_len if paged else None, p.table if paged else None)
    out, lse = torch.full_like(pad(p.q, 0), 9.0), torch.full((p.rows + 9, 4), 9.0, device=p.q.device)
    q = pad(p.q, float("nan"))
    if paged:
        cache = A.PagedKVCache(p.kp, p.vp)
        A.attention_prompt_paged(cache, sq, q, out=out, lse=lse)
    else:
        A.attention_prompt(sq, q, pad(p.k, float("nan")), pad(p.v, float("inf")), out=out, lse=lse)
    p.check(out[9:], lse[9:], True)
    assert (out[:9] == 9.0).all() and (lse[:9] == 9.0).all()
    if paged:
        k, v = (torch.randn(p.rows, 2, 64, device=p.q.device).to(p.dt) for _ in range(2))
        want = A.append_qkv(cache, seqs(A, p), p.q, k, v)
        after = p.kp.clone(), p.vp.clone()
        p.kp.fill_(1.0), p.vp.fill_(1.0)
        got = A.append_qkv(cache, sq, q, pad(k, float("nan")), pad(v, float("nan")), q_out=torch.full_like(q, 9.0))
        assert torch.equal(got[9:], want) and (got[:9] == 9.0).all()
        for b, (n, total) in enumerate(p.lens):
            for t in range(total - n, total):
                at = p.page_of(b, t), slice(None), t % 16
                assert torch.equal(p.kp[at], after[0][at]) and torch.equal(p.vp[at], after[1][at])
        assert p.kp.isfinite().all() and p.vp.isfinite().all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scores_that_are_all_minus_infinity(A, dtype):
    """Rows whose scores are all -infinity get zeros, like rows that see no key; one
    finite score among them, and its value is the result."""
    p = Problem([(1, 700), (1, 5), (1, 20000)], 4, 2, 64, dtype, 16, seed=3)
    p.q.zero_(), p.q[..., 0].fill_(-float("inf"))
    p.kp[..., 0] = 1.0
    cache, lse = A.PagedKVCache(p.kp, p.vp), torch.empty(3, 4, device=p.q.device)
    for call in (lambda: A.attention_decode(cache, seqs(A, p, decode=True), p.q, lse=lse),
                 lambda: A.attention_prompt_paged(cache, seqs(A, p), p.q, lse=lse)):
        assert (call() == 0).all() and lse.isneginf().all()
    packed = Problem([(300, 300)], 4, 2, 64, dtype, 0, seed=4)
    packed.q.zero_(), packed.q[..., 0].fill_(-float("inf"))
    packed.k[..., 0] = 1.0
    lse = torch.empty(300, 4, device=p.q.device)
    psq = seqs(A, packed, paged=False)
    assert (A.attention_prompt(psq, packed.q, packed.k, packed.v, lse=lse) == 0).all() and lse.isneginf().all()
    # -infinity through one column of the keys instead: key 170 alone is finite
    packed.q.fill_(1.0)
    packed.k[..., 0], packed.k[170] = -float("inf"), 0.25
    out = A.attention_prompt(psq, packed.q, packed.k, packed.v, lse=lse)
    assert (out[:170] == 0).all() and lse[:170].isneginf().all()
    assert torch.equal(out[170:], packed.v[170].repeat_interleave(2, 0).expand(130, 4, 64))
    # 64 * 0.25 / 8, through log2(e) and ln 2 of 24 bits each
    assert ((lse[170:].double() - 2.0).abs() <= 4 * U * 2.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_beyond_32_bits(A, dtype):
    """270000 rows of 64 heads: q and the output have more than 2^31 elements.  The last
    sequences against the oracle, and against the same rows by themselves."""
    n, count, hq, d = 900, 300, 64, 128
    tail = Problem([(n, n)], hq, 1, d, dtype, 0, seed=21)
    dev, rows = tail.q.device, n * count
    assert rows * hq * d > 1 << 31
    q = torch.zeros(rows, hq, d, dtype=tail.dt, device=dev)
    k, v = (torch.zeros(rows, 1, d, dtype=tail.dt, device=dev) for _ in range(2))
    q[-n:], k[-n:], v[-n:] = tail.q, tail.k, tail.v
    q[:n], k[:n], v[:n] = tail.q, tail.k, tail.v
    sq = A.Sequences(torch.arange(0, rows + 1, n, dtype=torch.int32, device=dev))
    lse = torch.empty(rows, hq, device=dev)
    out = A.attention_prompt(sq, q, k, v, lse=lse)
    assert torch.equal(out[-n:], out[:n]) and torch.equal(lse[-n:], lse[:n])
    tail.check(out[-n:], lse[-n:], True, rows=np.array([0, 1, 127, 128, 500, n - 1]))
    assert (out[n:-n] == 0).all()
    del out
    f, _ = A.rope_frequencies(d)
    rope = A.Rope(f.to(dev))
    got, gk = A.qk_norm_rope(sq, q, k, rope=rope, q_out=q)         # in place
    want, wk = A.qk_norm_rope(seqs(A, tail, paged=False), tail.q, tail.k, rope=rope)
    assert torch.equal(got[-n:], want) and torch.equal(gk[-n:], wk) and torch.equal(got[:n], want)
    del q, got, gk, k, v, lse
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("bf16", 16, 16, 64), ("fp32", 8, 2, 64)])
def test_steps_behind_each_other_see_what_was_just_written(A, dtype, hq, hkv, d):
    """300 decode steps over a prefix without a wait between them: lengths, queries,
    keys and tables of every step were written just before it, by small kernels and by
    the append.  The bits of the same steps with a wait after every call."""
    steps, count, prefix, page = 300, 5, 256, 16
    g = torch.Generator().manual_seed(5)
    p = Problem([(1, prefix + steps + 40)] * count, hq, hkv, d, dtype, page, prefix=prefix, seed=6)
    dev = p.q.device
    new = lambda h: torch.randn(steps, count, h, d, generator=g).to(p.dt).to(dev)  # noqa: E731
    qs, ks, vs = new(hq), new(hkv), new(hkv)
    first = torch.tensor([prefix + 3 * b for b in range(count)], dtype=torch.int32, device=dev)
    f, _ = A.rope_frequencies(d)
    rope = A.Rope(f.to(dev))
    before = p.kp.clone(), p.vp.clone()
    shuffled = torch.randperm(count, generator=g).to(dev)

    def run(wait):
        p.kp.copy_(before[0]), p.vp.copy_(before[1])
        kv, table = first.clone(), p.table.clone()
        q, k, v = (torch.empty_like(x[0]) for x in (qs, ks, vs))
        cache, sq = A.PagedKVCache(p.kp, p.vp), A.Sequences(None, kv, table)
        out = torch.empty(steps, count, hq, d, dtype=p.dt, device=dev)
        lse = torch.empty(steps, count, hq, device=dev)
        sync = torch.cuda.synchronize if wait else (lambda: None)
        sync()
        for s in range(steps):
            kv.add_(1), sync()
            if s % 7 == 3:                                         # the sequences change places
                table.copy_(table[shuffled]), sync()
                kv.copy_(kv[shuffled]), sync()
            for to, x in ((q, qs), (k, ks), (v, vs)):
                to.copy_(x[s]), sync()
            A.append_qkv(cache, sq, q, k, v, rope=rope, q_out=q), sync()
            A.attention_decode(cache, sq, q, prefix_len=prefix, prefix_table=p.prefix_table, out=out[s], lse=lse[s])
            sync()
        return out, lse, p.kp.clone()

    want = run(True)
    got = run(False)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()                                 # (no gaps between the launches)
    with torch.cuda.graph(graph):
        got = run(False)
    for _ in range(5):
        [x.fill_(0) for x in got]
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
