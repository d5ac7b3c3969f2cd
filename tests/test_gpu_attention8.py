"""The 8-bit cache on the GPU against the float64 oracle: append (codes, scales,
what is left alone), the values read back, prompts and single tokens over it, and a
run of them together."""

import numpy as np
import pytest
import torch

from attn8_parity import CODE, Problem8, decoded, random_codes, same
from attn_parity import HALF, U, f64, seqs
from oracle import attention as oa

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def A(lib):
    from sparse_expert_ffn_gb300 import attention
    return attention


# ----------------------------------------------------------------- append

def _blocks(p):
    """(sequence, page id, block of the page, first offset of the rows, kept rows, rows)."""
    row = 0
    for b, (n, total) in enumerate(p.lens):
        at = total - n
        while at < total:
            lo = at // p.block * p.block
            hi = min(total, lo + p.block)
            yield b, int(p.table_np[b, at // p.page]), lo % p.page // p.block, at % p.page, at - lo, (row, row + hi - at)
            row, at = row + hi - at, hi


def check_append(p, x, tol, codes, scale, old_codes, old_scale, exact):
    """Every block that got rows: its scale, the new codes and the earlier ones again.
    x: the exact rows; tol: how far the kernel's float32 rows may be from them; exact:
    codes are the nearest of x itself."""
    got, gs, was, ws = decoded(codes), f64(scale), decoded(old_codes), f64(old_scale)
    most = oa.CODE_MOST[p.code]
    left = np.ones(was.shape[:1] + was.shape[2:3], dtype=bool)          # page, row: not written
    touched = np.zeros(ws.shape[:1] + ws.shape[2:], dtype=bool)
    for b, pid, blk, off, kept, (r0, r1) in _blocks(p):
        touched[pid, blk] = True
        left[pid, off - kept:off + r1 - r0] = False
        for h in range(p.hkv):
            new, t = x[r0:r1, h], tol[r0:r1, h]
            s, old = gs[pid, h, blk], ws[pid, h, blk]
            top, slack = np.abs(new).max(), t.max()
            options = {oa.fitting_scale(top + slack, p.code), oa.fitting_scale(max(top - slack, 0), p.code)}
            if kept:
                keep = top - slack <= most * old, top + slack <= most * old
                options = ({old} if keep[0] else set()) | (set() if keep[1] else options)
            assert s in options, (b, pid, blk, h, s, options, top)
            y, ty = new / s, t / s + 4 * U * np.abs(new / s)
            mine = got[pid, h, off:off + r1 - r0]
            if exact and s in {2.0 ** e for e in range(-126, 128)}:
                assert np.array_equal(mine, oa.nearest_code(y, p.code)), (b, pid, blk, h)
            assert (np.abs(mine - y) <= 0.5 * oa.code_step(np.abs(y) + ty, p.code) + ty).all(), (b, pid, blk, h)
            before = was[pid, h, off - kept:off]
            # (a power of two by another, or a quotient that float32 rounds)
            again = before if s == old else oa.nearest_code(before * np.float64(np.float32(old) / np.float32(s)), p.code)
            assert np.array_equal(got[pid, h, off - kept:off], again, equal_nan=True), (b, pid, blk, h, "earlier rows")
    raw, raw_was = (t.view(torch.uint8).cpu().numpy() for t in (codes, old_codes))
    keep = np.broadcast_to(left[:, None, :, None], raw.shape)
    assert np.array_equal(raw[keep], raw_was[keep])
    fine = np.broadcast_to(~touched[:, None], gs.shape)
    assert np.array_equal(gs[fine], ws[fine], equal_nan=True)


APPEND = [
    # lens, hq, hkv, d, code, block, page, layout, style, rot, norm, spare, axes
    ([(1, 1)], 4, 1, 64, "e4m3", 16, 16, "heads", "half", 64, True, 0, 0),
    ([(1, 17), (1, 1), (1, 300), (1, 32)], 32, 8, 128, "e4m3", 16, 32, "heads", "half", 128, False, 3, 3),
    ([(5, 5), (0, 9), (31, 40), (1, 8)], 6, 2, 128, "int8", 32, 32, "rows", "interleaved", 128, True, 0, 0),
    ([(40, 1040), (3, 3)], 5, 5, 64, "int8", 64, 256, "rows", "half", 48, True, 0, 2),
    ([(130, 131), (257, 257)], 8, 4, 128, "e4m3", 64, 64, "heads", "interleaved", 32, False, 2, 0),
    ([(200, 777)], 16, 16, 128, "e4m3", 32, 64, "rows", "half", 16, True, 0, 0),
    ([(100, 177)], 80, 40, 64, "int8", 16, 16, "heads", "half", 32, True, 1, 4),
    ([(33, 64), (2, 66)], 4, 2, 64, "e4m3", 16, 128, "heads", None, 0, False, 0, 0),
]


@pytest.mark.parametrize("lens,hq,hkv,d,code,block,page,layout,style,rot,norm,spare,axes", APPEND)
def test_append8(A, lens, hq, hkv, d, code, block, page, layout, style, rot, norm, spare, axes):
    p = Problem8(lens, hq, hkv, d, code, block, page, layout, spare=spare, seed=5, pow2=len(lens) > 1)
    dev = p.q.device
    # scales of a thousandth: most blocks have to grow, some by far, one of 2^20 stays
    p.ks.nan_to_num_(1.0).mul_(1e-3)
    p.vs.nan_to_num_(1.0).mul_(1e-3)
    p.ks[:, 0] = 2.0 ** 20
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn(p.rows, hkv, d, generator=g).to(BF).to(dev) for _ in range(2))
    v[:, -1] = 0                                              # a head of zeros
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(BF).to(dev) if norm else None for _ in range(2)]
    freq = rope = positions = None
    n = int(p.start[-1])
    pos = np.concatenate([np.arange(t - c, t) for c, t in lens])
    if style:
        f, _ = A.rope_frequencies(rot, 10000.0)
        freq = f.numpy()
        if axes:
            which = A.rope_axes([rot // 2 - (axes - 1)] + [1] * (axes - 1), interleaved=axes == 3)
            positions = torch.randint(-50, 3000, (axes, p.rows), generator=g, dtype=torch.int32)
            pos = positions.numpy()[which.long().numpy(), :n].T
            positions = positions.to(dev)
            rope = A.Rope(f.to(dev), style, axes=which.to(dev))
        else:
            rope = A.Rope(f.to(dev), style)
    olds = [t.clone() for t in (p.kc, p.ks, p.vc, p.vs)]
    out = torch.full((p.rows, hq, d), 7.0, dtype=BF, device=dev)
    r = A.append_qkv(p.cache(A), seqs(A, p), p.q, k, v, rope=rope, positions=positions, q_norm=w[0], k_norm=w[1],
                     eps=1e-5, q_out=out)
    torch.cuda.synchronize()
    assert r is out and (out[n:] == 7.0).all()

    def exact(x, weight):
        """The rows in 64 bits, and what their float32 error is a multiple of."""
        weight = None if weight is None else f64(weight)
        mag = np.abs(oa.norm_rotate(f64(x)[:n], pos, None, weight=weight, eps=1e-5))
        if freq is not None:
            half = len(freq)
            sl = (slice(0, half), slice(half, 2 * half)) if style == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
            both = mag[..., sl[0]] + mag[..., sl[1]]
            mag[..., sl[0]], mag[..., sl[1]] = both, both
        return oa.norm_rotate(f64(x)[:n], pos, freq, style, 1.0, weight, 1e-5), mag

    want, mag = exact(p.q, w[0])
    r = HALF[BF]
    assert (np.abs(f64(out)[:n] - want) <= r * np.abs(want) + (1 + r) * 32 * U * mag).all()
    if style is None and not norm:
        assert torch.equal(out[:n], p.q[:n])
    want, mag = exact(k, w[1])
    check_append(p, want, 32 * U * mag, p.kc, p.ks, olds[0], olds[1], style is None and not norm)
    check_append(p, f64(v)[:n], np.zeros((n, hkv, d)), p.vc, p.vs, olds[2], olds[3], True)
    # what the codes stand for, of all pages and of some, ids that do not exist among them
    kv, vv = p.cache(A).values()
    pages = torch.tensor([2 % kv.shape[0], -1, 0, kv.shape[0], 0], dtype=torch.int32, device=dev)
    some = p.cache(A).values(pages)
    for c, s, x, y in ((p.kc, p.ks, kv, some[0]), (p.vc, p.vs, vv, some[1])):
        f = (c.float() * s.repeat_interleave(block, 2)[..., None]).to(BF)
        assert torch.equal(x.nan_to_num(5.0), f.nan_to_num(5.0))
        assert torch.equal(y[[0, 2, 4]].nan_to_num(5.0), x[[2 % kv.shape[0], 0, 0]].nan_to_num(5.0))
        assert (y[[1, 3]] == 0).all()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_tokens_one_by_one_and_at_once(A, code):
    """A block filled token by token, its rows growing, ends with the scale that it gets
    at once, and with codes off by what roundings at smaller scales leave: half a step
    of the final scale each time that it grew."""
    d, hkv, T = 128, 3, 40
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(T, hkv, d, generator=g).cuda().to(BF) * torch.linspace(0.01, 6, T, device="cuda")[:, None, None]
            .to(BF) for _ in range(2))
    q = torch.randn(T, 6, d, generator=g).cuda().to(BF)
    at_once, by_one = (A.PagedKVCache8.empty(4, 32, hkv, d, 16, CODE[code]) for _ in range(2))
    for c in (at_once, by_one):
        for t in (c.k, c.v):
            t.view(torch.uint8).fill_(0x55)
        c.k_scale.fill_(float("nan")), c.v_scale.fill_(float("nan"))
    table = torch.tensor([[2, 1]], dtype=torch.int32, device="cuda")
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    A.append_qkv(at_once, A.Sequences(ints(0, T), ints(T), table), q, k, v)
    for t in range(T):
        A.append_qkv(by_one, A.Sequences(None, ints(t + 1), table), q[t:t + 1], k[t:t + 1], v[t:t + 1])
    for pid, rows in ((2, 32), (1, 8)):
        n = -(-rows // 16)
        for a, b in ((at_once.k_scale, by_one.k_scale), (at_once.v_scale, by_one.v_scale)):
            assert torch.equal(a[pid, :, :n], b[pid, :, :n])
        for a, b, x, s in ((at_once.k, by_one.k, k, at_once.k_scale), (at_once.v, by_one.v, v, at_once.v_scale)):
            first = 0 if pid == 2 else 32
            scale = f64(s)[pid].repeat(16, -1)[:, :rows, None]
            y = f64(x)[first:first + rows].swapaxes(0, 1) / scale
            one = decoded(b)[pid, :, :rows]
            assert np.array_equal(decoded(a)[pid, :, :rows], oa.nearest_code(y, code))
            # e4m3: only numbers that end below the smallest normal one lose anything more
            off = np.abs(one - y) / oa.code_step(np.maximum(np.abs(y), np.abs(one)), code)
            assert off.max() <= (0.5 + 0.5 + 2.0 ** -3 if code == "e4m3" else 1.0)


def test_rows_without_a_place(A):
    """Positions before 0, pages that do not exist and lengths beyond the table store
    nothing; the queries are written all the same."""
    p = Problem8([(6, 2), (4, 40), (4, 100)], 2, 2, 64, "e4m3", 16, 16, seed=4)
    p.table[1, 2] = -5                                         # positions 36 .. 39
    table = p.table[:, :5].contiguous()                        # 80 positions: 96 .. 99 are beyond
    k, v = (torch.randn(14, 2, 64, device="cuda:0").to(BF) for _ in range(2))
    olds = [t.clone() for t in (p.kc, p.ks, p.vc, p.vs)]
    out = A.append_qkv(p.cache(A), A.Sequences(p.seq_start, p.kv_len, table), p.q, k, v)
    assert torch.equal(out, p.q)
    page = int(p.table_np[0, 0])
    for c, s, was, ws, new in ((p.kc, p.ks, *olds[:2], k), (p.vc, p.vs, *olds[2:], v)):
        # positions 0 and 1 of sequence 0
        want = oa.nearest_code(f64(new)[4:6].swapaxes(0, 1) / f64(s)[page, :, :1, None], "e4m3")
        assert np.array_equal(decoded(c)[page, :, :2], want)
        raw = was.view(torch.uint8)
        raw[page, :, :2] = c.view(torch.uint8)[page, :, :2]
        ws[page] = s[page]
        assert same(c, was) and torch.equal(s.nan_to_num(3.0), ws.nan_to_num(3.0))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_elements_that_are_not_finite(A, bad, code):
    """They make their block of their head NaN, whatever comes behind them, until the
    block is written from its first row on; other blocks and heads stay numbers."""
    d, hkv = 64, 2
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(40, h, d, generator=g).cuda().to(BF) for h in (4, hkv, hkv))
    k[3, 1, 17], v[20, 0, 63] = bad, bad
    c = A.PagedKVCache8.empty(3, 32, hkv, d, 16, CODE[code])
    table = torch.tensor([[0, 2]], dtype=torch.int32, device="cuda")
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for lo, hi in ((0, 10), (10, 27), (27, 40)):
        A.append_qkv(c, A.Sequences(ints(0, hi - lo), ints(hi), table), q[lo:hi], k[lo:hi], v[lo:hi])
    kv, vv = c.values()
    dead = [torch.zeros(3, hkv, 32, dtype=torch.bool, device="cuda") for _ in range(2)]
    dead[0][0, 1, :16] = True
    dead[1][0, 0, 16:] = True
    for x, m, src in ((kv, dead[0], k), (vv, dead[1], v)):
        held = torch.cat([x[0], x[2, :, :8]], 1)               # [hkv, 40, d]
        mark = torch.cat([m[0], m[2, :, :8]], 1)
        assert torch.equal(held.isnan(), mark[..., None].expand_as(held))
        near = (held - src.transpose(0, 1)).abs().nan_to_num(0.0)
        assert (near <= 0.07 * src.transpose(0, 1).abs().nan_to_num(0.0, 0.0, 0.0) + 0.05)[~mark].all()
    A.append_qkv(c, A.Sequences(ints(0, 5), ints(5), table), q[:5], torch.ones_like(k[:5]), torch.ones_like(v[:5]))
    assert (c.values()[0][0, :, :5] == 1).all()


# -------------------------------------------------------------- attention

PROMPT = [
    # lens, hq, hkv, d, code, block, page, layout
    ([(1, 1)], 4, 2, 128, "e4m3", 16, 16, "heads"), ([(10, 210), (130, 130)], 8, 2, 128, "int8", 16, 16, "heads"),
    ([(64, 300), (3, 517), (0, 40), (5, 5)], 4, 1, 64, "e4m3", 32, 32, "rows"),
    ([(100, 1000)], 6, 3, 128, "e4m3", 64, 64, "rows"), ([(129, 400), (1, 128), (2, 129)], 16, 16, 64, "int8", 32, 128, "heads"),
    ([(33, 600)], 7, 1, 128, "int8", 64, 256, "heads"), ([(50, 2000), (700, 700)], 2, 2, 64, "e4m3", 16, 16, "rows"),
    ([(40, 25), (4, 0), (3, 2)], 4, 2, 64, "e4m3", 16, 16, "heads"),   # fewer keys than rows: the first rows see none
    ([(16, 5000)], 8, 1, 128, "e4m3", 16, 32, "heads"),                # few rows far into a context
    ([(2, 900), (5, 33), (7, 1031), (3, 3)], 32, 8, 128, "int8", 32, 64, "rows"),   # drafts
    ([(3, 40)], 128, 1, 64, "e4m3", 16, 16, "heads"),
    ([(5, 700), (0, 100), (12, 12), (1, 2000), (9, 31)], 6, 2, 64, "e4m3", 32, 32, "heads"),
    ([(1, 300)] * 5 + [(2, 64)] + [(1, 0)], 3, 3, 128, "int8", 16, 16, "rows"),
    ([(6, 1500 + 40 * i) for i in range(40)], 16, 4, 128, "e4m3", 16, 64, "heads"),   # more drafts than shares' ends
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,hq,hkv,d,code,block,page,layout", PROMPT)
def test_prompt8(A, lens, hq, hkv, d, code, block, page, layout, causal):
    p = Problem8(lens, hq, hkv, d, code, block, page, layout, seed=page + d, spare=1, pow2=d == 64)
    lse = torch.full((p.rows, hq), 9.0, device=p.q.device)
    out = A.attention_prompt_paged(p.cache(A), seqs(A, p), p.q, causal=causal, out=torch.full_like(p.q, 9.0), lse=lse)
    torch.cuda.synchronize()
    p.check(out, lse, causal)
    assert (out[-1] == 9.0).all() and (lse[-1] == 9.0).all()


DECODE = [
    # kv_len, hq, hkv, d, code, block, page, layout, prefix
    ([1], 1, 1, 64, "e4m3", 16, 16, "heads", 0), ([0, 5, 16, 17], 8, 2, 128, "int8", 16, 16, "heads", 0),
    ([1000, 1, 333], 32, 8, 128, "e4m3", 64, 64, "rows", 0), ([4097], 7, 1, 128, "int8", 32, 32, "heads", 0),
    ([200, 300, 1, 0, 129], 16, 16, 64, "e4m3", 32, 128, "heads", 0), ([515] * 3, 24, 1, 64, "int8", 16, 16, "rows", 0),
    ([777, 64], 64, 1, 128, "e4m3", 16, 16, "heads", 0), ([90, 4000], 128, 1, 64, "int8", 64, 256, "heads", 0),
    ([140, 129, 200, 128], 8, 2, 128, "e4m3", 16, 16, "heads", 128), ([64, 300, 10, 0, 65], 4, 4, 64, "int8", 32, 32, "rows", 64),
    ([2100 + i for i in range(40)], 8, 2, 128, "e4m3", 16, 16, "heads", 2048),
    ([700 + 3 * i for i in range(9)], 32, 1, 128, "int8", 32, 64, "heads", 640), ([512, 512], 6, 2, 128, "e4m3", 64, 256, "heads", 512),
    ([31, 32, 33, 63, 64, 65, 95, 96], 3, 1, 128, "e4m3", 16, 64, "rows", 0),
]


@pytest.mark.parametrize("kv,hq,hkv,d,code,block,page,layout,prefix", DECODE)
def test_decode8(A, kv, hq, hkv, d, code, block, page, layout, prefix):
    p = Problem8([(1, t) for t in kv], hq, hkv, d, code, block, page, layout, prefix=prefix, seed=prefix + d, wide=5, pow2=page == 64)
    lse = torch.full((p.rows, hq), 9.0, device=p.q.device)
    out = A.attention_decode(p.cache(A), seqs(A, p, decode=True), p.q, prefix_len=prefix,
                             prefix_table=p.prefix_table if prefix else None, out=torch.full_like(p.q, 9.0), lse=lse)
    torch.cuda.synchronize()
    p.check(out, lse, False)
    if not prefix:                                             # the prompt form of the same rows
        lse2 = torch.empty_like(lse)
        p.check(A.attention_prompt_paged(p.cache(A), seqs(A, p), p.q, lse=lse2), lse2, True)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
def test_every_code(A, d, code):
    """One key per head, so that its value comes out as it is: all codes."""
    g = torch.Generator().manual_seed(0)
    hkv = 8
    c = A.PagedKVCache8.empty(1, 16, hkv, d, 16, CODE[code])
    every = torch.arange(256, dtype=torch.uint8)
    if code == "e4m3":
        every[[0x7f, 0xff]] = 0                                # (no numbers)
    raw = every[torch.arange(hkv * d) % 256].view(1, hkv, 1, d).expand(1, hkv, 16, d).cuda()
    for t in (c.k, c.v):
        t.view(torch.uint8).copy_(raw)
    c.k_scale.fill_(2.0 ** -10), c.v_scale.fill_(0.375)
    q = torch.randn(1, hkv, d, generator=g).cuda().to(BF)
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    want = (c.v[0, :, 0].float() * 0.375).to(BF)               # (exact)
    lse = torch.empty(1, hkv, device="cuda")
    got = A.attention_decode(c, A.Sequences(None, one, table), q, lse=lse)
    assert (got[0].float() - want.float()).abs().max() <= 2.0 ** -8 * 2 * 168
    scores = (f64(q)[0] * decoded(c.k)[0, :, 0]).sum(-1) * 2.0 ** -10 * d ** -0.5
    assert np.abs(lse[0].double().cpu().numpy() - scores).max() <= 2.0 ** -20 * (1 + np.abs(scores).max())
    for t in (got, A.attention_prompt_paged(c, A.Sequences(torch.tensor([0, 1], dtype=torch.int32, device="cuda"), one,
                                                           table), q)):
        e = (t[0].float() - c.v[0, :, 0].float() * 0.375).abs()
        assert (e <= (2.0 ** -7 + 2.0 ** -15) * c.v[0, :, 0].float().abs() * 0.375).all()


def test_page_ids_out_of_range_read_zeros(A):
    p = Problem8([(1, 40), (1, 64)], 4, 2, 64, "e4m3", 16, 16, seed=2)
    p.table[0, 1], p.table[1, 3] = -1, 10 ** 6
    out = A.attention_decode(p.cache(A), seqs(A, p, decode=True), p.q)
    rows = A.attention_prompt_paged(p.cache(A), seqs(A, p), p.q)
    q = f64(p.q)
    for b, hole in ((0, range(16, 32)), (1, range(48, 64))):
        k, v = (x.copy() for x in p.keys(b))
        k[list(hole)], v[list(hole)] = 0, 0
        want, _, spread = oa.attend(q[b:b + 1], k, v, [p.kv[b]], 64 ** -0.5)
        for got in (out, rows):
            assert (np.abs(f64(got)[b:b + 1] - want) <= 2.0 ** -7 * spread + 2.0 ** -8 * np.abs(want) + 1e-5).all()


def test_refusals(A):
    p = Problem8([(3, 20)], 4, 2, 64, "e4m3", 16, 16)
    c, sq = p.cache(A), seqs(A, p)
    with pytest.raises(ValueError, match="float8"):
        A.PagedKVCache8(p.kp, p.vp, p.ks, p.vs)
    with pytest.raises(ValueError, match="scale"):
        A.PagedKVCache8(p.kc, p.vc, p.ks.double(), p.vs)
    with pytest.raises(ValueError, match="scale"):
        A.PagedKVCache8(p.kc, p.vc, p.ks[:, :1], p.vs)
    with pytest.raises(ValueError):
        A.append_qkv(c, sq, p.q.float(), p.q[:, :2], p.q[:, :2])
    with pytest.raises(ValueError, match="share dtype"):
        A.attention_prompt_paged(c, sq, p.q.float())
    freq = A.rope_frequencies(64)[0].cuda()
    with pytest.raises(ValueError, match="rope"):
        A.append_qkv(c, sq, p.q, p.q[:, :2].contiguous(), p.q[:, :2].contiguous(),
                     positions=torch.zeros(1, 3, dtype=torch.int32, device="cuda"))
    for bad in (torch.zeros(2, 4, dtype=torch.int32, device="cuda"), torch.zeros(3, 3, device="cuda"),
                torch.zeros(9, 3, dtype=torch.int32, device="cuda"), torch.zeros(2, 3, dtype=torch.int32)):
        with pytest.raises(ValueError, match="positions"):
            A.qk_norm_rope(sq, p.q, p.q[:, :2].contiguous(), rope=A.Rope(freq), positions=bad)
    with pytest.raises(ValueError, match="axes"):
        A.Rope(freq, axes=torch.zeros(31, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="out"):
        c.values(out=(p.kp, p.vp[:1]))


def test_block_of_prompt_chunks_and_tokens(A):
    """A cache lived in: a prompt in chunks, then tokens, against attention in 64 bits
    over the values that the cache holds at each step."""
    hq, hkv, d, block = 8, 2, 128, 32
    g = torch.Generator().manual_seed(4)
    c = A.PagedKVCache8.empty(12, 64, hkv, d, block, torch.float8_e4m3fn)
    table = torch.tensor([[3, 0, 5, 9], [7, 1, 11, 2]], dtype=torch.int32, device="cuda")
    rope = A.Rope(A.rope_frequencies(d)[0].cuda(), axes=A.rope_axes([16, 24, 24]).cuda())
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    have = np.zeros(2, dtype=int)
    for new in ((70, 33), (40, 1), (1, 1), (1, 1), (5, 2)):
        have += new
        n = sum(new)
        q, k, v = (torch.randn(n, h, d, generator=g).cuda().to(BF) for h in (hq, hkv, hkv))
        single = new == (1, 1)
        sq = A.Sequences(None if single else ints(0, new[0], n), ints(*have), table)
        positions = torch.randint(0, 500, (3, n), generator=g, dtype=torch.int32).cuda()
        q = A.append_qkv(c, sq, q, k, v, rope=rope, positions=positions)
        out = A.attention_decode(c, sq, q) if single else A.attention_prompt_paged(c, sq, q)
        kv, vv = (f64(x) for x in c.values())
        row = 0
        for b, m in enumerate(new):
            at = np.arange(have[b])
            pid = table[b].cpu().numpy()[at // 64]
            K, V = kv[pid, :, at % 64], vv[pid, :, at % 64]
            want, _, spread = oa.attend(f64(q)[row:row + m], K, V, have[b] - m + np.arange(m) + 1, d ** -0.5)
            assert (np.abs(f64(out)[row:row + m] - want) <= 2.0 ** -7 * spread + 2.0 ** -8 * np.abs(want)).all()
            row += m


def test_graph_replays_with_new_contents(A):
    """Append and attention captured once, replayed with other lengths, tables and rows."""
    hq, hkv, d = 8, 2, 64
    probs = [Problem8([(1, t) for t in kv], hq, hkv, d, "e4m3", 16, 16, seed=s, wide=w) for kv, s, w in
             (((40, 7, 100), 1, 2), ((63, 64, 3), 2, 5))]
    width = min(x.table.shape[1] for x in probs)
    a, b = probs
    pages = min(a.kc.shape[0], b.kc.shape[0])
    state = [x[:pages].clone() for x in (a.kc, a.vc)] + [torch.ones(pages, hkv, 1, device="cuda") for _ in range(2)]
    cache = A.PagedKVCache8(*state)
    g = torch.Generator().manual_seed(8)
    rows = [[torch.randn(3, h, d, generator=g).cuda().to(BF) for h in (hq, hkv, hkv)] for _ in probs]
    tables = [(x.table[:, :width] % pages).contiguous() for x in probs]
    for t in tables:
        t[:] = torch.randperm(pages, generator=g)[:3 * min(width, pages // 3)].view(3, -1)[:, :1].to(torch.int32).cuda() \
            if width * 3 > pages else t
    q, k, v = (x.clone() for x in rows[0])
    table, kv = tables[0].clone(), a.kv_len.clone()
    sq = A.Sequences(None, kv, table)

    def step():
        return A.attention_decode(cache, sq, A.append_qkv(cache, sq, q, k, v))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    start = [x.clone() for x in state]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for x, r, t in zip(probs, rows, tables):
        for s, o in zip(state, start):
            s.view(torch.uint8).copy_(o.view(torch.uint8))
        for dst, src in zip((q, k, v), r):
            dst.copy_(src)
        table.copy_(t), kv.copy_(x.kv_len.clamp(max=16 * width))
        graph.replay()
        torch.cuda.synchronize()
        replayed, after = got.clone(), [s.clone() for s in state]
        for s, o in zip(state, start):
            s.view(torch.uint8).copy_(o.view(torch.uint8))
        assert torch.equal(step().nan_to_num(9.0), replayed.nan_to_num(9.0))
        assert all(same(s, o) for s, o in zip(state, after))
