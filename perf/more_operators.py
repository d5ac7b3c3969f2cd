"""Cases, inputs and plain forms of the operators around an 8-bit cache.

Four operators of ``sparse_expert_ffn_gb300.attention``, beside the 16- and
32-bit ones of the same names:

* ``axes``: rows whose rotary positions have several axes (time, height, width
  of images and video, given per row), normalised, rotated and written to a
  cache (``append_qkv(..., positions=)``) or to rows (``qk_norm_rope``);
* ``append8``: rows written to a cache of 8-bit codes with a scale for each
  block of tokens and key head (``append_qkv`` with a ``PagedKVCache8``), whose
  pages are then read back as the values they stand for (``values``);
* ``prompt8``: attention of a few to many rows per sequence over such a cache
  (``attention_prompt_paged``): chunks of prompts, drafts of some tokens;
* ``decode8``: attention of one token per sequence over it, with an optional
  prefix that all sequences share (``attention_decode``).

The 8-bit form.  Codes are e4m3 numbers or whole numbers -127 .. 127; element x
of a block is held as code * scale, code = x * (1 / scale) rounded to nearest
even.  A block that had no rows before the call gets the smallest power of two
2^e, e >= -100, with |x| <= largest code * 2^e for all its elements.  A block
that had rows keeps its scale where the new rows fit under it, and otherwise
gets that power of two, its earlier codes being rounded again.

``lens`` holds one ``new:total`` pair per sequence: its rows in this call, and
its keys after the call.
"""

import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
_MOST = {"e4m3": 448.0, "int8": 127.0}


# ------------------------------------------------------------------ cases

def _text(pairs):
    return " ".join("%d:%d" % p for p in pairs)


def _pairs(case):
    return [tuple(int(x) for x in t.split(":")) for t in case["lens"].split()]


def _spread(rng, lo, hi):
    """A whole number in lo..hi, its logarithm uniform."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def listed():
    r = random.Random(53)
    return [
        # prompts of text, images and video before the attention of a block: three axes of positions
        {"name": "axes_video", "op": "axes", "dtype": "bf16", "hq": 32, "hkv": 8, "d": 128, "page": 64, "paged": True,
         "layout": "heads", "norm": True, "style": "half", "rot": 128, "sections": "16 24 24", "turns": False,
         "lens": "8192:8192 4801:9001 1:700 900:900"},
        # a decode step of the same models: the positions of its tokens do not follow from their places
        {"name": "axes_step_16", "op": "axes", "dtype": "bf16", "hq": 32, "hkv": 8, "d": 128, "page": 16, "paged": True,
         "layout": "heads", "norm": False, "style": "half", "rot": 128, "sections": "16 24 24", "turns": True,
         "lens": _text((1, r.randint(40, 6000)) for _ in range(16))},
        # an image encoder's patches, height and width, float32, no cache
        {"name": "axes_patches_fp32", "op": "axes", "dtype": "fp32", "hq": 16, "hkv": 16, "d": 64, "page": 0,
         "paged": False, "layout": "heads", "norm": False, "style": "interleaved", "rot": 64, "sections": "16 16",
         "turns": False, "lens": "1369:1369 1156:1156 77:77"},
        # one decode step of a batch into an 8-bit cache: latency, and blocks whose scale may grow
        {"name": "append8_step_32", "op": "append8", "code": "e4m3", "block": 16, "hq": 32, "hkv": 8, "d": 128,
         "page": 16, "layout": "heads", "norm": False, "style": "half", "rot": 128, "sections": "", "turns": False,
         "lens": _text((1, r.randint(40, 6000)) for _ in range(32))},
        # packed prompts, heads normalised
        {"name": "append8_prompts", "op": "append8", "code": "e4m3", "block": 32, "hq": 32, "hkv": 8, "d": 128,
         "page": 64, "layout": "heads", "norm": True, "style": "half", "rot": 128, "sections": "", "turns": False,
         "lens": "8192:8192 5003:9001 2177:2177 1:700"},
        # whole-number codes, rows interleaved in the cache, chunks that begin inside a block, image positions
        {"name": "append8_int8_axes", "op": "append8", "code": "int8", "block": 64, "hq": 16, "hkv": 16, "d": 64,
         "page": 128, "layout": "rows", "norm": True, "style": "interleaved", "rot": 32, "sections": "6 5 5",
         "turns": True, "lens": "1531:20001 257:257 64:1064"},
        # chunks of prompts whose first part is in the cache already
        {"name": "prompt8_chunks", "op": "prompt8", "code": "e4m3", "block": 16, "hq": 32, "hkv": 8, "d": 128,
         "page": 16, "layout": "heads", "causal": True, "lens": "1024:9000 512:4100 1024:1024"},
        # drafts of some tokens to be verified, for a batch far into its contexts
        {"name": "prompt8_drafts_12", "op": "prompt8", "code": "int8", "block": 32, "hq": 32, "hkv": 8, "d": 128,
         "page": 64, "layout": "heads", "causal": True,
         "lens": _text((r.randint(2, 7), r.randint(900, 9000)) for _ in range(12))},
        # a short question behind a cached text, small heads: latency
        {"name": "prompt8_question", "op": "prompt8", "code": "e4m3", "block": 32, "hq": 16, "hkv": 4, "d": 64,
         "page": 32, "layout": "rows", "causal": True, "lens": "37:421"},
        # one sequence far into its context
        {"name": "decode8_1_long", "op": "decode8", "code": "e4m3", "block": 16, "hq": 32, "hkv": 8, "d": 128,
         "page": 16, "layout": "heads", "prefix": 0, "lens": "1:65421"},
        # a served batch of uneven lengths, one slot of it idle
        {"name": "decode8_64", "op": "decode8", "code": "int8", "block": 64, "hq": 32, "hkv": 8, "d": 128,
         "page": 64, "layout": "heads", "prefix": 0,
         "lens": _text([(1, r.randint(100, 8000)) for _ in range(63)] + [(1, 0)])},
        # many answers to one long document
        {"name": "decode8_shared_48", "op": "decode8", "code": "e4m3", "block": 16, "hq": 32, "hkv": 8, "d": 128,
         "page": 16, "layout": "heads", "prefix": 16384,
         "lens": _text((1, 16384 + r.randint(1, 700)) for _ in range(48))},
    ]


def draw(rng):
    op = rng.choice(["axes", "append8", "prompt8", "decode8"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 5, 8, 16])
    group = rng.choice([1, 2, 3, 4, 6, 7, 8, 16])
    hq = hkv * min(group, max(1, 32 // hkv))
    page = rng.choice([16, 32, 64, 128, 256])
    case = {"op": op, "hq": hq, "hkv": hkv, "d": d, "page": page, "layout": rng.choice(["heads", "rows"])}
    if op == "axes":
        case.update(dtype=rng.choice(["bf16", "bf16", "fp32"]), paged=rng.random() < 0.7)
    else:
        case.update(code=rng.choice(["e4m3", "int8"]), block=min(page, rng.choice([16, 32, 64])))
    if op in ("axes", "append8"):
        rot = rng.choice([d, d, d // 2])
        cuts = sorted(rng.sample(range(1, rot // 2), 2))
        sections = rng.choice([[cuts[0], cuts[1] - cuts[0], rot // 2 - cuts[1]], [cuts[0], rot // 2 - cuts[0]]])
        if op == "append8" and rng.random() < 0.5:
            sections = []
        total, pairs = _spread(rng, 8, 14000), []
        while total > 0 and len(pairs) < 64:
            n = min(total, _spread(rng, 1, 6000))
            pairs.append((n, n + rng.choice([0, 0, _spread(rng, 1, 100000 if len(pairs) < 3 else 3000)])))
            total -= n
        case.update(norm=rng.random() < 0.5, style=rng.choice(["half", "interleaved"]), rot=rot,
                    sections=" ".join(map(str, sections)), turns=rng.random() < 0.5)
    elif op == "prompt8":
        longest = _spread(rng, 2, 2000)
        count, pairs = _spread(rng, 1, 16), []
        for _ in range(count):
            n = rng.randint(1, longest)
            pairs.append((n, n + rng.choice([0, _spread(rng, 1, 9000)])))
        case.update(causal=rng.random() < 0.8)
    else:
        prefix = rng.choice([0, 0, page * _spread(rng, 1, 8192 // page)])
        batch = _spread(rng, 1, 64)
        longest = _spread(rng, 16, 30000 // batch + 400)
        pairs = [(1, prefix + rng.randint(1, longest)) for _ in range(batch)]
        case.update(prefix=prefix)
    case["lens"] = _text(pairs)
    # no more work than the largest listed cases
    while len(pairs) > 1 and (work(case)["flops"] > 1.4e11 or work(case)["bytes"] > 3.7e8):
        pairs.pop()
        case["lens"] = _text(pairs)
    return case


# ----------------------------------------------------------------- inputs

def _axis_of_pairs(case):
    """Which axis each rotated pair turns by: runs of pairs, or the axes in turn while they have pairs left."""
    left = [int(x) for x in case["sections"].split()]
    if not case["turns"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    order = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                order.append(a)
                left[a] -= 1
    return order


def _grid_positions(h, n, past, axes):
    """Positions of n rows behind `past` earlier ones: runs of text, whose axes agree, and grids."""
    out, at = [[] for _ in range(axes)], past
    while len(out[0]) < n:
        side = [h.randint(1, 40) for _ in range(axes)]
        if h.random() < 0.5:
            k = min(n - len(out[0]), h.randint(1, 600))
            run = torch.arange(at, at + k)
            cols = [run] * axes
        else:
            grid = torch.meshgrid(*[torch.arange(x) for x in side], indexing="ij")
            cols = [at + g.reshape(-1)[:n - len(out[0])] for g in grid]
        at = 1 + max(int(c.max()) for c in cols)
        for a in range(axes):
            out[a] += cols[a].tolist()
    return out


def _coded(x, case):
    """8-bit codes and block scales of pages [count, hkv, page, d]."""
    count, hkv, page, d = x.shape
    blocks = x.float().reshape(count, hkv, page // case["block"], case["block"], d)
    scale = _power(blocks.abs().amax((-1, -2)), case["code"])
    y = blocks / scale[..., None, None]
    y = y.round() if case["code"] == "int8" else y
    return y.reshape(x.shape).to(_CODE[case["code"]]), scale


def _power(most, code):
    """The smallest power of two that codes reach `most` with."""
    m, e = torch.frexp(most.float())
    top, shift = (0.875, 9) if code == "e4m3" else (127 / 128, 7)
    e = torch.where(m <= top, e, e + 1) - shift
    e = torch.where(most > 0, e, -100).clamp(min=-100)
    return ((e + 127) << 23).view(torch.float32)


def prepare(case, seed):
    dev = torch.device("cuda")
    dt = _DT[case.get("dtype", "bf16")]
    g = torch.Generator(device=dev).manual_seed(seed)
    h = random.Random(seed)
    pairs = _pairs(case)
    op, hq, hkv, d, page = case["op"], case["hq"], case["hkv"], case["d"], case["page"]
    eight, appends = op != "axes", op in ("axes", "append8")
    prefix = case.get("prefix", 0)
    new, total = [p[0] for p in pairs], [p[1] for p in pairs]
    rows = sum(new)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dt)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s = {"case": case, "start": ints(start), "kv_len": ints(total), "n_max": max(new), "kv_max": max(total),
         "q": normal(rows, hq, d, scale=1.5), "out": torch.zeros(rows, hq, d, dtype=dt, device=dev)}
    if page:
        shared = prefix // page
        # appends hold the pages that their rows lie in, attention all
        first = [(t - n) // page if appends else shared for n, t in pairs]
        need = [max(0, -(-t // page) - f) for t, f in zip(total, first)]
        count = shared + sum(need) + 1
        ids = list(range(count))
        h.shuffle(ids)
        s["prefix_table"] = ints(ids[:shared])
        width = max(f + max(n, 1) for f, n in zip(first, need))
        table, at = torch.zeros(len(pairs), width, dtype=torch.int32), shared
        for b, (f, n) in enumerate(zip(first, need)):
            table[b, f:f + n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
            at += n
        s["table"] = table.to(dev)

        def pages():
            if not eight:
                x = normal(count, hkv, page, d)
            else:
                # magnitudes differ between blocks of tokens and between channels
                x = torch.randn(count, hkv, page, d, generator=g, device=dev, dtype=dt)
                size = torch.randn(count, hkv, page // case["block"], 1, generator=g, device=dev).mul_(0.3).exp_()
                x *= size.to(dt).repeat_interleave(case["block"], 2)
                x[..., 5] *= 4
            return x

        def stored(x):
            return x.transpose(1, 2).contiguous().transpose(1, 2) if case["layout"] == "rows" else x

        for n in ("k", "v"):
            x = pages()
            if eight:
                x, s[n + "_scale"] = _coded(x, case)
            s[n + "_pages"] = stored(x)
    if appends:
        s["k"], s["v"] = normal(rows, hkv, d), normal(rows, hkv, d)
        rot = case["rot"]
        s["freq"] = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
        s["q_norm"], s["k_norm"] = ((1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(dt) if case["norm"] else None
                                    for _ in range(2))
        s["k_out"] = torch.zeros(rows, hkv, d, dtype=dt, device=dev)
        s["axis"] = s["positions"] = None
        if case["sections"]:
            axes = len(case["sections"].split())
            s["axis"] = torch.tensor(_axis_of_pairs(case), dtype=torch.uint8, device=dev)
            cols = [[] for _ in range(axes)]
            for n, t in pairs:
                for a, c in enumerate(_grid_positions(h, n, t - n, axes)):
                    cols[a] += c
            s["positions"] = ints(cols)
    # what a program that calls the framework keeps beside its tensors
    s["keep"] = {}
    if own:
        from sparse_expert_ffn_gb300 import attention as A
        keep = s["keep"]
        keep["seqs"] = A.Sequences(None if op == "decode8" else s["start"], s["kv_len"], s["table"] if page else None)
        if eight:
            keep["cache"] = A.PagedKVCache8(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
        elif page:
            keep["cache"] = A.PagedKVCache(s["k_pages"], s["v_pages"])
        if appends:
            keep["rope"] = A.Rope(s["freq"], style=case["style"], axes=s["axis"])
    return s


# ------------------------------------------------------------ plain forms

def _plain_rows(s):
    """Each row's sequence and place, and its rotated query and key heads in float32."""
    case = s["case"]
    rot = case["rot"]
    row = torch.arange(s["q"].shape[0], device=s["q"].device)
    seq = torch.searchsorted(s["start"][1:].long(), row, right=True)
    pos = row - s["start"][seq + 1] + s["kv_len"][seq]
    at = pos[:, None] if s["axis"] is None else s["positions"].T[:, s["axis"].long()]
    angle = at.double() * s["freq"][None, :]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        t = x[..., :rot]
        if case["style"] == "half":
            a, b = t[..., :rot // 2], t[..., rot // 2:]
            t = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = t[..., 0::2], t[..., 1::2]
            t = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([t, x[..., rot:]], -1)

    return seq, pos, one(s["q"], s["q_norm"]), one(s["k"], s["k_norm"])


def _plain_axes(s):
    case, dt = s["case"], s["q"].dtype
    seq, pos, q, k = _plain_rows(s)
    s["out"][:] = q.to(dt)
    if not case["paged"]:
        s["k_out"][:] = k.to(dt)
        return s["out"], s["k_out"]
    page = case["page"]
    pid = s["table"][seq, pos // page].long()
    s["k_pages"][pid, :, pos % page] = k.to(dt)
    s["v_pages"][pid, :, pos % page] = s["v"]
    return s["out"], s["k_pages"], s["v_pages"]


def _round(y, code):
    return (y.round() if code == "int8" else y).to(_CODE[code])


def _values(codes, scale, case):
    """What the codes stand for, [count, hkv, page, d]."""
    return (codes.float() * scale.repeat_interleave(case["block"], 2)[..., None]).to(torch.bfloat16)


def _store8(s, name, x, seq, pos):
    """Rows x [rows, hkv, d] into the pages: scales first, then the codes of the rows before them, then theirs."""
    case, codes, scale = s["case"], s[name + "_pages"], s[name + "_scale"]
    page, block, code = case["page"], case["block"], case["code"]
    count, hkv, _, d = codes.shape
    per = page // block
    pid = s["table"][seq, pos // page].long()
    flat = pid * per + pos % page // block
    most = torch.zeros(count * per, hkv, device=x.device)
    most.scatter_reduce_(0, flat[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
    touched = torch.zeros(count * per, dtype=torch.bool, device=x.device)
    touched[flat] = True
    begin = s["start"][:-1].long()
    kept = torch.zeros(count * per, dtype=torch.long, device=x.device)
    kept[flat[begin]] = pos[begin] % block
    old = scale.transpose(1, 2).reshape(count * per, hkv)
    stays = (kept > 0)[:, None] & (most <= _MOST[code] * old)
    new = torch.where(touched[:, None] & ~stays, _power(most, code), old)
    before = torch.arange(block, device=x.device)[None, :] < kept[:, None]                     # [blocks, block]
    again = before.view(count, 1, per, block, 1).expand(count, hkv, per, block, d).reshape(codes.shape)
    ratio = (old / new).view(count, per, hkv).transpose(1, 2).repeat_interleave(block, 2)[..., None]
    recoded = _round(codes.float() * ratio, code).view(torch.uint8)
    scale[:] = new.view(count, per, hkv).transpose(1, 2)
    held = codes.view(torch.uint8)
    held[:] = torch.where(again, recoded, held)
    held[pid, :, pos % page] = _round(x * (1 / new[flat])[..., None], code).view(torch.uint8)
    return _values(codes, scale, case)


def _plain_append8(s):
    seq, pos, q, k = _plain_rows(s)
    s["out"][:] = q.to(s["out"].dtype)
    return s["out"], _store8(s, "k", k, seq, pos), _store8(s, "v", s["v"].float(), seq, pos)


def _plain_keys(s):
    """Keys and values of every sequence, padded: [B, hkv, L, d] in float32."""
    case = s["case"]
    page, block = case["page"], case["block"]
    L = max(s["kv_max"], 1)
    j = torch.arange(L, device=s["q"].device)
    pid = s["table"][:, torch.clamp(j // page, max=s["table"].shape[1] - 1)].long()
    shared = s["prefix_table"]
    if len(shared):
        n = min(L, len(shared) * page)
        pid[:, :n] = shared[j[:n] // page].long()
    return [(s[n + "_pages"].view(torch.uint8)[pid, :, j % page].view(_CODE[case["code"]]).float() *
             s[n + "_scale"][pid, :, j % page // block][..., None]).transpose(1, 2) for n in ("k", "v")]


def _plain_attention(s):
    case, dt = s["case"], s["q"].dtype
    hq, hkv, d, dev = case["hq"], case["hkv"], case["d"], s["q"].device
    B, n, G = len(s["kv_len"]), s["n_max"], hq // hkv
    i = torch.arange(n, device=dev)
    at = s["start"][:-1, None] + i[None, :]
    live = at < s["start"][1:, None]
    at = at.clamp(max=s["q"].shape[0] - 1)
    k, v = _plain_keys(s)
    L = k.shape[2]
    if case.get("causal"):
        count = s["start"][1:] - s["start"][:-1]
        see = s["kv_len"][:, None] - count[:, None] + i[None, :] + 1
    else:
        see = s["kv_len"][:, None].expand(B, n)
    hide = torch.arange(L, device=dev)[None, None, :] >= see[:, :, None]          # [B, n, L]
    q = s["q"][at].float().view(B, n, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, n * G, d)
    x = torch.matmul(q, k.transpose(2, 3)).view(B, hkv, n, G, L)
    x *= d ** -0.5
    x.masked_fill_(hide[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    z = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, hkv, n * G, L), v).view(B, hkv, n, G, d)
    o = torch.where(z == 0, 0.0, o / z).permute(0, 2, 1, 3, 4).reshape(B, n, hq, d).to(dt)
    s["out"][at[live]] = o[live]
    return s["out"]


def run(state):
    case, keep, out = state["case"], state["keep"], state["out"]
    op = case["op"]
    if not own:
        return {"axes": _plain_axes, "append8": _plain_append8}.get(op, _plain_attention)(state)
    from sparse_expert_ffn_gb300 import attention as A
    if op == "decode8":
        return A.attention_decode(keep["cache"], keep["seqs"], state["q"], prefix_len=case["prefix"],
                                  prefix_table=state["prefix_table"] if case["prefix"] else None, out=out)
    if op == "prompt8":
        return A.attention_prompt_paged(keep["cache"], keep["seqs"], state["q"], causal=case["causal"], out=out)
    how = {"rope": keep["rope"], "positions": state["positions"], "q_norm": state["q_norm"],
           "k_norm": state["k_norm"], "eps": 1e-6, "q_out": out}
    if op == "axes" and not case["paged"]:
        A.qk_norm_rope(keep["seqs"], state["q"], state["k"], k_out=state["k_out"], **how)
        return out, state["k_out"]
    A.append_qkv(keep["cache"], keep["seqs"], state["q"], state["k"], state["v"], **how)
    if op == "axes":
        return out, state["k_pages"], state["v_pages"]
    return (out, *keep["cache"].values())


# ------------------------------------------------------- work and exactness

def work(case):
    hq, hkv, d, pairs, page = case["hq"], case["hkv"], case["d"], _pairs(case), case["page"]
    rows = sum(p[0] for p in pairs)
    if case["op"] == "axes":
        # q, k and (into a cache) v, read and written
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": rows * d * size * (2 * hq + (4 if case["paged"] else 2) * hkv),
                "flops": rows * (hq + hkv) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    if case["op"] == "append8":
        # q, k, v read, q and the codes written; the pages' codes read, their values written
        pages = 1 + sum(-(-t // page) - (t - n) // page for n, t in pairs)
        return {"bytes": rows * d * (4 * hq + 6 * hkv) + pages * page * hkv * d * 6,
                "flops": rows * (hq + hkv) * (3 * case["rot"] + (4 * d if case["norm"] else 0)) + 4 * rows * hkv * d}
    if case["op"] == "decode8":
        shared = case["prefix"]
        keys = min(shared, max(p[1] for p in pairs)) + sum(max(0, p[1] - shared) for p in pairs)
        seen = sum(p[1] for p in pairs)
    else:
        keys = sum(p[1] for p in pairs)
        seen = sum(n * t - (n * (n - 1) // 2 if case["causal"] else 0) for n, t in pairs)
    # q read and o written in bf16; codes, and two scales per block and head
    return {"bytes": 4 * rows * hq * d + 2 * keys * hkv * (d + 4 / case["block"]), "flops": 4 * d * hq * seen}


def _two(e):
    """2^e in 64 bits, by its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest(y, code):
    """y rounded to the code's numbers, ties to even, in 64 bits."""
    if code == "int8":
        return y.round()
    step = _two((torch.frexp(y)[1] - 4).clamp(min=-9))
    return (y / step).round() * step


def _exact_append8(s, name, x):
    """The values of all pages after rows x (64 bits), block by block of every sequence."""
    case = s["case"]
    page, block, most = case["page"], case["block"], _MOST[case["code"]]
    codes, scale = s[name + "_pages"].float().double(), s[name + "_scale"].double()
    row = 0
    for b, (n, total) in enumerate(_pairs(case)):
        at = total - n
        while at < total:
            lo = at // block * block
            hi = min(total, lo + block)
            pid, off, blk = int(s["table"][b, at // page]), lo % page, lo % page // block
            new = x[row:row + hi - at].transpose(0, 1)                            # [hkv, rows, d]
            top = new.abs().amax((1, 2))
            e = torch.frexp(top / most)[1]
            e = torch.where(most * _two(e - 1) >= top, e - 1, e)
            fresh = _two(torch.where(top > 0, e, -100).clamp(min=-100))
            held = scale[pid, :, blk].clone()
            if at > lo:
                fresh = torch.where(top <= most * held, held, fresh)
                part = codes[pid, :, off:off + at - lo]
                codes[pid, :, off:off + at - lo] = torch.where((fresh == held)[:, None, None], part, _nearest(
                    part * (held / fresh)[:, None, None], case["code"]))
            codes[pid, :, off + at - lo:off + hi - lo] = _nearest(new / fresh[:, None, None], case["code"])
            scale[pid, :, blk] = fresh
            row, at = row + hi - at, hi
    return codes * scale.repeat_interleave(block, 2)[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    pairs, d, page = _pairs(case), case["d"], case["page"]
    if case["op"] in ("axes", "append8"):
        rot, half = case["rot"], case["rot"] // 2
        # rotation by multiplying complex numbers, sequence by sequence
        q, k = s["q"].double(), s["k"].double()
        for x, w in ((q, s["q_norm"]), (k, s["k_norm"])):
            if w is not None:
                x /= (x.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt()
                x *= w.double()
        row = 0
        for b, (n, total) in enumerate(pairs):
            at = torch.arange(total - n, total, device=q.device)
            at = at[:, None].expand(n, half)
            if s["axis"] is not None:
                at = torch.stack([s["positions"][int(a), row:row + n] for a in s["axis"]], 1)
            turn = torch.polar(torch.ones(n, half, dtype=torch.float64, device=q.device),
                               at.double() * s["freq"][None])[:, None, :]
            for x in (q[row:row + n], k[row:row + n]):
                part = x[..., :rot]
                if case["style"] == "half":
                    z = torch.complex(part[..., :half].contiguous(), part[..., half:].contiguous()) * turn
                    x[..., :half], x[..., half:rot] = z.real, z.imag
                else:
                    z = torch.view_as_complex(part.reshape(*part.shape[:-1], half, 2).contiguous()) * turn
                    x[..., :rot] = torch.view_as_real(z).reshape(part.shape)
            row += n
        if case["op"] == "append8":
            return q, _exact_append8(s, "k", k), _exact_append8(s, "v", s["v"].double())
        if not case["paged"]:
            return q, k
        kp, vp, row = s["k_pages"].double(), s["v_pages"].double(), 0
        for b, (n, total) in enumerate(pairs):
            at = torch.arange(total - n, total, device=q.device)
            pid, off = s["table"][b].long()[at // page], at % page
            kp[pid, :, off] = k[row:row + n]
            vp[pid, :, off] = s["v"][row:row + n].double()
            row += n
        return q, kp, vp
    hq, hkv, block = case["hq"], case["hkv"], case["block"]
    group, out, row = hq // hkv, s["out"].double(), 0
    shared = case.get("prefix", 0)
    for b, (n, total) in enumerate(pairs):
        ids = torch.cat([s["prefix_table"].long(), s["table"][b].long()[shared // page:-(-max(total, 1) // page)]])
        for h in range(hkv):
            k, v = ((s[x + "_pages"][:, h].contiguous().view(torch.uint8)[ids].view(_CODE[case["code"]]).float().double()
                     .reshape(len(ids), page // block, block, d) * s[x + "_scale"][ids, h].double()[..., None, None])
                    .reshape(-1, d)[:total] for x in ("k", "v"))
            x = s["q"][row:row + n, h * group:(h + 1) * group].double()
            p = (x.reshape(n * group, d) @ k.T) / math.sqrt(d)
            if case.get("causal"):
                last = torch.arange(total - n, total, device=p.device).repeat_interleave(group)
                p[torch.arange(total, device=p.device)[None] > last[:, None]] = -math.inf
            out[row:row + n, h * group:(h + 1) * group] = (torch.softmax(p, -1) @ v).reshape(n, group, d) if total else 0.0
        row += n
    return out
