"""Cases, inputs and plain forms of the attention operators.

Three operators of ``sparse_expert_ffn_gb300.attention``, the other half of a
pre-norm decoder block around the MoE layer:

* ``append``: per-head RMSNorm of queries and keys (optional), rotary
  positions, and the new keys and values written to a paged cache, in one pass
  (``append_qkv``; without a cache ``qk_norm_rope``);
* ``prompt``: attention of packed sequences of different lengths with grouped
  heads, causal or full, over the prompt's own rows (``attention_prompt``) or
  over the pages of a cache (``attention_prompt_paged``);
* ``decode``: attention of one token per sequence over a paged cache, with an
  optional prefix that all sequences share (``attention_decode``).

``lens`` holds one ``new:total`` pair per sequence: its rows in this call, and
its keys after the call.
"""

import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def _text(pairs):
    return " ".join("%d:%d" % p for p in pairs)


def _pairs(case):
    return [tuple(int(x) for x in t.split(":")) for t in case["lens"].split()]


def _spread(rng, lo, hi):
    """A whole number in lo..hi, its logarithm uniform."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def listed():
    r = random.Random(41)
    return [
        # one decode step of a batch: latency is what counts
        {"name": "append_step_32", "op": "append", "dtype": "bf16", "hq": 32, "hkv": 8, "d": 128, "page": 16,
         "layout": "heads", "paged": True, "norm": False, "style": "half", "rot": 128, "scaling": "none",
         "lens": _text((1, r.randint(40, 6000)) for _ in range(32)), "spare": 3},
        # a packed batch of prompts before the attention of a block, heads normalised
        {"name": "append_prompts", "op": "append", "dtype": "bf16", "hq": 32, "hkv": 8, "d": 128, "page": 64,
         "layout": "heads", "paged": True, "norm": True, "style": "half", "rot": 128, "scaling": "yarn",
         "lens": "8192:8192 5003:9001 2177:2177 1:700", "spare": 0},
        # rows interleaved in the cache, half of each head rotated, pairs side by side, float32
        {"name": "append_fp32_partial", "op": "append", "dtype": "fp32", "hq": 16, "hkv": 16, "d": 64, "page": 32,
         "layout": "rows", "paged": True, "norm": True, "style": "interleaved", "rot": 32, "scaling": "linear",
         "lens": "1531:90001 257:257 64:1064", "spare": 0},
        # a long prompt, causal: the product of the longest rows
        {"name": "prompt_8192", "op": "prompt", "dtype": "bf16", "hq": 32, "hkv": 8, "d": 128, "page": 0,
         "paged": False, "causal": True, "lens": "8192:8192"},
        # a packed batch of uneven prompts, one key head per query head
        {"name": "prompt_packed_d64", "op": "prompt", "dtype": "bf16", "hq": 16, "hkv": 16, "d": 64, "page": 0,
         "paged": False, "causal": True,
         "lens": "1777:1777 33:33 1200:1200 1:1 640:640 1999:1999 129:129 900:900"},
        # chunks of prompts whose first part is in the cache already
        {"name": "prompt_chunks_paged", "op": "prompt", "dtype": "bf16", "hq": 32, "hkv": 8, "d": 128, "page": 16,
         "paged": True, "causal": True, "lens": "1024:9000 512:4100 1024:1024"},
        # one short prompt: latency
        {"name": "prompt_37", "op": "prompt", "dtype": "bf16", "hq": 32, "hkv": 8, "d": 128, "page": 32,
         "paged": True, "causal": True, "lens": "37:37"},
        # float32 layers
        {"name": "prompt_fp32", "op": "prompt", "dtype": "fp32", "hq": 16, "hkv": 4, "d": 64, "page": 0,
         "paged": False, "causal": True, "lens": "1021:1021 700:700"},
        # one sequence far into its context
        {"name": "decode_1_long", "op": "decode", "dtype": "bf16", "hq": 32, "hkv": 8, "d": 128, "page": 16,
         "paged": True, "prefix": 0, "lens": "1:65421"},
        # a served batch of uneven lengths, one slot of it idle
        {"name": "decode_64", "op": "decode", "dtype": "bf16", "hq": 32, "hkv": 8, "d": 128, "page": 64,
         "paged": True, "prefix": 0, "lens": _text([(1, r.randint(100, 8000)) for _ in range(63)] + [(1, 0)])},
        # many answers to one long document
        {"name": "decode_shared_48", "op": "decode", "dtype": "bf16", "hq": 32, "hkv": 8, "d": 128, "page": 16,
         "paged": True, "prefix": 16384, "lens": _text((1, 16384 + r.randint(1, 700)) for _ in range(48))},
        # float32 layers, a short shared instruction
        {"name": "decode_fp32", "op": "decode", "dtype": "fp32", "hq": 16, "hkv": 4, "d": 64, "page": 32,
         "paged": True, "prefix": 512, "lens": _text((1, 512 + r.randint(1, 1500)) for _ in range(8))},
    ]


def draw(rng):
    op = rng.choice(["append", "prompt", "decode"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 5, 8, 16])
    group = rng.choice([1, 2, 3, 4, 6, 7, 8, 16])
    hq = hkv * min(group, max(1, 32 // hkv))
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    case = {"op": op, "dtype": dtype, "hq": hq, "hkv": hkv, "d": d, "page": page, "paged": True}
    if op == "append":
        total, pairs = _spread(rng, 8, 14000), []
        while total > 0 and len(pairs) < 64:
            n = min(total, _spread(rng, 1, 6000))
            pairs.append((n, n + rng.choice([0, 0, _spread(rng, 1, 100000 if len(pairs) < 3 else 3000)])))
            total -= n
        case.update(layout=rng.choice(["heads", "rows"]), paged=rng.random() < 0.8, norm=rng.random() < 0.5,
                    style=rng.choice(["half", "interleaved"]), rot=rng.choice([d, d, d // 2, d // 4]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), spare=rng.choice([0, 0, 5]),
                    lens=_text(pairs))
    elif op == "prompt":
        paged = rng.random() < 0.5
        longest = _spread(rng, 8, 4000 if dtype == "bf16" else 1200)
        count, pairs = _spread(rng, 1, 8), []
        for _ in range(count):
            n = rng.randint(1, longest)
            pairs.append((n, n + (rng.choice([0, rng.randint(1, longest)]) if paged else 0)))
        case.update(paged=paged, causal=rng.random() < 0.8, lens=_text(pairs))
    else:
        prefix = rng.choice([0, 0, page * _spread(rng, 1, 8192 // page)])
        batch = _spread(rng, 1, 64)
        longest = _spread(rng, 16, 30000 // batch + 400)
        pairs = [(1, prefix + rng.randint(1, longest)) for _ in range(batch)]
        case.update(prefix=prefix, lens=_text(pairs))
    # no more work than the largest listed cases
    while len(pairs) > 1 and (work(case)["flops"] > 5.4e11 or work(case)["bytes"] > (3.7e8 if op == "append" else 9e8)):
        pairs.pop()
        case["lens"] = _text(pairs)
    return case


# ----------------------------------------------------------------- inputs

def _frequencies(case):
    """Radians per position of each rotated pair, and the factor of cos and sin
    (base 10000, contexts stretched 8 times from 4096 where they are scaled)."""
    rot, base, factor, trained = case["rot"], 10000.0, 8.0, 4096
    if case["scaling"] == "ntk" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "yarn":
        def at(turns):
            return rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    dev, dt = torch.device("cuda"), _DT[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    h = random.Random(seed)
    pairs = _pairs(case)
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    prefix = case.get("prefix", 0)
    new, total = [p[0] for p in pairs], [p[1] for p in pairs]
    rows = sum(new) + case.get("spare", 0)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dt)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s = {"case": case, "start": ints(start), "kv_len": ints(total), "n_max": max(new), "kv_max": max(total),
         "q": normal(rows, hq, d, scale=1.5), "out": torch.zeros(rows, hq, d, dtype=dt, device=dev)}
    if case["paged"]:
        shared = prefix // page
        need = [0 if t <= prefix else -(-t // page) - shared for t in total]
        count = shared + sum(need) + 2
        ids = list(range(count))
        h.shuffle(ids)
        s["prefix_table"] = ints(ids[:shared])
        width = shared + max(max(need), 1)
        table, at = [], shared
        for n in need:
            table.append([0] * shared + ids[at:at + n] + [0] * (width - shared - n))
            at += n
        s["table"] = ints(table)
        if case.get("layout") == "rows":
            store = [normal(count, page, hkv, d).transpose(1, 2) for _ in range(2)]
        else:
            store = [normal(count, hkv, page, d) for _ in range(2)]
        s["k_pages"], s["v_pages"] = store
    if case["op"] == "append" or not case["paged"]:
        s["k"], s["v"] = normal(rows, hkv, d), normal(rows, hkv, d)
    if case["op"] == "append":
        freq, s["mscale"] = _frequencies(case)
        s["freq"] = freq.to(dev)
        s["q_norm"], s["k_norm"] = ((1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(dt) if case["norm"] else None
                                    for _ in range(2))
        s["k_out"] = torch.zeros(rows, hkv, d, dtype=dt, device=dev)
    # what a program that calls the framework keeps beside its tensors
    s["keep"] = {}
    if own:
        from sparse_expert_ffn_gb300 import attention as A
        single = case["op"] == "decode"
        s["keep"]["seqs"] = A.Sequences(None if single else s["start"],
                                        s["kv_len"] if case["paged"] or case["op"] == "append" else None,
                                        s["table"] if case["paged"] else None)
        if case["paged"]:
            s["keep"]["cache"] = A.PagedKVCache(s["k_pages"], s["v_pages"])
        if case["op"] == "append":
            s["keep"]["rope"] = A.Rope(s["freq"], style=case["style"], mscale=s["mscale"])
    return s


# ------------------------------------------------------------ plain forms

def _plain_append(s):
    case, dt = s["case"], s["q"].dtype
    rows, rot = s["q"].shape[0], case["rot"]
    row = torch.arange(rows, device=s["q"].device)
    seq = torch.searchsorted(s["start"][1:].long(), row, right=True)
    live = seq < len(s["kv_len"])
    seq = seq.clamp(max=len(s["kv_len"]) - 1)
    pos = row - s["start"][seq + 1] + s["kv_len"][seq]
    angle = pos.double()[:, None] * s["freq"][None, :]
    cos, sin = (angle.cos() * s["mscale"]).float()[:, None, :], (angle.sin() * s["mscale"]).float()[:, None, :]

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
        return torch.cat([t, x[..., rot:]], -1).to(dt)

    out = s["out"]
    out[:] = torch.where(live[:, None, None], one(s["q"], s["q_norm"]), out)
    k = one(s["k"], s["k_norm"])
    if not case["paged"]:
        s["k_out"][:] = torch.where(live[:, None, None], k, s["k_out"])
        return out, s["k_out"]
    page = case["page"]
    at, seq, k, v = pos[live], seq[live], k[live], s["v"][live]
    pid = s["table"][seq, at // page].long()
    s["k_pages"][pid, :, at % page] = k
    s["v_pages"][pid, :, at % page] = v
    return out, s["k_pages"], s["v_pages"]


def _plain_keys(s):
    """Keys and values of every sequence, padded: [B, hkv, L, d] in float32."""
    case = s["case"]
    L, dev = max(s["kv_max"], 1), s["q"].device
    j = torch.arange(L, device=dev)
    if not case["paged"]:
        at = (s["start"][:-1, None] + j[None, :]).clamp(max=s["k"].shape[0] - 1)
        return [x[at].transpose(1, 2).float() for x in (s["k"], s["v"])]
    page = case["page"]
    pid = s["table"][:, torch.clamp(j // page, max=s["table"].shape[1] - 1)].long()
    shared = s["prefix_table"]
    if len(shared):
        n = min(L, len(shared) * page)
        pid[:, :n] = shared[j[:n] // page].long()
    return [x[pid, :, j % page].transpose(1, 2).float() for x in (s["k_pages"], s["v_pages"])]


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
    if case["op"] == "prompt" and case["causal"]:
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
    if not own:
        if state["case"]["op"] == "append":
            return _plain_append(state)
        return _plain_attention(state)
    from sparse_expert_ffn_gb300 import attention as A
    case, keep, out = state["case"], state["keep"], state["out"]
    if case["op"] == "append":
        if case["paged"]:
            A.append_qkv(keep["cache"], keep["seqs"], state["q"], state["k"], state["v"], rope=keep["rope"],
                         q_norm=state["q_norm"], k_norm=state["k_norm"], eps=1e-6, q_out=out)
            return out, state["k_pages"], state["v_pages"]
        A.qk_norm_rope(keep["seqs"], state["q"], state["k"], rope=keep["rope"], q_norm=state["q_norm"],
                       k_norm=state["k_norm"], eps=1e-6, q_out=out, k_out=state["k_out"])
        return out, state["k_out"]
    if case["op"] == "decode":
        return A.attention_decode(keep["cache"], keep["seqs"], state["q"], prefix_len=case["prefix"],
                                  prefix_table=state["prefix_table"] if case["prefix"] else None, out=out)
    if case["paged"]:
        return A.attention_prompt_paged(keep["cache"], keep["seqs"], state["q"], causal=case["causal"], out=out)
    return A.attention_prompt(keep["seqs"], state["q"], state["k"], state["v"], causal=case["causal"], out=out)


# ------------------------------------------------------- work and exactness

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    hq, hkv, d, pairs = case["hq"], case["hkv"], case["d"], _pairs(case)
    rows = sum(p[0] for p in pairs)
    if case["op"] == "append":
        # q read and written, k read and written, v read and written where there is a cache
        moved = rows * d * size * (2 * hq + (4 if case["paged"] else 2) * hkv)
        return {"bytes": moved, "flops": rows * (hq + hkv) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    if case["op"] == "decode":
        shared = case["prefix"]
        keys = min(shared, max(p[1] for p in pairs)) + sum(max(0, p[1] - shared) for p in pairs)
        seen = sum(p[1] for p in pairs)
    else:
        keys = sum(p[1] for p in pairs)
        seen = sum(n * t - (n * (n - 1) // 2 if case["causal"] else 0) for n, t in pairs)
    return {"bytes": 2 * rows * hq * d * size + 2 * keys * hkv * d * size, "flops": 4 * d * hq * seen}


def exact(case, seed):
    s = prepare(case, seed)
    pairs, d = _pairs(case), case["d"]
    if case["op"] == "append":
        rot, half = case["rot"], case["rot"] // 2
        # rotation by multiplying complex numbers, sequence by sequence
        q, k = s["q"].double(), s["k"].double()
        for x, w in ((q, s["q_norm"]), (k, s["k_norm"])):
            if w is not None:
                x /= (x.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt()
                x *= w.double()
        out, kout = s["out"].double(), s["k_out"].double()
        kp, vp = (s["k_pages"].double(), s["v_pages"].double()) if case["paged"] else (None, None)
        row = 0
        for b, (n, total) in enumerate(pairs):
            at = torch.arange(total - n, total, device=q.device)
            turn = torch.polar(torch.full((n, half), float(s["mscale"]), dtype=torch.float64, device=q.device),
                               at.double()[:, None] * s["freq"][None])[:, None, :]
            for x in (q[row:row + n], k[row:row + n]):
                part = x[..., :rot]
                if case["style"] == "half":
                    z = torch.complex(part[..., :half].contiguous(), part[..., half:].contiguous()) * turn
                    x[..., :half], x[..., half:rot] = z.real, z.imag
                else:
                    z = torch.view_as_complex(part.reshape(*part.shape[:-1], half, 2).contiguous()) * turn
                    x[..., :rot] = torch.view_as_real(z).reshape(part.shape)
            out[row:row + n] = q[row:row + n]
            kout[row:row + n] = k[row:row + n]
            if case["paged"]:
                pid, off = s["table"][b].long()[at // case["page"]], at % case["page"]
                kp[pid, :, off] = k[row:row + n]
                vp[pid, :, off] = s["v"][row:row + n].double()
            row += n
        return (out, kp, vp) if case["paged"] else (out, kout)
    hq, hkv = case["hq"], case["hkv"]
    group, out, row = hq // hkv, s["out"].double(), 0
    shared, page = case.get("prefix", 0), case["page"]
    for b, (n, total) in enumerate(pairs):
        for h in range(hkv):
            if case["paged"]:
                own_pages = s["table"][b].long()[shared // page:-(-max(total, 1) // page)]
                ids = torch.cat([s["prefix_table"].long(), own_pages])
                k, v = (x[ids, h].reshape(-1, d)[:total].double() for x in (s["k_pages"], s["v_pages"]))
            else:
                k, v = (x[row:row + n, h].double() for x in (s["k"], s["v"]))
            x = s["q"][row:row + n, h * group:(h + 1) * group].double()
            for lo in range(0, n, 2048):                         # row blocks bound the scores' memory
                y = x[lo:lo + 2048]
                m = len(y)
                p = (y.reshape(m * group, d) @ k.T) / math.sqrt(d)
                if case["op"] == "prompt" and case["causal"]:
                    last = torch.arange(total - n + lo, total - n + lo + m, device=p.device).repeat_interleave(group)
                    p[torch.arange(total, device=p.device)[None] > last[:, None]] = -math.inf
                out[row + lo:row + lo + m, h * group:(h + 1) * group] = \
                    (torch.softmax(p, -1) @ v).reshape(m, group, d) if total else 0.0
        row += n
    return out
