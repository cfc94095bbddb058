"""Work cases of the attention operators that stand beside the MoE step: a paged cache of
keys and values in 4 bits (Q4_0 blocks), the attention of single tokens that reads it, the
eviction that bounds it, and the causal attention of whole prompts.

Every case names one call as a serving program makes it.  `run` computes it in plain torch
(32 bits, rounded once at the end) or, where `own` is true, through the package's entry
points.  A cache page holds `page` tokens of every KV head; `table[b, i]` is the page of
tokens i * page .. of sequence b.

Quantisation (Q4_0): of 32 consecutive channels of one token and head, m is the first value
of the largest magnitude, d = -m / 8 limited to +-8188 (so that 8 |d| stays in the fp16 range), q = floor(x / d + 8.5)
limited to 0..15, and the cache holds q and fp16(d); it stands for (q - 8) * fp16(d).
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_TILE = 16  # tokens of one cache tile


def listed():
    return [
        # one new token for each of 32 running sequences: the cache write of a decode step
        {"name": "store 32 tokens", "op": "store", "seqs": 32, "new": 32, "most": 4096, "hkv": 4, "dim": 128, "page": 64, "type": "bf16"},
        # the prompts of 8 sequences written at once, odd lengths, narrow heads
        {"name": "store prompts", "op": "store", "seqs": 8, "new": 16383, "most": 0, "hkv": 8, "dim": 64, "page": 32, "type": "fp16"},
        # one user, a short chat: latency counts
        {"name": "attend one short", "op": "attend", "seqs": 1, "most": 700, "least": 700, "hq": 32, "hkv": 4, "dim": 128, "page": 64, "type": "bf16", "score": False},
        # one user, a long document: few rows, a long axis
        {"name": "attend one long", "op": "attend", "seqs": 1, "most": 131072, "least": 131072, "hq": 32, "hkv": 4, "dim": 128, "page": 64, "type": "bf16", "score": False},
        # a batch of sequences of very different lengths: the ordinary decode step of a server
        {"name": "attend batch", "op": "attend", "seqs": 64, "most": 8192, "least": 129, "hq": 32, "hkv": 4, "dim": 128, "page": 64, "type": "bf16", "score": False},
        # a batch whose attention weights are summed for later eviction, small pages
        {"name": "attend scored", "op": "attend", "seqs": 24, "most": 5001, "least": 40, "hq": 16, "hkv": 4, "dim": 64, "page": 16, "type": "fp16", "score": True},
        # one sequence cut down to its budget
        {"name": "evict one", "op": "evict", "seqs": 1, "most": 4096, "least": 4096, "keep": 1024, "recent": 128, "hkv": 2, "dim": 128, "page": 64, "type": "bf16"},
        # a batch cut down together, odd budget
        {"name": "evict batch", "op": "evict", "seqs": 32, "most": 8192, "least": 2200, "keep": 2047, "recent": 256, "hkv": 4, "dim": 128, "page": 64, "type": "bf16"},
        # a short question
        {"name": "prompt short", "op": "prompt", "seqs": 1, "tokens": 37, "hq": 16, "hkv": 4, "dim": 64, "type": "fp16"},
        # one prompt of the length that the batched prefill is timed on
        {"name": "prompt 2048", "op": "prompt", "seqs": 1, "tokens": 2048, "hq": 16, "hkv": 4, "dim": 128, "type": "bf16"},
        # prompts of different lengths packed into one call
        {"name": "prompt packed", "op": "prompt", "seqs": 9, "tokens": 8191, "hq": 16, "hkv": 2, "dim": 64, "type": "fp16"},
        # a whole document at once
        {"name": "prompt long", "op": "prompt", "seqs": 1, "tokens": 16384, "hq": 16, "hkv": 4, "dim": 128, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "attend", "attend", "evict", "prompt", "prompt"])
    c = {"op": op, "dim": rng.choice([64, 128]), "type": rng.choice(["bf16", "fp16"])}
    if op == "prompt":
        c["hkv"] = rng.choice([1, 2, 4])
        c["hq"] = c["hkv"] * rng.choice([1, 2, 3, 4])
        c["tokens"] = _log(rng, 1, 12000)
        c["seqs"] = min(c["tokens"], _log(rng, 1, 24))
        return c
    c["page"] = rng.choice([16, 32, 48, 64, 128])
    c["hkv"] = rng.choice([1, 2, 3, 4])
    c["seqs"] = _log(rng, 1, 48)
    if op == "store":
        c["new"] = c["seqs"] + _log(rng, 1, 8000) - 1
        c["most"] = rng.choice([0, _log(rng, 1, 3000)])
    elif op == "attend":
        c["hq"] = c["hkv"] * rng.choice([1, 2, 5, 7, 8, 12, 16])
        c["most"] = _log(rng, 1, min(90000, 250000 // c["seqs"]))
        c["least"] = rng.randint(1, c["most"])
        c["score"] = rng.random() < 0.35
    else:
        c["keep"] = _log(rng, 2, 4000)
        c["recent"] = rng.randint(0, c["keep"])
        c["least"] = c["keep"] + rng.randint(0, 500)
        c["most"] = c["least"] + _log(rng, 1, max(2, min(60000, 150000 // c["seqs"])))
    return c


# ------------------------------------------------------------------ inputs


def _spread(n, lo, hi, seed):
    """n lengths from lo to hi, evenly spaced, in an order that the seed gives: their sum does not depend on it."""
    v = [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]
    random.Random(seed).shuffle(v)
    return v


def _parts(total, n, seed):
    """n lengths of at least 1 that sum to total, the i-th in proportion to i + 1, in an order that the seed gives."""
    rest, w = total - n, n * (n + 1) // 2
    v = [1 + rest * (i + 1) // w for i in range(n)]
    v[-1] += total - sum(v)
    random.Random(seed).shuffle(v)
    return v


def _starts(v):
    s = [0]
    for x in v:
        s.append(s[-1] + x)
    return s


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _quantise(x):
    """(q, d) of x [..., dim] in blocks of 32 channels: q [..., dim / 32, 32] float, d [..., dim / 32, 1] rounded to fp16."""
    x = x.float().unflatten(-1, (-1, 32))
    m = x.gather(-1, x.abs().argmax(-1, keepdim=True))
    d = (m / -8).clamp(-8188.0, 8188.0)
    q = torch.floor(x / torch.where(d == 0, torch.ones_like(d), d) + 8.5).clamp(0, 15)
    return q, d.half().float()


def _pack(k, v):
    """Cache tiles [n, 18 * dim] uint8 of k, v [n, 16, dim], the layout that moe_cache.h gives."""
    n, _, dim = k.shape
    nb = dim // 32

    def parts(x):
        q, d = _quantise(x)
        q = q.to(torch.uint8)
        return q[..., :16] | (q[..., 16:] << 4), d.half().squeeze(-1).contiguous().view(torch.uint8).view(n, _TILE, nb, 2)

    kb, kd = parts(k)  # bytes [n, 16, nb, 16], scales [n, 16, nb, 2 bytes]
    vb, vd = parts(v)
    kb = kb.view(n, _TILE, nb, 4, 4).permute(0, 1, 3, 2, 4)  # row, word, block, byte
    vb = vb.view(n, 8, 2, nb, 8, 2).permute(0, 1, 4, 3, 2, 5)  # pair, word, block, token of the pair, byte
    vd = vd.view(n, 8, 2, nb, 2).permute(0, 1, 3, 2, 4)  # pair, block, token of the pair
    return torch.cat([x.reshape(n, -1) for x in (kb, vb, kd, vd)], 1)


def _pool(pages, hkv, page, dim, g):
    """A cache of `pages` pages that holds keys and values of normal distribution."""
    n = pages * hkv * page // _TILE
    out = torch.empty(n, 18 * dim, dtype=torch.uint8, device="cuda")
    for i in range(0, n, 1 << 15):
        m = min(n - i, 1 << 15)
        k, v = (torch.randn(m, _TILE, dim, device="cuda", generator=g) for _ in range(2))
        out[i:i + m] = _pack(k, v)
    return out.view(pages, hkv, page // _TILE, 18 * dim)


def _table(seqs, width, first, seed):
    """Page numbers first .. first + seqs * width - 1 in an order that the seed gives."""
    v = list(range(first, first + seqs * width))
    random.Random(seed + 1).shuffle(v)
    return _ints(v).view(seqs, width)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _TYPES[c["type"]]
    s = {"case": c}

    def rand(*shape, std=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * std).to(dt)

    if c["op"] == "prompt":
        s["cu"] = _ints(_starts(_parts(c["tokens"], c["seqs"], seed)))
        s["q"] = rand(c["tokens"], c["hq"], c["dim"], std=2.0)
        s["k"], s["v"] = (rand(c["tokens"], c["hkv"], c["dim"]) for _ in range(2))
        return s
    if c["op"] == "store":
        n = _parts(c["new"], c["seqs"], seed) if c["new"] > c["seqs"] else [1] * c["seqs"]
        start = _spread(c["seqs"], 0, c["most"], seed)
        width = -(-(c["most"] + max(n)) // c["page"])
        s["cu"], s["start"] = _ints(_starts(n)), _ints(start)
        s["k"], s["v"] = (rand(c["new"], c["hkv"], c["dim"]) for _ in range(2))
        s["table"] = _table(c["seqs"], width, 0, seed)
        s["pool"] = torch.zeros(c["seqs"] * width, c["hkv"], c["page"] // _TILE, 18 * c["dim"], dtype=torch.uint8, device="cuda")
        return s
    width = -(-c["most"] // c["page"])
    more = c["seqs"] * -(-c["keep"] // c["page"]) if c["op"] == "evict" else 0
    s["pool"] = _pool(c["seqs"] * width + more, c["hkv"], c["page"], c["dim"], g)
    s["table"] = _table(c["seqs"], width, 0, seed)
    lens = _spread(c["seqs"], c["least"], c["most"], seed)
    s["lens"] = _ints(lens)
    if c["op"] == "attend":
        s["q"] = rand(c["seqs"], c["hq"], c["dim"], std=2.0)
        s["score"] = torch.rand(c["seqs"], c["hkv"], c["most"], device="cuda", generator=g) if c["score"] else None
    else:
        s["score"] = torch.rand(c["seqs"], c["hkv"], c["most"], device="cuda", generator=g) ** 8 * 20
        s["out_table"] = _table(c["seqs"], -(-c["keep"] // c["page"]), c["seqs"] * width, seed)
        s["cu"] = _ints([i * c["keep"] for i in range(c["seqs"] + 1)])
        s["start"] = torch.zeros(c["seqs"], dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------ the operators in plain torch


def _unpack(pool, table, dim):
    """Keys and values [seqs, hkv, width * page, dim] in 32 bits that the pages of `table` stand for."""
    nb = dim // 32
    t = pool[table.long()].permute(0, 2, 1, 3, 4)  # seqs, hkv, width, tiles, bytes
    lead = t.shape[:2] + (t.shape[2] * t.shape[3],)
    t = t.reshape(*lead, 18 * dim)
    kb = t[..., :8 * dim].reshape(*lead, _TILE, 4, nb, 4).transpose(-3, -2)
    vb = t[..., 8 * dim:16 * dim].reshape(*lead, 8, 8, nb, 2, 2).permute(0, 1, 2, 3, 6, 5, 4, 7)
    d = t[..., 16 * dim:].contiguous().view(torch.float16).float()
    kd = d[..., :_TILE * nb].reshape(*lead, _TILE, nb, 1)
    vd = d[..., _TILE * nb:].reshape(*lead, 8, nb, 2).transpose(-1, -2).reshape(*lead, _TILE, nb, 1)

    def values(b, d):
        b = b.reshape(*lead, _TILE, nb, 16)
        return (torch.cat([b & 15, b >> 4], -1).float().sub_(8) * d).view(lead[0], lead[1], -1, dim)

    return values(kb, kd), values(vb, vd)


def _plain_store(s):
    k, v = ((q - 8) * d for q, d in (_quantise(s["k"]), _quantise(s["v"])))
    return k.flatten(-2).to(s["k"].dtype), v.flatten(-2).to(s["v"].dtype)


def _plain_attend(s):
    c, q = s["case"], s["q"].float()
    k, v = _unpack(s["pool"], s["table"], c["dim"])
    k, v = k[:, :, :c["most"]], v[:, :, :c["most"]]
    q = q.view(c["seqs"], c["hkv"], -1, c["dim"])
    z = (q @ k.transpose(-1, -2)) * c["dim"] ** -0.5
    held = torch.arange(c["most"], device="cuda") < s["lens"][:, None, None, None]
    z = z.masked_fill(~held, -math.inf)
    p = torch.exp(z - z.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    out = (p @ v).view(c["seqs"], c["hq"], c["dim"]).to(s["q"].dtype)
    if s["score"] is None:
        return out
    s["score"] += p.sum(2)
    return out, s["score"]


def _plain_evict(s):
    c = s["case"]
    at = torch.arange(c["most"], device="cuda")
    lens = s["lens"][:, None, None]
    rank = torch.where(at >= lens - c["recent"], math.inf, s["score"]).masked_fill(at >= lens, -math.inf)
    kept = torch.sort(rank, dim=-1, descending=True, stable=True)[1][..., :c["keep"]].sort(-1)[0]
    k, v = _unpack(s["pool"], s["table"], c["dim"])
    rows = kept[..., None].expand(-1, -1, -1, c["dim"])
    k, v = (x.gather(2, rows).transpose(1, 2).flatten(0, 1).to(_TYPES[c["type"]]) for x in (k, v))
    return s["lens"].clamp(max=c["keep"]), kept.int(), s["score"].gather(-1, kept), k, v


def _plain_prompt(s):
    c = s["case"]
    q, k, v = (s[n].float().transpose(0, 1) for n in "qkv")
    k, v = (x.repeat_interleave(c["hq"] // c["hkv"], 0) for x in (k, v))
    at = torch.arange(c["tokens"], device="cuda")
    seq = torch.searchsorted(s["cu"][1:].contiguous(), at.int(), right=True)
    seen = (seq[:, None] == seq) & (at[:, None] >= at)
    z = (q @ k.transpose(-1, -2)).mul_(c["dim"] ** -0.5).masked_fill_(~seen, -math.inf)
    z = z.sub_(z.amax(-1, keepdim=True)).exp_()
    return (z @ v).div_(z.sum(-1, keepdim=True)).transpose(0, 1).to(s["q"].dtype)


# ------------------------------------------------------------------ the package's calls


def _own_store(s):
    import expert_cache_host_router_b200 as moe
    moe.kv_store(s["pool"], s["k"], s["v"], s["table"], s["cu"], s["start"])
    return moe.kv_load(s["pool"], s["table"], s["cu"], s["start"], s["case"]["new"], s["k"].dtype)


def _own_attend(s):
    import expert_cache_host_router_b200 as moe
    out = moe.kv_attend(s["pool"], s["q"], s["table"], s["lens"], s["case"]["most"], score=s["score"])
    return out if s["score"] is None else (out, s["score"])


def _own_evict(s):
    import expert_cache_host_router_b200 as moe
    c = s["case"]
    lens, kept, score = moe.kv_evict(s["pool"], s["table"], s["lens"], c["most"], s["score"], c["keep"], c["recent"], s["out_table"])
    k, v = moe.kv_load(s["pool"], s["out_table"], s["cu"], s["start"], c["seqs"] * c["keep"], _TYPES[c["type"]])
    return lens, kept, score, k, v


def _own_prompt(s):
    import expert_cache_host_router_b200 as moe
    return moe.attend_prompt(s["q"], s["k"], s["v"], s["cu"])


_PLAIN = {"store": _plain_store, "attend": _plain_attend, "evict": _plain_evict, "prompt": _plain_prompt}
_OWN = {"store": _own_store, "attend": _own_attend, "evict": _own_evict, "prompt": _own_prompt}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    c = case
    row = c["hkv"] * c["dim"]  # channels of one token, keys or values
    held = row * 2 * 9 // 16  # bytes of one cached token
    if c["op"] == "store":  # write the rows, read them back
        return {"bytes": c["new"] * (4 * row + held + held + 4 * row), "flops": c["new"] * row * 2 * 6}
    if c["op"] == "prompt":
        n = _parts(c["tokens"], c["seqs"], 0)
        return {"bytes": c["tokens"] * c["dim"] * 2 * (2 * c["hq"] + 2 * c["hkv"]), "flops": sum(x * (x + 1) // 2 for x in n) * 4 * c["hq"] * c["dim"]}
    n = sum(_spread(c["seqs"], c["least"], c["most"], 0))
    if c["op"] == "attend":
        return {"bytes": n * held + n * c["hkv"] * 8 * c["score"] + c["seqs"] * c["hq"] * c["dim"] * 4, "flops": n * 4 * c["hq"] * c["dim"]}
    kept = c["seqs"] * c["keep"]  # read the scores, move the rows that stay, read them back
    return {"bytes": n * c["hkv"] * 4 + kept * (c["hkv"] * 12 + 3 * held + 4 * row), "flops": n * c["hkv"]}


# ------------------------------------------------------------------ the definitions in 64 bits


def _exact_rows(x):
    """What the cache holds for rows x [n, heads, dim]."""
    x = x.double().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    big = x.abs().max(-1, keepdim=True)[0]
    first = torch.argmax((x.abs() == big).to(torch.int8), -1, keepdim=True)
    d = (-torch.gather(x, -1, first) / 8).clamp(-8188, 8188)
    q = torch.where(d == 0, torch.full_like(x, 8.0), torch.floor(x / d + 8.5)).clamp(0, 15)
    return ((q - 8) * d.to(torch.float16).double()).flatten(-2)


def _exact_cache(pool, pages, n, dim):
    """Keys and values [hkv, n, dim] in 64 bits of one sequence whose pages are given in order."""
    nb = dim // 32
    raw = pool[pages.long()].transpose(0, 1).reshape(pool.shape[1], -1, 18 * dim)
    out = []
    for which in (0, 1):
        body = raw[..., which * 8 * dim:(which + 1) * 8 * dim]
        d = raw[..., (16 + which) * dim:(17 + which) * dim].contiguous().view(torch.float16).double()
        x = torch.empty(raw.shape[0], raw.shape[1], _TILE, nb, 32, dtype=torch.float64, device=raw.device)
        for r in range(_TILE):
            for b in range(nb):
                for j in range(16):  # byte j of the block: channel j in the low half, j + 16 in the high one
                    if which == 0:
                        at, sc = r * 16 * nb + (j // 4) * 4 * nb + b * 4 + j % 4, r * nb + b
                    else:
                        at, sc = (r // 2) * 32 * nb + (j // 2) * 4 * nb + b * 4 + (r % 2) * 2 + j % 2, (r // 2) * 2 * nb + b * 2 + r % 2
                    byte = body[..., at]
                    x[..., r, b, j] = ((byte & 15).double() - 8) * d[..., sc]
                    x[..., r, b, j + 16] = ((byte >> 4).double() - 8) * d[..., sc]
        out.append(x.reshape(raw.shape[0], -1, dim)[:, :n])
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "store":
        return _exact_rows(s["k"]), _exact_rows(s["v"])
    if c["op"] == "prompt":
        cu, rep = s["cu"].tolist(), c["hq"] // c["hkv"]
        out = torch.empty(c["tokens"], c["hq"], c["dim"], dtype=torch.float64, device="cuda")
        for a, b in zip(cu, cu[1:]):
            for h in range(c["hq"]):
                z = s["q"][a:b, h].double() @ s["k"][a:b, h // rep].double().T / math.sqrt(c["dim"])
                z += torch.triu(torch.full_like(z, -math.inf), 1)
                out[a:b, h] = torch.softmax(z, -1) @ s["v"][a:b, h // rep].double()
        return out
    lens = s["lens"].tolist()
    if c["op"] == "attend":
        out = torch.empty(c["seqs"], c["hq"], c["dim"], dtype=torch.float64, device="cuda")
        score = None if s["score"] is None else s["score"].double()
        for b, n in enumerate(lens):
            k, v = _exact_cache(s["pool"], s["table"][b], n, c["dim"])
            z = torch.einsum("hgd,hnd->hgn", s["q"][b].double().view(c["hkv"], -1, c["dim"]), k) / math.sqrt(c["dim"])
            p = torch.softmax(z, -1)
            out[b] = torch.einsum("hgn,hnd->hgd", p, v).reshape(c["hq"], c["dim"])
            if score is not None:
                score[b, :, :n] += p.sum(1)
        return out if score is None else (out, score)
    keep, ks, vs, kepts, scores = c["keep"], [], [], [], []
    for b, n in enumerate(lens):
        k, v = _exact_cache(s["pool"], s["table"][b], n, c["dim"])
        old = s["score"][b, :, :n - c["recent"]].double()
        order = torch.argsort(old, dim=-1, descending=True, stable=True)[:, :keep - c["recent"]]
        new = torch.arange(n - c["recent"], n, device="cuda").expand(c["hkv"], -1)
        kept = torch.sort(torch.cat([order, new], 1), -1)[0]
        kepts.append(kept.int())
        scores.append(torch.gather(s["score"][b].double(), 1, kept))
        for x, to in ((k, ks), (v, vs)):
            to.append(torch.stack([x[h][kept[h]] for h in range(c["hkv"])], 1))
    return torch.tensor([min(n, keep) for n in lens], dtype=torch.int32), torch.stack(kepts), torch.stack(scores), torch.cat(ks), torch.cat(vs)
