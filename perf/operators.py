"""Cases of the operators that serve from the 4-bit key/value cache, with their plain forms.

append     rope (several axes), the per-head Hadamard R3 and the 4-bit write into pages, then the read back of what
           was written (the values that the codes stand for)
attention  softmax(scale q K^T) V over the cache, causal or not, one token or many
mass       the attention weight that each cached token received, added to a running sum
evict      the choice of the tokens that stay, by that sum, and their move to other pages

Sequence b brings new_b tokens and holds len_b afterwards.  Codes are nibbles c in [-8, 7], two per byte, element 2j in the
low one; a group of `group` values has a scale s and a zero z and stands for s (c - z).
"""
import functools
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    llama2 = dict(q_heads=32, kv_heads=32, d=128, group=128)        # 32 heads of 128, as the KV workload has
    llama3 = dict(q_heads=64, kv_heads=8, d=128, group=128)         # 8192 wide, 8 queries to a key head
    return [
        # one decode step of 64 sequences, text positions
        dict(name="append decode 64", op="append", seqs=64, new=1, ctx=8192, page=16, axes=1, **llama3),
        # a prompt with images: time, height and width positions, three ragged sequences
        dict(name="append image prompt", op="append", seqs=3, new=2731, ctx=4096, page=64, axes=3, **llama2),
        # the smallest call: one sequence, one token, a short context, where latency counts
        dict(name="decode 1 x 300", op="attention", seqs=1, new=1, ctx=300, page=64, causal=True, **llama2),
        # a serving batch in the middle of its answers, ragged lengths
        dict(name="decode 64 x 8192", op="attention", seqs=64, new=1, ctx=8192, page=64, causal=True, **llama3),
        # one user with a long document
        dict(name="decode 1 x 131072", op="attention", seqs=1, new=1, ctx=131072, page=256, causal=True, **llama3),
        # five drafted tokens verified at once, 7 queries to a key head, pages that end inside any tile
        dict(name="draft 16 x 5 x 4096", op="attention", seqs=16, new=5, ctx=4096, page=100, causal=True,
             q_heads=28, kv_heads=4, d=128, group=128),
        # a chunk of a prompt behind what is already cached
        dict(name="chunk 2048 of 8192", op="attention", seqs=1, new=2048, ctx=8192, page=64, causal=True, **llama3),
        # a decoder's queries over an encoder's states of other lengths
        dict(name="cross 8 x 449 x 1500", op="attention", seqs=8, new=449, ctx=1500, page=1500, causal=False,
             q_heads=16, kv_heads=16, d=64, group=128),
        # the running sum during decode
        dict(name="mass decode 32 x 4096", op="mass", seqs=32, new=1, ctx=4096, page=64, causal=True, **llama3),
        # the running sum of a whole prompt
        dict(name="mass prompt 2048", op="mass", seqs=1, new=2048, ctx=2048, page=64, causal=True, **llama2),
        # a batch over its budget
        dict(name="evict 32 x 2048", op="evict", seqs=32, ctx=2048, keep=1024, recent=256, page=64, **llama2),
        # long contexts halved
        dict(name="evict 4 x 32768", op="evict", seqs=4, ctx=32768, keep=16384, recent=1000, page=64, **llama3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice([32, 64, 128, 128, 128, 256])
    group = rng.choice([g for g in (128, 256) if g >= d])
    kv_heads = rng.choice([1, 2, 3, 5, 8, 16]) * (group // d)
    case = dict(q_heads=kv_heads * rng.choice([1, 2, 4, 5, 7, 8]), kv_heads=kv_heads, d=d, group=group,
                page=rng.choice([16, 33, 64, 100, 256]))
    op = rng.choice(["append", "attention", "attention", "attention", "mass", "evict"])
    heads = max(1, case["q_heads"] * d // 4096)
    if op == "append":
        seqs = _log(rng, 1, 128)
        new = _log(rng, 1, max(1, 8192 // (seqs * heads)))
        return dict(case, op=op, seqs=seqs, new=new, ctx=new + _log(rng, 1, 4096), axes=rng.choice([1, 2, 3]))
    if op == "evict":
        seqs = _log(rng, 1, 32)
        ctx = _log(rng, 64, max(64, 65536 // (seqs * max(1, kv_heads * d // 1024))))
        keep = rng.randint(ctx // 4, ctx)
        return dict(case, op=op, seqs=seqs, ctx=ctx, keep=max(1, keep), recent=rng.randint(0, max(1, keep // 2)))
    if rng.random() < 0.6:                                         # single tokens and drafts
        seqs, new = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 8])
        ctx = new + _log(rng, 1, max(2, 131072 // (seqs * max(1, kv_heads * d // 1024))))
    else:                                                          # prompts
        seqs, new = rng.choice([1, 1, 2, 3]), _log(rng, 16, 2048)
        new = max(1, new // (seqs * heads))
        ctx = new + _log(rng, 1, max(2, 4096 // heads))
    return dict(case, op=op, seqs=seqs, new=new, ctx=ctx, causal=rng.random() < 0.75)


def _sizes(case):
    """(new_b, len_b) of each sequence: the largest as the case says, the others spread below it, by the case alone."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    new = [case.get("new", 0)] + [r.randint(max(1, case.get("new", 0) // 2), case["new"]) if case.get("new") else 0
                                  for _ in range(case["seqs"] - 1)]
    lens = [case["ctx"]] + [r.randint(max(n, case["ctx"] // 4, 1), case["ctx"]) for n in new[1:]]
    return new, lens


def _pairs(case):
    """(query, key) pairs that the mask leaves, of one head."""
    new, lens = _sizes(case)
    return sum(q * n - (q * (q - 1) // 2 if case["causal"] else 0) for q, n in zip(new, lens))


def work(case):
    new, lens = _sizes(case)
    d, hq, hk = case["d"], case["q_heads"], case["kv_heads"]
    groups = hk * d // case["group"]
    side = hk * d // 2 + 8 * groups                                # codes, scales and zeros of a token's keys, or its values
    if case["op"] == "append":
        t = sum(new)
        return {"bytes": t * (2 * (hq + 2 * hk) * d + 2 * hq * d + 2 * side + 2 * side + 4 * hk * d),
                "flops": t * (hq + hk) * d * (3 + int(math.log2(d)))}
    if case["op"] == "attention":
        return {"bytes": sum(lens) * 2 * side + sum(new) * hq * d * 4, "flops": 4 * d * hq * _pairs(case)}
    if case["op"] == "mass":
        return {"bytes": sum(lens) * (side + 8 * groups) + sum(new) * hq * (2 * d + 4), "flops": 2 * d * hq * _pairs(case)}
    stay = sum(min(n, case["keep"]) for n in lens)
    return {"bytes": sum(lens) * 4 * groups + stay * (4 * side + 8 * groups), "flops": 0}


# ---------------------------------------------------------------- inputs

def _rand(shape, gen, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * scale


def _codes(x, group):
    """Group-wise asymmetric 4-bit codes of the rows of x, as a cache holds them: (bytes, scales, zeros)."""
    t, w = x.shape
    x = x.reshape(t, w // group, group)
    lo, hi = x.amin(2), x.amax(2)
    s = (hi - lo) / 15
    z = torch.round(-lo / s)
    c = (torch.round(x / s[..., None]) + z[..., None]).clamp(0, 15).to(torch.uint8).reshape(t, w) ^ 8
    return c[:, 0::2] | (c[:, 1::2] << 4), s, (z - 8).to(torch.int32)


def prepare(case, seed):
    new, lens = _sizes(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    d, hq, hk, group, page = case["d"], case["q_heads"], case["kv_heads"], case["group"], case["page"]
    w, tokens, seqs = hk * d, sum(new), case["seqs"]
    per = -(-case["ctx"] // page)                                  # pages of a sequence
    evict = case["op"] == "evict"
    pages = seqs * per * (2 if evict else 1)
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32).reshape(-1, per)
    s = {"case": dict(case), "table": order[:seqs].contiguous(),
         "cu": torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV),
         "lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    rows = pages * page
    chan = torch.ones(w, device=DEV)
    if case["op"] == "append":
        s["cache"] = [torch.zeros((rows, w // 2), dtype=torch.uint8, device=DEV),
                      torch.zeros((rows, w // group), device=DEV),
                      torch.zeros((rows, w // group), dtype=torch.int32, device=DEV)]
        s["cache"] += [x.clone() for x in s["cache"]]
        chan[torch.randperm(w, generator=gen, device=DEV)[:max(1, w // 128)]] = 20.0   # key channels that stand out
        s["q"] = _rand((tokens, hq * d), gen).half()
        s["k"] = (_rand((tokens, w), gen) * chan).half()
        s["v"] = _rand((tokens, w), gen).half()
        s["inv_freq"] = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) * 2 / d)).float().to(DEV)
        axes = case["axes"]
        s["axis"] = (torch.arange(d // 2) * axes // (d // 2)).to(torch.int32).to(DEV)
        at = torch.cat([torch.arange(n - q, n) for q, n in zip(new, lens)])
        side = max(1, int(math.sqrt(case["new"])))                 # image tokens: rows and columns run within the picture
        s["pos"] = torch.stack([at, at // side, at % side][:axes]).to(torch.int32).to(DEV)
        return s
    if evict:
        s["cache"] = [x for _ in range(2) for x in (
            torch.randint(0, 256, (rows, w // 2), generator=gen, device=DEV, dtype=torch.uint8),
            torch.rand((rows, w // group), generator=gen, device=DEV),
            torch.randint(-16, 1, (rows, w // group), generator=gen, device=DEV, dtype=torch.int32))]
        mass = torch.exp(2.0 * _rand((seqs, w // group, per * page), gen))
        s["mass"] = torch.where(torch.rand(mass.shape, generator=gen, device=DEV) < 0.05, torch.zeros_like(mass), mass)
        s["table_out"] = order[seqs:].contiguous()
        return s
    sides = []
    for _ in range(2):
        parts = [_codes(_rand((min(8192, rows - r), w), gen, 1.0), group) for r in range(0, rows, 8192)]
        sides += [torch.cat(x) for x in zip(*parts)]
    s["cache"] = sides
    # queries that look at some keys more than at others: scores with a spread of 2
    s["q"] = _rand((tokens, hq * d), gen, 2.0).half()
    if case["op"] == "mass":
        s["mass"] = torch.rand((seqs, w // group, per * page), generator=gen, device=DEV)
        s["lse"] = _attention(s)[1]
    return s


# ---------------------------------------------------------------- plain forms

def _values(cache, side, slots, group):
    """The values of the cache's rows `slots`, in 32 bits: [..., w]."""
    c, s, z = (x[slots] for x in cache[3 * side:3 * side + 3])
    c = torch.stack([c & 15, c >> 4], -1).flatten(-2).to(torch.int32)
    c = torch.where(c > 7, c - 16, c).unflatten(-1, (-1, group))
    return ((c - z[..., None]).float() * s[..., None]).flatten(-2)


def _slots(table, page, count):
    """Slot of each of the first `count` tokens of each sequence: [seqs, count]."""
    t = torch.arange(count, device=DEV)
    return table.long()[:, t // page] * page + t % page


def _new_slots(s):
    """Slot of each new token, in the order of the rows."""
    case = s["case"]
    row = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.searchsorted(s["cu"].long(), row, right=True) - 1
    t = s["lens"].long()[b] - s["cu"].long()[b + 1] + row
    return s["table"].long()[b, t // case["page"]] * case["page"] + t % case["page"]


def _hadamard(x, d):
    """Unnormalised Hadamard transform of each run of d values, by sums and differences."""
    def stage(x, h):
        x = x.unflatten(-1, (-1, 2, h))
        a, b = x[..., 0, :], x[..., 1, :]
        return torch.stack([a + b, a - b], -2).flatten(-3)
    return functools.reduce(stage, [1 << i for i in range(int(math.log2(d)))], x)


def _append(s):
    case = s["case"]
    d, group = case["d"], case["group"]
    angle = s["pos"].long()[s["axis"].long()].t().double() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turn(x):
        x = x.float().unflatten(1, (-1, d))
        a, b = x[..., :d // 2], x[..., d // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).flatten(1)

    def quantize(x, unit):
        x = x.unflatten(1, (-1, group))
        lo, hi = x.amin(2), x.amax(2)
        r = torch.where(hi > lo, torch.tensor(15.0, device=DEV) / (hi - lo), torch.zeros_like(lo))
        z = torch.round(-lo * r)
        # a code is the whole number next to x r + z: next to a border the product keeps all its bits
        c = torch.round(x.double() * r.double()[..., None] + z.double()[..., None]).clamp(0, 15).to(torch.int32)
        return c, (hi - lo) * unit / 15, z.to(torch.int32)

    unit = torch.tensor(1 / math.sqrt(d), dtype=torch.float32, device=DEV)
    slots, out = _new_slots(s), []
    sides = [quantize(_hadamard(turn(s["k"]), d), unit), quantize(s["v"].float(), torch.ones_like(unit))]
    for_cache = [y for c, sc, z in sides
                 for y in (((c ^ 8).flatten(1)[:, 0::2] | ((c ^ 8).flatten(1)[:, 1::2] << 4)).to(torch.uint8), sc, z - 8)]
    [x.index_copy_(0, slots, y) for x, y in zip(s["cache"], for_cache)]
    q = (_hadamard(turn(s["q"]), d) * unit).half()
    return [q] + [_values(s["cache"], side, slots, group).half() for side in (0, 1)]


def _scores(s):
    """Scores of every padded (query, key) pair, -inf where there is none: [seqs, kv_heads, G, new, ctx], and the rows."""
    case = s["case"]
    d, hk, n, ctx = case["d"], case["kv_heads"], case["new"], case["ctx"]
    new, lens = (s["cu"][1:] - s["cu"][:-1]).long(), s["lens"].long()
    i, t = torch.arange(n, device=DEV), torch.arange(ctx, device=DEV)
    here = i < new[:, None]                                        # [seqs, new]: rows that there are
    rows = torch.where(here, s["cu"][:-1].long()[:, None] + i, 0)
    k = _values(s["cache"], 0, _slots(s["table"], case["page"], ctx), case["group"]).unflatten(2, (hk, d))
    q = s["q"].float()[rows].unflatten(2, (hk, -1, d)).permute(0, 2, 3, 1, 4)            # [seqs, hk, G, new, d]
    x = (q.flatten(2, 3) @ k.permute(0, 2, 3, 1)).unflatten(2, (-1, n)) * (1 / math.sqrt(d))
    limit = (lens - new)[:, None] + i + 1 if case["causal"] else lens[:, None].expand(-1, n)
    seen = here[..., None] & (t < limit[..., None])                # [seqs, new, ctx]
    return x.masked_fill_(~seen[:, None, None], -math.inf), rows, here


def _attention(s):
    case = s["case"]
    x, rows, here = _scores(s)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(m == -math.inf, 0, m)).exp_()
    total = p.sum(-1, keepdim=True)
    v = _values(s["cache"], 1, _slots(s["table"], case["page"], case["ctx"]), case["group"])
    v = torch.where((torch.arange(case["ctx"], device=DEV) < s["lens"].long()[:, None])[..., None], v, 0)
    v = v.unflatten(2, (case["kv_heads"], case["d"])).permute(0, 2, 1, 3)
    o = (p.flatten(2, 3) @ v).unflatten(2, p.shape[2:4]) / torch.where(total == 0, 1, total)
    lse = (m + total.log()).squeeze(-1)
    o, lse = o.permute(0, 3, 1, 2, 4).flatten(2), lse.permute(0, 3, 1, 2).flatten(2)     # [seqs, new, heads (d)]
    return [o[here].half(), lse[here]]


def _mass(s):
    case = s["case"]
    x, rows, here = _scores(s)
    lse = s["lse"][rows].unflatten(2, (case["kv_heads"], -1)).permute(0, 2, 3, 1)[..., None]
    p = x.sub_(lse).exp_().sum((2, 3))                             # [seqs, kv_heads, ctx]
    p = p.unflatten(1, (-1, case["group"] // case["d"])).sum(2)
    s["mass"][:, :, :case["ctx"]] += p
    return s["mass"]


def _evict(s):
    case = s["case"]
    keep, recent, ctx, group = case["keep"], case["recent"], case["ctx"], case["group"]
    lens, mass = s["lens"].long(), s["mass"]
    t = torch.arange(mass.shape[2], device=DEV)
    n = lens[:, None, None]
    newest = (t >= n - recent) & (t < n)
    gone = t >= n
    # the newest first, then by mass; equal ones by their place
    key = torch.where(newest, math.inf, torch.where(gone, -math.inf, mass))
    first = torch.sort(key, dim=2, descending=True, stable=True).indices[:, :, :keep]
    stay = torch.where(n <= keep, t[:first.shape[2]].expand(first.shape), torch.sort(first, 2).values)
    there = torch.arange(stay.shape[2], device=DEV) < n
    kept = torch.where(there, stay, -1)
    out_mass = torch.zeros_like(mass)
    out_mass[:, :, :stay.shape[2]] = torch.where(there, torch.gather(mass, 2, stay), 0)
    src = torch.gather(_slots(s["table"], case["page"], t.numel())[:, None].expand(-1, mass.shape[1], -1), 2, stay)
    dst = _slots(s["table_out"], case["page"], t.numel())[:, None, :stay.shape[2]].expand(src.shape)
    at = torch.arange(mass.shape[1], device=DEV)[None, :, None].expand(src.shape)

    def move(x):
        x = x.unflatten(1, (mass.shape[1], -1))
        x[dst[there.expand(src.shape)], at[there.expand(src.shape)]] = x[src[there.expand(src.shape)],
                                                                        at[there.expand(src.shape)]]
    [move(x) for x in s["cache"]]
    kept = torch.nn.functional.pad(kept, (0, keep - kept.shape[2]), value=-1)
    return [kept.to(torch.int32), torch.clamp(s["lens"], max=keep), out_mass] + s["cache"]


# ---------------------------------------------------------------- one pass

def _sequences(s):
    """The framework's handle of a batch on a cache: tensors' places and sizes, built once as a serving loop does."""
    if "handle" not in s:
        import w4a4_rotation_quantized_b200 as Q
        case, c = s["case"], s["cache"]
        cache = Q.KVCache(tuple(c[:3]), tuple(c[3:]), case["d"], case["group"], case["page"])
        s["handle"] = Q.KVSequences(cache, s["lens"], None if case["op"] == "evict" else s["cu"], s["table"])
        s["rope"] = Q.Rope(s["inv_freq"], s["axis"]) if case["op"] == "append" else None
    return s["handle"]


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import w4a4_rotation_quantized_b200 as Q
        seqs, case = _sequences(s), s["case"]
        if op == "append":
            q = Q.kv_append(seqs, s["q"], s["k"], s["v"], s["rope"], s["pos"])
            return [q, *Q.kv_dequantize(seqs, q.shape[0])]
        if op == "attention":
            return list(Q.kv_attention(seqs, s["q"], causal=case["causal"], return_lse=True))
        if op == "mass":
            return Q.kv_attention_mass(seqs, s["q"], s["lse"], s["mass"], causal=case["causal"])
        kept, lens, mass = Q.kv_evict(seqs, s["mass"], case["keep"], case["recent"], table_out=s["table_out"])
        return [kept, lens, mass] + s["cache"]
    if op == "append":
        return _append(s)
    if op == "attention":
        return _attention(s)
    return _mass(s) if op == "mass" else _evict(s)


# ---------------------------------------------------------------- 64 bits

def _wide(cache, side, slots, d, group):
    """Values of some rows of the cache in 64 bits: [rows, heads, d]."""
    c, s, z = (x[slots] for x in cache[3 * side:3 * side + 3])
    v = torch.empty((c.shape[0], 2 * c.shape[1]), dtype=torch.float64, device=DEV)
    v[:, 0::2], v[:, 1::2] = ((c & 15).double() + 8) % 16 - 8, ((c >> 4).double() + 8) % 16 - 8
    v = (v.reshape(c.shape[0], -1, group) - z.double()[..., None]) * s.double()[..., None]
    return v.reshape(c.shape[0], -1, d)


def exact(case, seed):
    s = prepare(case, seed)
    d, group, hk, page = case["d"], case["group"], case["kv_heads"], case["page"]
    new, lens = _sizes(case)
    if case["op"] == "evict":                                      # the rest are whole numbers and values that only move
        mass = s["mass"].double().cpu().numpy()
        moved = np.zeros_like(mass)
        for b, n in enumerate(lens):
            for j in range(mass.shape[1]):
                old = max(0, n - case["recent"])
                best = np.argsort(-mass[b, j, :old], kind="stable")[:case["keep"] - (n - old)]
                stay = np.arange(n) if n <= case["keep"] else np.concatenate([np.sort(best), np.arange(old, n)])
                moved[b, j, :len(stay)] = mass[b, j, stay]
        return [None, None, moved] + [None] * 6
    if case["op"] == "append":
        h = torch.ones((1, 1), dtype=torch.float64, device=DEV)
        while h.shape[0] < d:
            h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
        h = h / math.sqrt(d)
        phase = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                            s["pos"].double()[s["axis"].long()].T * s["inv_freq"].double())
        got = []
        for name in ("q", "k", "v"):
            x = s[name].double().reshape(s[name].shape[0], -1, d)
            if name != "v":
                y = torch.complex(x[..., :d // 2], x[..., d // 2:]) * phase[:, None]
                x = torch.cat([y.real, y.imag], -1) @ h
            if name != "q":
                x = x.reshape(x.shape[0], -1, group)
                lo, hi = x.min(2, keepdim=True).values, x.max(2, keepdim=True).values
                # the factor to codes is held in 32 bits: values of 16 bits lie on borders often, and it says which side is theirs
                r = (15 / (hi - lo)).float().double()
                z = torch.round(-lo * r)
                x = (torch.clamp(torch.round(x * r + z), 0, 15) - z) * ((hi - lo) / 15)
            got.append(x.reshape(x.shape[0], -1))
        return got
    out, all_lse, mass = [], [], s["mass"].double() if case["op"] == "mass" else None
    start = 0
    for b, (q, n) in enumerate(zip(new, lens)):
        t = torch.arange(n, device=DEV)
        slots = s["table"][b].long()[t // page] * page + t % page
        k = _wide(s["cache"], 0, slots, d, group)
        v = _wide(s["cache"], 1, slots, d, group) if mass is None else None
        x = s["q"][start:start + q].double().reshape(q, hk, -1, d)
        seen = (t[None] <= torch.arange(n - q, n, device=DEV)[:, None]) if case["causal"] else torch.ones((q, n), dtype=torch.bool, device=DEV)
        o, norm = torch.empty_like(x), torch.empty_like(x[..., 0])
        for j in range(hk):
            w = torch.einsum("igd,td->git", x[:, j], k[:, j]) / math.sqrt(d)
            w = torch.where(seen, w, -math.inf)
            if mass is None:
                norm[:, j] = torch.logsumexp(w, -1).T
                o[:, j] = torch.einsum("git,td->igd", torch.softmax(w, -1), v[:, j])
            else:
                lse = s["lse"][start:start + q].double().reshape(q, hk, -1)[:, j].T
                mass[b, j * d // group, :n] += torch.exp(w - lse[..., None]).sum((0, 1))
        out.append(o.reshape(q, -1))
        all_lse.append(norm.reshape(q, -1))
        start += q
    return [torch.cat(out), torch.cat(all_lse)] if mass is None else mass
