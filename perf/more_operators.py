"""Measured cases of the parts of a serving step around paged attention.

Four operators, in the order in which one step of a running batch uses them:

    tables  the batch's block tables, lengths, slot map and positions brought up
            to date from how many tokens each request gains or loses
            (pa.update_tables)
    rope    queries and keys normalised per head and turned to their positions,
            keys and values written into the paged cache in the same pass
            (pa.rope_and_cache)
    chunk4  a prefill chunk written into a cache of 4-bit codes and the
            sequences' whole contexts read back as dense 16-bit rows
            (pa.int4_reshape_and_cache, pa.int4_gather)
    decode4 one query token per sequence attending over such a cache
            (pa.int4_decode)

With ``own`` false, ``run`` computes the same results with elementary torch
operations in 32 bits; with ``own`` true it calls this package.

4-bit codes, for a group x of 64 neighbouring values of a row (one token, one KV
head), in 32-bit arithmetic, bf16() rounding to nearest even:
    s = bf16(max((max x / 2 - min x / 2) / 7.5, max |x| / 256, 2^-60))
    z = bf16(min x / s)
    u = round(x (1 / s) - z), at least 0 and at most 15
and the value stands for s (u + z).  Element 2 i of a row is the low half of
byte i, element 2 i + 1 the high half.

Rotation of a row at position p, for the pairs (a, b) of its first 2 F elements,
pair i turned by the angle p f_i:
    (a, b) -> m (a cos - b sin, b cos + a sin)
A pair is the elements (i, i + F), or interleaved (2 i, 2 i + 1).  The norm before
it is x w / sqrt(mean x^2 + eps).
"""
import math
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
GROUP = 64


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # The smallest decode step: four requests, one token each.
        {"name": "tables tiny", "op": "tables", "seqs": 4, "law": "step", "hi": 100, "new": 1, "lens": 1, "bs": 16},
        # One step of a full batch: most requests decode, some end, some take drafts back, some prefill a chunk.
        {"name": "tables mixed", "op": "tables", "seqs": 256, "law": "mixed", "hi": 2048, "new": 512, "lens": 2, "bs": 16},
        # The largest batch: 4,096 requests with long contexts, chunks of up to 256 tokens.
        {"name": "tables large", "op": "tables", "seqs": 4096, "law": "mixed", "hi": 4096, "new": 256, "lens": 3, "bs": 32},
        # The smallest decode step of the tests: 4 sequences, 4 heads of 64.
        {"name": "rope tiny", "op": "rope", "tokens": 4, "hq": 4, "hkv": 4, "d": 64, "rot": 64, "inter": False, "norm": False,
         "scaling": "none", "far": 100, "bs": 16, "dtype": "f16"},
        # One decode step of a 13B-shaped layer: 256 sequences, 40 heads.
        {"name": "rope 13b step", "op": "rope", "tokens": 256, "hq": 40, "hkv": 40, "d": 128, "rot": 128, "inter": False,
         "norm": False, "scaling": "none", "far": 2048, "bs": 16, "dtype": "bf16"},
        # A chunked prefill of a grouped-query model with norms of queries and keys, far into long contexts.
        {"name": "rope gqa chunk", "op": "rope", "tokens": 8192, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "inter": False,
         "norm": True, "scaling": "parts", "far": 131072, "bs": 16, "dtype": "bf16"},
        # The same with a quarter of each head turned, pairs interleaved, an odd number of tokens.
        {"name": "rope partial", "op": "rope", "tokens": 1021, "hq": 32, "hkv": 8, "d": 128, "rot": 32, "inter": True,
         "norm": True, "scaling": "linear", "far": 32768, "bs": 32, "dtype": "f16"},
        # One request's prefix hit on a grouped-query model: a 77-token tail over 1,500 cached tokens.
        {"name": "chunk4 tail", "op": "chunk4", "seqs": 1, "new": 77, "lo": 1500, "hi": 1500, "lens": 4, "hkv": 8, "d": 128,
         "bs": 16, "dtype": "f16"},
        # A 13B-shaped chunked prefill: 16 sequences, 512 new tokens each over 0 to 2,048 cached ones.
        {"name": "chunk4 13b", "op": "chunk4", "seqs": 16, "new": 512, "lo": 0, "hi": 2048, "lens": 5, "hkv": 40, "d": 128,
         "bs": 16, "dtype": "bf16"},
        # The smallest decode step: contexts of up to 100 tokens, where the call's latency counts.
        {"name": "decode4 tiny", "op": "decode4", "seqs": 4, "law": "uniform", "lo": 1, "hi": 100, "lens": 6, "hq": 4,
         "hkv": 4, "d": 64, "bs": 16, "dtype": "f16"},
        # 13B-shaped serving batch: 256 sequences, contexts lognormal around 300 tokens, at most 2,048.
        {"name": "decode4 13b", "op": "decode4", "seqs": 256, "law": "lognormal", "lo": 1, "hi": 2048, "lens": 7, "hq": 40,
         "hkv": 40, "d": 128, "bs": 16, "dtype": "bf16"},
        # Long contexts with grouped queries: 16 sequences of 16 K to 32 K tokens, 32 query heads on 8 KV heads.
        {"name": "decode4 gqa long", "op": "decode4", "seqs": 16, "law": "uniform", "lo": 16384, "hi": 32768, "lens": 8,
         "hq": 32, "hkv": 8, "d": 128, "bs": 32, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "chunk4", "decode4"])
    dtype = rng.choice(["f16", "bf16"])
    d, bs, lens = rng.choice([64, 128, 128]), rng.choice([8, 16, 16, 32, 64]), rng.randrange(1 << 30)
    if op == "tables":
        seqs = _log(rng, 1, 4096)
        return {"op": op, "seqs": seqs, "law": rng.choice(["step", "mixed"]), "hi": _log(rng, 16, 4096),
                "new": _log(rng, 1, max(1, min(4096, 131072 // seqs))), "lens": lens, "bs": bs}
    if op == "rope":
        group = rng.choice([1, 2, 4, 8])
        hkv = rng.choice([1, 2, 3, 4, 5, 8, 8, 12, 32, 40])
        hq = hkv * group if hkv <= 12 else hkv
        tokens = _log(rng, 1, max(1, 8192 * 48 * 128 // ((hq + 2 * hkv) * d)))
        return {"op": op, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "rot": rng.choice([d, d, d // 2, d // 4, 16]),
                "inter": rng.choice([False, True]), "norm": rng.choice([False, True]),
                "scaling": rng.choice(["none", "linear", "parts"]), "far": _log(rng, 64, 1 << 20), "bs": bs, "dtype": dtype}
    if op == "chunk4":
        hi = _log(rng, 1, 2048)
        return {"op": op, "seqs": _log(rng, 1, 16), "new": _log(rng, 1, 512), "lo": rng.randrange(hi), "hi": hi,
                "lens": lens, "hkv": rng.choice([1, 2, 5, 8, 32, 40]), "d": d, "bs": bs, "dtype": dtype}
    group = rng.choice([1, 2, 4, 8])
    hkv = rng.choice([1, 2, 3, 4, 8, 8, 12, 16, 32, 40])
    seqs = _log(rng, 1, 256)
    most = max(64, min(32768, 5_000_000 // (seqs * hkv)))   # at most the tokens x heads of the largest listed case
    hi = _log(rng, 16, most)
    return {"op": op, "seqs": seqs, "law": rng.choice(["uniform", "lognormal"]), "lo": rng.choice([1, max(1, hi // 2)]),
            "hi": hi, "lens": lens, "hq": hkv * min(group, 64 // hkv or 1) if hkv > 16 else hkv * group, "hkv": hkv,
            "d": d, "bs": bs, "dtype": dtype}


def _lengths(case):
    """The case's lengths, a function of the case alone.

    tables: (lengths, changes) per sequence; rope: None; chunk4: cached tokens per
    sequence; decode4: context lengths."""
    if case["op"] == "rope":
        return None
    rng = random.Random(case["lens"])
    if case["op"] == "chunk4":
        return [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    if case["op"] == "decode4":
        if case["law"] == "uniform":
            return [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
        mid = min(300.0, (case["lo"] + case["hi"]) / 2)
        return [min(case["hi"], max(case["lo"], round(rng.lognormvariate(math.log(mid), 1.0)))) for _ in range(case["seqs"])]
    lens, change = [], []
    for _ in range(case["seqs"]):
        n = rng.randint(1, case["hi"])
        c = 1
        if case["law"] == "mixed":
            kind = rng.random()
            if kind < 0.05:
                c = -n                                 # ended
            elif kind < 0.15:
                c = -rng.randint(1, min(n, 8))         # drafted tokens taken back
            elif kind < 0.25:
                c = rng.randint(1, case["new"])        # a prefill chunk, of a new request every second time
                n = rng.choice([0, n])
            elif kind < 0.3:
                c = 0                                  # waiting
        lens.append(n)
        change.append(c)
    return lens, change


def _rope_rows(case):
    return case["tokens"] * case["hq"], case["tokens"] * case["hkv"]


def work(case):
    if case["op"] == "tables":
        lens, change = _lengths(case)
        bs = case["bs"]
        tokens = sum(c for c in change if c > 0)
        moved = sum(abs(-(-(n + c) // bs) - -(-n // bs)) for n, c in zip(lens, change))
        # lengths and changes in, lengths and bounds out, moved block ids in and out, a slot and a position per token
        return {"bytes": 16 * len(lens) + 8 * moved + 16 * tokens, "flops": 8 * (len(lens) + tokens)}
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "rope":
        q, k = _rope_rows(case)
        return {"bytes": (2 * q + 4 * k) * 2 * d + 16 * case["tokens"], "flops": (q + k) * (3 * case["rot"] + 4 * d * case["norm"])}
    row = d // 2 + 4 * (d // GROUP)                    # one quantised row: its codes, and scale and zero of each group
    lens = _lengths(case)
    if case["op"] == "chunk4":
        new = 2 * case["seqs"] * case["new"] * hkv
        both = 2 * (sum(lens) + case["seqs"] * case["new"]) * hkv
        # the new rows are read, quantised and written; every row of the contexts is read and written dense
        return {"bytes": new * (2 * d + row) + both * (row + 2 * d), "flops": 5 * new * d + 2 * both * d}
    tokens = sum(lens)
    return {"bytes": 2 * tokens * hkv * row + 4 * len(lens) * case["hq"] * d + 4 * -(-tokens // case["bs"]),
            "flops": 4 * tokens * case["hq"] * d}


# ---------------------------------------------------------------- the inputs

def _rows(gen, n, hkv, d, dtype, key):
    """n rows of K (with a few strong channels, as keys have) or V."""
    x = torch.randn(n, hkv, d, generator=gen, device="cuda")
    if key:
        ch = torch.exp(0.7 * torch.randn(hkv, d, generator=gen, device="cuda"))
        x *= ch / ch.square().mean(-1, keepdim=True).sqrt()
    else:
        x *= torch.exp(0.5 * torch.randn(n, hkv, 1, generator=gen, device="cuda"))
    return x.to(dtype)


def _pages(gen, blocks, width, spare=None):
    """A block table: a random order of the pool's blocks dealt out to the sequences, -1 past a row's end.

    Returns the table, the pool's size and its blocks that no sequence holds."""
    used = sum(blocks)
    pool = max(1, used + (used // 8 + 1 if spare is None else spare))
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    begin = torch.tensor([0] + blocks[:-1], device="cuda").cumsum(0)
    count = torch.tensor(blocks, device="cuda")
    col = torch.arange(width, device="cuda")
    at = (begin[:, None] + col).clamp(max=pool - 1)
    table = torch.where(col < count[:, None], order[at], torch.full_like(order[:1], -1)).contiguous()
    return table, pool, order[used:].contiguous()


def _quantised(gen, slots, hkv, d, dtype, key):
    """Codes [slots, hkv, d / 2] and (scale, zero) [slots, hkv, d / 64, 2] of a whole cache of token slots."""
    codes = torch.empty(slots, hkv, d // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(slots, hkv, d // GROUP, 2, dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 27) // (hkv * d))
    for a in range(0, slots, step):
        n = min(step, slots - a)
        codes[a:a + n], scales[a:a + n] = _quantise(_rows(gen, n, hkv, d, dtype, key))
    return codes, scales


def _frequencies(case):
    """Angle per position of each pair, and the factor on the turned pairs."""
    n, base = case["rot"] // 2, 10000.0
    freq = [base ** (-i / n) for i in range(n)]
    if case["scaling"] == "linear":                    # positions pressed together
        return [f / 4.0 for f in freq], 1.0
    if case["scaling"] == "parts":                     # slow pairs pressed together, fast ones kept, a ramp between
        out = []
        for f in freq:
            turns = 4096 * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - 1.0) / (32.0 - 1.0)))
            out.append(f * keep + f / 32.0 * (1.0 - keep))
        return out, 0.1 * math.log(32.0) + 1.0
    return freq, 1.0


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    bs, lens = case["bs"], _lengths(case)
    s = {"op": case["op"], "bs": bs}
    if case["op"] == "tables":
        old, change = lens
        width = max(1, max(-(-max(n, n + c) // bs) for n, c in zip(old, change)))
        need = sum(max(0, -(-(n + c) // bs) - -(-n // bs)) for n, c in zip(old, change))
        held = [-(-n // bs) for n in old]
        s["bt"], pool, free = _pages(gen, held, width, spare=need + 8)
        s["free"] = torch.full((pool,), -1, dtype=torch.int32, device="cuda")   # a stack of free blocks, its top last
        s["free"][:free.numel()] = free
        s["count"], s["lens"], s["change"] = _int32([free.numel()]), _int32(old), _int32(change)
        room = sum(c for c in change if c > 0) + 5     # a fixed buffer of a captured step is wider than what it holds
        s["slots"] = torch.empty(room, dtype=torch.int64, device="cuda")
        s["pos"] = torch.empty(room, dtype=torch.int64, device="cuda")
        s["cu"] = torch.empty(len(old) + 1, dtype=torch.int32, device="cuda")
        s["new_lens"], s["new_count"] = torch.empty_like(s["lens"]), torch.empty_like(s["count"])
        return s
    hkv, d, dtype = case["hkv"], case["d"], DT[case["dtype"]]
    s["dtype"], s["sm"] = dtype, 1.0 / math.sqrt(d)
    if case["op"] == "rope":
        t, hq = case["tokens"], case["hq"]
        nb = -(-t // bs) + 3
        for name in "kv":
            s[name + "c"] = torch.zeros(nb, bs, hkv, d, dtype=dtype, device="cuda")
        s["slots"] = torch.randperm(nb * bs, generator=gen, device="cuda")[:t].contiguous()
        start = torch.randint(0, case["far"], (1,), generator=gen, device="cuda")
        # runs of neighbouring positions, as chunks have
        s["pos"] = (start + torch.arange(t, device="cuda") * 7 // 3) % case["far"]
        # queries, keys and values as one projection's output
        wide = torch.empty(t, (hq + 2 * hkv) * d, dtype=dtype, device="cuda")
        s["q"] = wide[:, :hq * d].view(t, hq, d)
        s["key"] = wide[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
        s["value"] = wide[:, (hq + hkv) * d:].view(t, hkv, d)
        s["q"].copy_(1.5 * torch.randn(t, hq, d, generator=gen, device="cuda"))
        s["key"].copy_(_rows(gen, t, hkv, d, dtype, True))
        s["value"].copy_(_rows(gen, t, hkv, d, dtype, False))
        freq, s["factor"] = _frequencies(case)
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")
        s["inter"], s["eps"] = case["inter"], 1e-6
        s["qw"] = s["kw"] = None
        if case["norm"]:
            s["qw"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dtype)
            s["kw"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dtype)
        s["out_q"] = torch.empty(t, hq, d, dtype=dtype, device="cuda")
        return s

    def cache(nb):
        for n in "kv":
            codes, sc = _quantised(gen, nb * bs, hkv, d, dtype, n == "k")
            s[n + "c"] = codes.view(nb, bs, hkv, d // 2)
            s[n + "s"] = sc.view(nb, bs, hkv, d // GROUP, 2).transpose(1, 2).contiguous()   # heads before tokens

    if case["op"] == "chunk4":
        n, new = case["seqs"], case["new"]
        total = [c + new for c in lens]
        s["bt"], nb, _ = _pages(gen, [-(-x // bs) for x in total], -(-max(total) // bs))
        cache(nb)
        pos = (_int32(lens)[:, None] + torch.arange(new, device="cuda")).long()
        s["slots"] = (s["bt"].gather(1, pos // bs).long() * bs + pos % bs).reshape(-1).contiguous()
        s["key"], s["value"] = _rows(gen, n * new, hkv, d, dtype, True), _rows(gen, n * new, hkv, d, dtype, False)
        ends = torch.tensor([0] + total, device="cuda").cumsum(0)
        s["cu"] = ends.to(torch.int32)
        # where each dense row comes from, for the plain form: its sequence and position
        s["row_seq"] = torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor(total, device="cuda"))
        s["row_pos"] = torch.arange(sum(total), device="cuda") - ends[s["row_seq"]]
        s["out_k"] = torch.empty(sum(total), hkv, d, dtype=dtype, device="cuda")
        s["out_v"] = torch.empty_like(s["out_k"])
        return s
    n, hq = case["seqs"], case["hq"]
    s["bt"], nb, _ = _pages(gen, [-(-x // bs) for x in lens], -(-max(lens) // bs))
    cache(nb)
    s["q"] = (2.0 * torch.randn(n, hq, d, generator=gen, device="cuda")).to(dtype)
    s["ctx"], s["max_ctx"] = _int32(lens), max(lens)
    s["out"] = torch.empty_like(s["q"])
    return s


# ------------------------------------------------------------ the plain form

def _plain_tables(s):
    """The step's tables; the pool is large enough and the lengths are in range."""
    bs, bt = s["bs"], s["bt"]
    old = s["lens"].long()
    new = (old + s["change"]).clamp(min=0)
    had, has = (old + bs - 1) // bs, (new + bs - 1) // bs
    need, back = (has - had).clamp(min=0), (had - has).clamp(min=0)
    need_at, back_at = need.cumsum(0) - need, back.cumsum(0) - back
    top = s["count"].long() + back.sum()
    col = torch.arange(bt.shape[1], device=bt.device)
    # released blocks go onto the stack, the last sequence's last block first
    gone = (col >= has[:, None]) & (col < had[:, None])
    cell = top - 1 - (back_at[:, None] + col - has[:, None])
    free = torch.cat([s["free"], s["free"][:1]])       # one more cell takes what does not go anywhere
    free[torch.where(gone, cell, torch.full_like(cell, free.numel() - 1))] = bt
    s["free"].copy_(free[:-1])
    # and the sequences in order take theirs off it
    taken = (col >= had[:, None]) & (col < has[:, None])
    cell = (top - 1 - (need_at[:, None] + col - had[:, None])).clamp(0, s["free"].numel() - 1)
    bt.copy_(torch.where(taken, s["free"][cell], bt))
    s["new_lens"].copy_(new)
    s["new_count"].copy_(top - need.sum())
    s["cu"][:1] = 0
    s["cu"][1:] = s["change"].clamp(min=0).cumsum(0)
    t = torch.arange(s["slots"].numel(), device=bt.device)
    seq = torch.searchsorted(s["cu"][1:].contiguous(), t.to(torch.int32), right=True).clamp(max=old.numel() - 1)
    live = t < s["cu"][-1]
    pos = torch.where(live, old[seq] + t - s["cu"][seq], torch.zeros_like(t))
    s["pos"].copy_(pos)
    s["slots"].copy_(torch.where(live, bt[seq, (pos // bs).clamp(max=bt.shape[1] - 1)].long() * bs + pos % bs,
                                 torch.full_like(t, -1)))
    return _tables_out(s)


def _tables_out(s):
    return {n: s[n] for n in ("bt", "free", "new_lens", "new_count", "cu", "slots", "pos")}


def _turn(s, x, w):
    """Rows [t, heads, d] normalised (w given) and turned to their positions, in 32 bits."""
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
    n = s["freq"].numel()
    angle = s["pos"].double()[:, None, None] * s["freq"]
    cos, sin = (angle.cos() * s["factor"]).float(), (angle.sin() * s["factor"]).float()
    head, rest = y[..., :2 * n], y[..., 2 * n:]
    if s["inter"]:
        a, b = head[..., 0::2], head[..., 1::2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)
    a, b = head[..., :n], head[..., n:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _plain_rope(s):
    s["out_q"].copy_(_turn(s, s["q"], s["qw"]))
    s["kc"].flatten(0, 1)[s["slots"]] = _turn(s, s["key"], s["kw"]).to(s["dtype"])
    s["vc"].flatten(0, 1)[s["slots"]] = s["value"]
    return {"q": s["out_q"], "k": s["kc"], "v": s["vc"]}


def _quantise(x):
    """(codes, (scale, zero)) of rows [..., d], by the definition above."""
    x = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = x.amin(-1), x.amax(-1)
    # tensors on both sides of a division: a true one, not a reciprocal's product
    sc = torch.maximum((hi * 0.5 - lo * 0.5) / torch.full_like(lo, 7.5), torch.maximum(hi, -lo) * 2.0 ** -8)
    sc = sc.clamp(min=2.0 ** -60).bfloat16().float()
    zero = (lo / sc).bfloat16().float()
    u = (x * (torch.ones_like(sc) / sc)[..., None] - zero[..., None]).round().clamp(0, 15).to(torch.uint8).flatten(-2)
    return u[..., 0::2] | (u[..., 1::2] << 4), torch.stack([sc, zero], -1).bfloat16()


def _values(codes, scales):
    """Values of codes [..., d / 2] with (scale, zero) [..., d / 64, 2], in 32 bits."""
    u = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    return ((u + scales[..., 1:].float()) * scales[..., :1].float()).flatten(-2)


def _store(s, name, rows):
    codes, scales = _quantise(rows)
    s[name + "c"].flatten(0, 1)[s["slots"]] = codes
    s[name + "s"][s["slots"] // s["bs"], :, s["slots"] % s["bs"]] = scales


def _read(s, name, slots):
    return _values(s[name + "c"].flatten(0, 1)[slots], s[name + "s"][slots // s["bs"], :, slots % s["bs"]])


def _attend(s, k, v):
    """softmax(q k^T sm) v for k, v [n, hkv, length, d] in 32 bits, positions at or past ctx left out."""
    n, hq, d = s["q"].shape
    hkv, length = k.shape[1:3]
    q = s["q"].float().view(n, hkv, hq // hkv, d)
    x = torch.matmul(q, k.transpose(2, 3)) * s["sm"]
    dead = torch.arange(length, device=x.device) >= s["ctx"][:, None]
    x = x.masked_fill(dead[:, None, None], float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    return o.view(n, hq, d).to(s["dtype"])


def _plain(s):
    if s["op"] == "tables":
        return _plain_tables(s)
    if s["op"] == "rope":
        return _plain_rope(s)
    if s["op"] == "chunk4":
        _store(s, "k", s["key"])
        _store(s, "v", s["value"])
        slots = s["bt"][s["row_seq"], s["row_pos"] // s["bs"]].long() * s["bs"] + s["row_pos"] % s["bs"]
        return {"k": _read(s, "k", slots).to(s["dtype"]), "v": _read(s, "v", slots).to(s["dtype"]),
                "k_scales": s["ks"], "v_scales": s["vs"]}
    # cache slot of every position of every sequence, [n, length]; block 0 stands for missing blocks
    slots = (s["bt"].clamp(min=0).long()[:, :, None] * s["bs"] + torch.arange(s["bs"], device="cuda")).flatten(1)
    return _attend(s, _read(s, "k", slots).transpose(1, 2), _read(s, "v", slots).transpose(1, 2))


# ----------------------------------------------------------- this package

def _ours(s):
    import paged_kv_cache_140_gb300 as pa

    if s["op"] == "tables":
        pa.update_tables(s["bt"], s["lens"], s["change"], s["free"], s["count"], s["slots"], s["pos"], s["cu"], s["bs"],
                         out_lens=s["new_lens"], out_free_count=s["new_count"])
        return _tables_out(s)
    if s["op"] == "rope":
        pa.rope_and_cache(s["out_q"], s["q"], s["key"], s["value"], s["kc"], s["vc"], s["slots"], s["pos"], s["freq"],
                          interleaved=s["inter"], factor=s["factor"], q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"])
        return {"q": s["out_q"], "k": s["kc"], "v": s["vc"]}
    if s["op"] == "decode4":
        pa.int4_decode(s["out"], s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["bt"], s["ctx"], s["sm"],
                       max_context_len=s["max_ctx"])
        return s["out"]
    pa.int4_reshape_and_cache(s["key"], s["value"], s["kc"], s["vc"], s["ks"], s["vs"], s["slots"])
    pa.int4_gather(s["out_k"], s["out_v"], s["kc"], s["vc"], s["ks"], s["vs"], s["bt"], s["cu"])
    return {"k": s["out_k"], "v": s["out_v"], "k_scales": s["ks"], "v_scales": s["vs"]}


def run(state):
    return _ours(state) if own else _plain(state)


# ------------------------------------------------------- the definition, 64 bits

def _exact_tables(s):
    """One request after another, on the host."""
    bs, bt = s["bs"], s["bt"].tolist()
    old, change = s["lens"].tolist(), s["change"].tolist()
    stack, count = s["free"].tolist(), s["count"].item()
    new = [max(0, n + c) for n, c in zip(old, change)]
    for i in reversed(range(len(old))):
        for b in reversed(range(-(-new[i] // bs), -(-old[i] // bs))):
            stack[count] = bt[i][b]
            count += 1
    cu, slots, pos = [0], [], []
    for i in range(len(old)):
        for b in range(-(-old[i] // bs), -(-new[i] // bs)):
            count -= 1
            bt[i][b] = stack[count]
        for p in range(old[i], new[i]):
            slots.append(bt[i][p // bs] * bs + p % bs)
            pos.append(p)
        cu.append(len(pos))
    rest = s["slots"].numel() - len(pos)

    def like(name, v):
        return torch.tensor(v, dtype=s[name].dtype, device="cuda").view(s[name].shape)
    return {"bt": like("bt", bt), "free": like("free", stack), "new_lens": like("new_lens", new),
            "new_count": like("new_count", [count]), "cu": like("cu", cu), "slots": like("slots", slots + [-1] * rest),
            "pos": like("pos", pos + [0] * rest)}


def _exact_turn(s, case, x, w):
    y = x.double()
    if w is not None:
        size = torch.linalg.vector_norm(y, dim=-1, keepdim=True) / math.sqrt(y.shape[-1])
        y = y / torch.hypot(size, torch.full_like(size, math.sqrt(s["eps"]))) * w.double()
    n = case["rot"] // 2
    i = torch.arange(n, device="cuda")
    first, second = (2 * i, 2 * i + 1) if case["inter"] else (i, i + n)
    # the pairs as complex numbers, times factor e^(i angle)
    pairs = torch.complex(y[..., first], y[..., second])
    angle = s["pos"].double()[:, None] * s["freq"]
    turned = pairs * torch.polar(torch.full_like(angle, s["factor"]), angle)[:, None]
    out = y.clone()
    out[..., first], out[..., second] = turned.real, turned.imag
    return out


def _exact_codes(x):
    """Values that the codes of rows x stand for, and (scale, zero), in 64 bits; the definition's roundings alone."""
    f32 = lambda t: t.to(torch.float32).double()          # noqa: E731
    b16 = lambda t: t.to(torch.float32).bfloat16().double()   # noqa: E731
    g = x.double().reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    lo, hi = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
    step = f32(f32(0.5 * hi - 0.5 * lo) / 7.5)
    least = torch.where(g.abs().max(-1, keepdim=True).values / 256 > 2.0 ** -60,
                        g.abs().max(-1, keepdim=True).values / 256, torch.full_like(lo, 2.0 ** -60))
    s = b16(torch.where(step > least, step, least))
    z = b16(f32(lo / s))
    u = torch.special.round(f32(f32(g * f32(1.0 / s)) - z))
    u = torch.where(u < 0, torch.zeros_like(u), torch.where(u > 15, torch.full_like(u, 15.0), u))
    return (s * (u + z)).reshape(x.shape), torch.cat([s, z], -1)


def _exact_read(s, name, slot):
    """Rows of the cache in 64 bits, from the bytes."""
    c = s[name + "c"].flatten(0, 1)[slot].to(torch.int32)
    u = torch.empty(*c.shape[:-1], 2 * c.shape[-1], dtype=torch.float64, device="cuda")
    u[..., 0::2], u[..., 1::2] = (c % 16).double(), (c // 16).double()
    sz = s[name + "s"][slot // s["bs"], :, slot % s["bs"]].double()
    per = [torch.repeat_interleave(sz[..., j], GROUP, -1) for j in (0, 1)]
    return per[0] * (u + per[1])


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "tables":
        return _exact_tables(s)
    if s["op"] == "rope":
        got = {"q": _exact_turn(s, case, s["q"], s["qw"])}
        for n, rows in (("k", _exact_turn(s, case, s["key"], s["kw"])), ("v", s["value"].double())):
            c = torch.zeros(s[n + "c"].shape, dtype=torch.float64, device="cuda")
            c.view(-1, *c.shape[2:]).index_copy_(0, s["slots"], rows)
            got[n] = c
        return got
    if s["op"] == "chunk4":
        got = {}
        new = case["new"]
        for n, rows in (("k", s["key"]), ("v", s["value"])):
            values, sz = _exact_codes(rows)
            all_sz = s[n + "s"].double().transpose(1, 2).flatten(0, 1)
            all_sz.index_copy_(0, s["slots"], sz)
            nb = s[n + "s"].shape[0]
            got[n + "_scales"] = all_sz.view(nb, -1, *all_sz.shape[1:]).transpose(1, 2).contiguous()
            dense = torch.empty(s["out_k"].shape, dtype=torch.float64, device="cuda")
            ends = s["cu"].tolist()
            for i in range(len(ends) - 1):
                p = torch.arange(ends[i + 1] - ends[i], device="cuda")
                slot = s["bt"][i].long()[p // s["bs"]] * s["bs"] + p % s["bs"]
                dense[ends[i]:ends[i + 1]] = _exact_read(s, n, slot)
                dense[ends[i + 1] - new:ends[i + 1]] = values[i * new:(i + 1) * new]
            got[n] = dense
        return got
    n, hq, d = s["q"].shape
    hkv = case["hkv"]
    out = torch.empty(n, hq, d, dtype=torch.float64, device="cuda")
    for i, length in enumerate(s["ctx"].tolist()):
        p = torch.arange(length, device="cuda")
        slot = s["bt"][i].long()[p // s["bs"]] * s["bs"] + p % s["bs"]
        x = torch.einsum("hgd,lhd->hgl", s["q"][i].double().view(hkv, hq // hkv, d), _exact_read(s, "k", slot)) * s["sm"]
        out[i] = torch.einsum("hgl,lhd->hgd", torch.softmax(x, -1), _exact_read(s, "v", slot)).reshape(hq, d)
    return out
