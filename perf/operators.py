"""Measured cases of the quantised paged KV cache and of shared-prefix decode.

Four operators of one decode or prefill step of one layer:

    write   K/V rows quantised into cache slots as they are written, one scale
            per token and KV head (pa.quant_reshape_and_cache)
    chunk   a prefill chunk written that way and the sequences' whole contexts
            read back as dense 16-bit rows (pa.quant_gather)
    decode  one query token per sequence attending over such a cache
            (pa.quant_decode)
    shared  one query token per sequence over a 16-bit cache, where groups of
            sequences share a long prefix that is computed once for all of the
            group (pa.decode_shared)

With ``own`` false, ``run`` computes the same results with elementary torch
operations in 32 bits; with ``own`` true it calls this package.

Quantisation, for a row x of head_dim values (one token, one KV head) and
qmax = 448 (e4m3) or 127 (int8), all in 32-bit arithmetic:
    a = max(max |x|, 2^-60),  scale = a / qmax,  code = round(x * (qmax / a))
with rounding to nearest, ties to even; the row stands for code * scale.
"""
import math
import random

import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}
AMAX_FLOOR = 2.0 ** -60
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # The smallest decode step of the tests: 4 sequences, 4 heads of 64.
        {"name": "write tiny", "op": "write", "tokens": 4, "hkv": 4, "d": 64, "bs": 16, "dtype": "f16", "fmt": "e4m3"},
        # One decode step's new rows of a 13B-shaped layer: 256 sequences, 40 heads.
        {"name": "write 13b step", "op": "write", "tokens": 256, "hkv": 40, "d": 128, "bs": 16, "dtype": "bf16",
         "fmt": "e4m3"},
        # One request's prefix hit on a grouped-query model: a 77-token tail over 1,500 cached tokens.
        {"name": "chunk tail", "op": "chunk", "seqs": 1, "new": 77, "lo": 1500, "hi": 1500, "lens": 1, "hkv": 8, "d": 128,
         "bs": 16, "dtype": "f16", "fmt": "int8"},
        # A 13B-shaped chunked prefill: 16 sequences, 512 new tokens each over 0 to 2,048 cached ones.
        {"name": "chunk 13b", "op": "chunk", "seqs": 16, "new": 512, "lo": 0, "hi": 2048, "lens": 2, "hkv": 40, "d": 128,
         "bs": 16, "dtype": "bf16", "fmt": "int8"},
        # The smallest decode step: contexts of up to 100 tokens, where the call's latency counts.
        {"name": "decode tiny", "op": "decode", "seqs": 4, "law": "uniform", "lo": 1, "hi": 100, "lens": 3, "hq": 4,
         "hkv": 4, "d": 64, "bs": 16, "dtype": "f16", "fmt": "e4m3"},
        # 13B-shaped serving batch: 256 sequences, contexts lognormal around 300 tokens, at most 2,048.
        {"name": "decode 13b", "op": "decode", "seqs": 256, "law": "lognormal", "lo": 1, "hi": 2048, "lens": 4, "hq": 40,
         "hkv": 40, "d": 128, "bs": 16, "dtype": "bf16", "fmt": "e4m3"},
        # 7B-shaped batch: 64 sequences of 32 to 2,048 tokens.
        {"name": "decode 7b", "op": "decode", "seqs": 64, "law": "uniform", "lo": 32, "hi": 2048, "lens": 5, "hq": 32,
         "hkv": 32, "d": 128, "bs": 16, "dtype": "f16", "fmt": "int8"},
        # Long contexts with grouped queries: 16 sequences of 16 K to 32 K tokens, 32 query heads on 8 KV heads.
        {"name": "decode gqa long", "op": "decode", "seqs": 16, "law": "uniform", "lo": 16384, "hi": 32768, "lens": 6,
         "hq": 32, "hkv": 8, "d": 128, "bs": 32, "dtype": "bf16", "fmt": "e4m3"},
        # Four samples of one short prompt on the smallest model.
        {"name": "shared tiny", "op": "shared", "groups": 1, "mlo": 4, "mhi": 4, "slo": 64, "shi": 64, "plo": 1, "phi": 37,
         "lens": 7, "hq": 4, "hkv": 4, "d": 64, "bs": 16, "dtype": "f16"},
        # Parallel sampling: 64 prompts of 1,000 tokens with 4 samples each, 1 to 257 private tokens.
        {"name": "shared samples", "op": "shared", "groups": 64, "mlo": 4, "mhi": 4, "slo": 1000, "shi": 1000, "plo": 1,
         "phi": 257, "lens": 8, "hq": 32, "hkv": 32, "d": 128, "bs": 16, "dtype": "f16"},
        # One system prompt of 8,192 tokens before every request of a batch of 256.
        {"name": "shared system prompt", "op": "shared", "groups": 1, "mlo": 256, "mhi": 256, "slo": 8192, "shi": 8192,
         "plo": 1, "phi": 512, "lens": 9, "hq": 32, "hkv": 8, "d": 128, "bs": 16, "dtype": "bf16"},
        # A mixed batch: 24 groups of 1 to 24 requests over prefixes of 0 to 4,096 tokens.
        {"name": "shared mixed", "op": "shared", "groups": 24, "mlo": 1, "mhi": 24, "slo": 0, "shi": 4096, "plo": 1,
         "phi": 700, "lens": 10, "hq": 32, "hkv": 8, "d": 128, "bs": 16, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["write", "chunk", "decode", "shared"])
    dtype, fmt = rng.choice(["f16", "bf16"]), rng.choice(["e4m3", "int8"])
    d, bs, lens = rng.choice([64, 128, 128]), rng.choice([8, 16, 16, 32, 64]), rng.randrange(1 << 30)
    if op == "write":
        return {"op": op, "tokens": _log(rng, 1, 2048), "hkv": rng.choice([1, 2, 3, 4, 8, 12, 32, 40]), "d": d, "bs": bs,
                "dtype": dtype, "fmt": "e4m3"}
    if op == "chunk":
        hi = _log(rng, 1, 2048)
        return {"op": op, "seqs": _log(rng, 1, 16), "new": _log(rng, 1, 512), "lo": rng.randrange(hi), "hi": hi,
                "lens": lens, "hkv": rng.choice([1, 2, 5, 8, 32, 40]), "d": d, "bs": bs, "dtype": dtype, "fmt": fmt}
    group = rng.choice([1, 2, 4, 8])
    if op == "decode":
        hkv = rng.choice([1, 2, 3, 4, 8, 8, 12, 16, 32, 40])
        seqs = _log(rng, 1, 256)
        # at most the tokens x heads of the largest listed case
        most = max(64, min(32768, 5_000_000 // (seqs * hkv)))
        hi = _log(rng, 16, most)
        return {"op": op, "seqs": seqs, "law": rng.choice(["uniform", "lognormal"]), "lo": rng.choice([1, max(1, hi // 2)]),
                "hi": hi, "lens": lens, "hq": hkv * min(group, 64 // hkv or 1) if hkv > 16 else hkv * group, "hkv": hkv,
                "d": d, "bs": bs, "dtype": dtype, "fmt": fmt}
    hkv = rng.choice([1, 2, 4, 8, 8])
    groups = _log(rng, 1, 32)
    mhi = _log(rng, 1, 256 // groups)
    shi = _log(rng, 16, max(64, min(8192, 16_000_000 // (groups * mhi * hkv))))
    return {"op": op, "groups": groups, "mlo": rng.choice([1, mhi]), "mhi": mhi, "slo": rng.choice([0, shi]), "shi": shi,
            "plo": 1, "phi": _log(rng, 1, 512), "lens": lens, "hq": hkv * group, "hkv": hkv, "d": d, "bs": bs,
            "dtype": dtype}


def _lengths(case):
    """The case's lengths, a function of the case alone.

    write: None; chunk: cached tokens per sequence; decode: context lengths;
    shared: (members per group, prefix per group, private tokens per sequence)."""
    if case["op"] == "write":
        return None
    rng = random.Random(case["lens"])
    if case["op"] == "chunk":
        return [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    if case["op"] == "decode":
        if case["law"] == "uniform":
            return [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
        mid = min(300.0, (case["lo"] + case["hi"]) / 2)
        return [min(case["hi"], max(case["lo"], round(rng.lognormvariate(math.log(mid), 1.0)))) for _ in range(case["seqs"])]
    members = [rng.randint(case["mlo"], case["mhi"]) for _ in range(case["groups"])]
    shared = [rng.randint(case["slo"], case["shi"]) for _ in range(case["groups"])]
    private = [rng.randint(case["plo"], case["phi"]) for _ in range(sum(members))]
    return members, shared, private


def work(case):
    d, hkv = case["d"], case["hkv"]
    row = d + 4                                        # one quantised row: its codes and its scale
    if case["op"] == "write":
        n = 2 * case["tokens"] * hkv
        return {"bytes": n * (2 * d + row) + 8 * case["tokens"], "flops": 3 * n * d}
    lens = _lengths(case)
    if case["op"] == "chunk":
        new = 2 * case["seqs"] * case["new"] * hkv
        both = 2 * (sum(lens) + case["seqs"] * case["new"]) * hkv
        # the new rows are read, quantised and written; every row of the contexts is read and written dense
        return {"bytes": new * (2 * d + row) + both * (row + 2 * d), "flops": 3 * new * d + both * d}
    hq = case["hq"]
    if case["op"] == "decode":
        tokens = sum(lens)
        return {"bytes": 2 * tokens * hkv * row + 4 * len(lens) * hq * d + 4 * -(-tokens // case["bs"]),
                "flops": 4 * tokens * hq * d}
    members, shared, private = lens
    once = sum(shared) + sum(private)                  # each shared token is read once for its whole group
    each = sum(m * s for m, s in zip(members, shared)) + sum(private)
    return {"bytes": 4 * once * hkv * d + 4 * len(private) * hq * d + 4 * -(-once // case["bs"]), "flops": 4 * each * hq * d}


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


def _pages(gen, blocks, width):
    """A block table: a random order of the pool's blocks dealt out to the sequences, -1 past a row's end."""
    order = torch.randperm(max(1, sum(blocks) + sum(blocks) // 8 + 1), generator=gen, device="cuda").to(torch.int32)
    begin = torch.tensor([0] + blocks[:-1], device="cuda").cumsum(0)
    count = torch.tensor(blocks, device="cuda")
    col = torch.arange(width, device="cuda")
    at = (begin[:, None] + col).clamp(max=order.numel() - 1)
    return torch.where(col < count[:, None], order[at], torch.full_like(order[:1], -1)).contiguous(), order.numel()


def _quantised(gen, slots, hkv, d, dtype, fmt, key):
    """Codes and scales of a whole cache of `slots` token slots."""
    codes = torch.empty(slots, hkv, d, dtype=torch.uint8 if fmt == "e4m3" else torch.int8, device="cuda")
    scales = torch.empty(slots, hkv, device="cuda")
    step = max(1, (1 << 28) // (hkv * d))
    for a in range(0, slots, step):
        n = min(step, slots - a)
        codes[a:a + n], scales[a:a + n] = _quantise(_rows(gen, n, hkv, d, dtype, key), fmt)
    return codes, scales


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    hkv, d, bs, dtype = case["hkv"], case["d"], case["bs"], DT[case["dtype"]]
    lens = _lengths(case)
    s = {"op": case["op"], "fmt": case.get("fmt"), "bs": bs, "dtype": dtype, "sm": 1.0 / math.sqrt(d)}

    def quantised_cache(nb, fill):
        for n in "kv":
            if fill:
                codes, scales = _quantised(gen, nb * bs, hkv, d, dtype, case["fmt"], n == "k")
            else:
                codes = torch.zeros(nb * bs, hkv, d, dtype=torch.uint8 if case["fmt"] == "e4m3" else torch.int8,
                                    device="cuda")
                scales = torch.zeros(nb * bs, hkv, device="cuda")
            s[n + "c"], s[n + "s"] = codes.view(nb, bs, hkv, d), scales.view(nb, bs, hkv)

    if case["op"] == "write":
        t = case["tokens"]
        nb = t + t // 8 + 1                            # each token goes into a block of its own, as in a decode step
        quantised_cache(nb, False)
        block = torch.randperm(nb, generator=gen, device="cuda")[:t]
        s["slots"] = block * bs + torch.randint(0, bs, (t,), generator=gen, device="cuda")
        s["key"], s["value"] = _rows(gen, t, hkv, d, dtype, True), _rows(gen, t, hkv, d, dtype, False)
        return s
    if case["op"] == "chunk":
        n, new = case["seqs"], case["new"]
        total = [c + new for c in lens]
        s["bt"], nb = _pages(gen, [-(-x // bs) for x in total], -(-max(total) // bs))
        quantised_cache(nb, True)
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
    hq = case["hq"]
    if case["op"] == "decode":
        n, ctx = case["seqs"], lens
        s["bt"], nb = _pages(gen, [-(-x // bs) for x in ctx], -(-max(ctx) // bs))
        quantised_cache(nb, True)
    else:
        members, shared, private = lens
        n = sum(members)
        group = [g for g, m in enumerate(members) for _ in range(m)]
        ctx = [shared[g] + private[i] for i, g in enumerate(group)]
        # whole prefix blocks are shared; the block where a prefix ends is each sequence's own copy
        common = [x // bs for x in shared]
        width = -(-max(ctx) // bs)
        front, nf = _pages(gen, [max(1, x) for x in common], max(1, max(common)))
        own_blocks = [-(-ctx[i] // bs) - common[g] for i, g in enumerate(group)]
        back, nback = _pages(gen, own_blocks, max(1, max(own_blocks)))
        gi, ci = torch.tensor(group, device="cuda"), _int32(common)
        col = torch.arange(width, device="cuda")
        head = ci[gi][:, None].long()
        in_front = front[gi][:, torch.clamp(col, max=front.shape[1] - 1)]
        in_back = back.gather(1, (col - head).clamp(0, back.shape[1] - 1))
        used = col < torch.tensor([-(-x // bs) for x in ctx], device="cuda")[:, None]
        bt = torch.where(col < head, in_front, torch.where(in_back >= 0, in_back + nf, in_back))
        s["bt"] = torch.where(used, bt, torch.full_like(bt, -1)).contiguous()
        nb = nf + nback
        for name in "kv":
            s[name + "c"] = torch.empty(nb * bs, hkv, d, dtype=dtype, device="cuda")
            step = max(1, (1 << 28) // (hkv * d))
            for a in range(0, nb * bs, step):
                m = min(step, nb * bs - a)
                s[name + "c"][a:a + m] = _rows(gen, m, hkv, d, dtype, name == "k")
            s[name + "c"] = s[name + "c"].view(nb, bs, hkv, d)
        # the copies of a block where a prefix ends hold the same prefix rows
        first = torch.tensor([sum(members[:g]) for g in range(len(members))], device="cuda")[gi]
        tail = _int32(shared)[gi] % bs
        at = (ci[gi].long()[:, None]).clamp(max=width - 1)
        src, dst = s["bt"][first].gather(1, at)[:, 0].long(), s["bt"].gather(1, at)[:, 0].long()
        keep = torch.arange(bs, device="cuda") < tail[:, None]
        keep &= (src >= 0)[:, None] & (dst >= 0)[:, None]
        for name in "kv":
            c = s[name + "c"]
            c[dst] = torch.where(keep[:, :, None, None], c[src], c[dst])
        s["cu_groups"] = _int32([0] + members).cumsum(0).to(torch.int32)
        s["shared"] = _int32([shared[g] for g in group])
        s["max_group"], s["max_shared"] = max(members), max(shared)
    s["q"] = (2.0 * torch.randn(n, hq, d, generator=gen, device="cuda")).to(dtype)
    s["ctx"], s["max_ctx"] = _int32(ctx), max(ctx)
    s["out"] = torch.empty_like(s["q"])
    return s


# ------------------------------------------------------------ the plain form

def _quantise(x, fmt):
    """(codes, scales) of rows [..., d], by the definition above."""
    x = x.float()
    a = x.abs().amax(-1).clamp(min=AMAX_FLOOR)
    top = torch.full_like(a, QMAX[fmt])                # tensors on both sides: a true division, not a reciprocal's product
    y = x * (top / a)[..., None]
    codes = y.to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "e4m3" else y.round().to(torch.int8)
    return codes, a / top


def _values(codes, fmt):
    return codes.view(torch.float8_e4m3fn).float() if fmt == "e4m3" else codes.float()


def _store(s, name, rows):
    codes, scales = _quantise(rows, s["fmt"])
    s[name + "c"].view(-1, *codes.shape[1:])[s["slots"]] = codes
    s[name + "s"].view(-1, scales.shape[1])[s["slots"]] = scales


def _read(s, name, slots):
    c, sc = s[name + "c"], s[name + "s"]
    return _values(c.view(-1, *c.shape[2:])[slots], s["fmt"]) * sc.view(-1, sc.shape[2])[slots][..., None]


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


def _slots_of(s):
    """Cache slot of every position of every sequence, [n, length]; block 0 stands for missing blocks."""
    at = s["bt"].clamp(min=0).long()[:, :, None] * s["bs"] + torch.arange(s["bs"], device="cuda")
    return at.view(at.shape[0], -1)


def _plain(s):
    if s["op"] == "write":
        _store(s, "k", s["key"])
        _store(s, "v", s["value"])
        return _written(s)
    if s["op"] == "chunk":
        _store(s, "k", s["key"])
        _store(s, "v", s["value"])
        slots = s["bt"][s["row_seq"], s["row_pos"] // s["bs"]].long() * s["bs"] + s["row_pos"] % s["bs"]
        return {"k": _read(s, "k", slots).to(s["dtype"]), "v": _read(s, "v", slots).to(s["dtype"]),
                "k_scales": s["ks"], "v_scales": s["vs"]}
    slots = _slots_of(s)
    if s["op"] == "decode":
        k, v = _read(s, "k", slots), _read(s, "v", slots)
    else:
        k, v = s["kc"].flatten(0, 1)[slots].float(), s["vc"].flatten(0, 1)[slots].float()
    return _attend(s, k.transpose(1, 2), v.transpose(1, 2))


def _written(s):
    return {"k": s["kc"].view(torch.float8_e4m3fn), "v": s["vc"].view(torch.float8_e4m3fn),
            "k_scales": s["ks"], "v_scales": s["vs"]}


# ----------------------------------------------------------- this package

def _ours(s):
    import paged_kv_cache_140_gb300 as pa

    if s["op"] == "decode":
        pa.quant_decode(s["out"], s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["bt"], s["ctx"], s["sm"],
                        max_context_len=s["max_ctx"])
        return s["out"]
    if s["op"] == "shared":
        pa.decode_shared(s["out"], s["q"], s["kc"], s["vc"], s["bt"], s["ctx"], s["cu_groups"], s["shared"], s["sm"],
                         max_group_size=s["max_group"], max_shared_len=s["max_shared"], max_context_len=s["max_ctx"])
        return s["out"]
    pa.quant_reshape_and_cache(s["key"], s["value"], s["kc"], s["vc"], s["ks"], s["vs"], s["slots"])
    if s["op"] == "write":
        return _written(s)
    pa.quant_gather(s["out_k"], s["out_v"], s["kc"], s["vc"], s["ks"], s["vs"], s["bt"], s["cu"])
    return {"k": s["out_k"], "v": s["out_v"], "k_scales": s["ks"], "v_scales": s["vs"]}


def run(state):
    return _ours(state) if own else _plain(state)


# ------------------------------------------------------- the definition, 64 bits

def _grid(x, fmt):
    """(code values, scales) of rows x in 64 bits; the three 32-bit roundings are the definition's own."""
    f32 = lambda t: t.to(torch.float32).double()  # noqa: E731
    x = x.double()
    a = x.abs().max(dim=-1).values
    a = torch.where(a < AMAX_FLOOR, torch.full_like(a, AMAX_FLOOR), a)
    scale, inverse = f32(a / QMAX[fmt]), f32(QMAX[fmt] / a)
    y = f32(x * inverse.unsqueeze(-1))
    if fmt == "int8":
        return torch.special.round(y), scale
    e = torch.frexp(y).exponent.double() - 1.0         # 2^e <= |y| < 2^(e + 1)
    step = torch.exp2(torch.where(e < -6.0, torch.full_like(e, -6.0), e) - 3.0)
    return (torch.special.round(y / step) * step).clamp(-448.0, 448.0), scale


def _code_values(codes, fmt):
    """Values of stored codes in 64 bits, from their bits."""
    if fmt == "int8":
        return codes.double()
    c = codes.to(torch.int32)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2(e.double() - 10.0))
    return torch.where(c >= 128, -v, v)


def exact(case, seed):
    s = prepare(case, seed)
    fmt = s["fmt"]
    if s["op"] in ("write", "chunk"):
        got = {}
        for n, rows in (("k", s["key"]), ("v", s["value"])):
            values, scales = _grid(rows, fmt)
            sc = s[n + "s"].double().flatten(0, 1)
            sc.index_copy_(0, s["slots"], scales)
            got[n + "_scales"] = sc.view(s[n + "s"].shape)
            if s["op"] == "write":
                cache = torch.zeros(s[n + "c"].shape, dtype=torch.float64, device="cuda").flatten(0, 1)
                cache.index_copy_(0, s["slots"], values)
                got[n] = cache.view(s[n + "c"].shape)
                continue
            codes = s[n + "c"].flatten(0, 1)
            dense = torch.empty(s["out_k"].shape, dtype=torch.float64, device="cuda")
            ends, at = s["cu"].tolist(), 0
            for i in range(len(ends) - 1):
                rows_i = ends[i + 1] - ends[i]
                p = torch.arange(rows_i, device="cuda")
                slot = s["bt"][i].long()[p // s["bs"]] * s["bs"] + p % s["bs"]
                dense[ends[i]:ends[i + 1]] = _code_values(codes[slot], fmt) * sc[slot].unsqueeze(-1)
                new = values[at:at + case["new"]] * scales[at:at + case["new"]].unsqueeze(-1)
                dense[ends[i + 1] - case["new"]:ends[i + 1]] = new
                at += case["new"]
            got[n] = dense
        return got
    n, hq, d = s["q"].shape
    hkv = case["hkv"]
    out = torch.empty(n, hq, d, dtype=torch.float64, device="cuda")
    for i, length in enumerate(s["ctx"].tolist()):
        p = torch.arange(length, device="cuda")
        slot = s["bt"][i].long()[p // s["bs"]] * s["bs"] + p % s["bs"]

        def rows(name):
            c = s[name + "c"].flatten(0, 1)[slot]
            if s["op"] == "shared":
                return c.double()
            return _code_values(c, fmt) * s[name + "s"].flatten(0, 1)[slot].double().unsqueeze(-1)

        x = torch.einsum("hgd,lhd->hgl", s["q"][i].double().view(hkv, hq // hkv, d), rows("k")) * s["sm"]
        out[i] = torch.einsum("hgl,lhd->hgd", torch.softmax(x, -1), rows("v")).reshape(hq, d)
    return out
