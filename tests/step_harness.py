"""Plain forms of the 4-bit cache, of the rotation with the cache write and of the
block tables' update, and the inputs their tests share (CPU tensors)."""
from __future__ import annotations

import numpy as np
import torch

GROUP = 64
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------- 4-bit codes

def quantise4(x: torch.Tensor):
    """(bytes [..., D/2], scale and zero [..., D/64, 2]) of rows [..., D] by the
    definition, each fp32 step rounded once."""
    g = x.float().unflatten(-1, (-1, GROUP))
    bad = ~torch.isfinite(g).all(-1)
    g = torch.where(bad[..., None], torch.zeros_like(g), g)
    lo, hi = g.amin(-1), g.amax(-1)
    s = torch.maximum((0.5 * hi - 0.5 * lo) / 7.5, torch.maximum(hi, -lo) / 256).clamp(min=2.0 ** -60)
    s = s.bfloat16().float()
    z = (lo / s).bfloat16().float()
    u = torch.round(g * (1.0 / s)[..., None] - z[..., None]).clamp(0, 15)
    u = torch.where(bad[..., None], torch.zeros_like(u), u).to(torch.uint8).flatten(-2)
    s, z = torch.where(bad, torch.full_like(s, float("nan")), s), torch.where(bad, torch.zeros_like(z), z)
    return u[..., 0::2] | (u[..., 1::2] << 4), torch.stack([s, z], -1).bfloat16()


def values4(codes: torch.Tensor, words: torch.Tensor) -> torch.Tensor:
    """s (u + z) in 64 bits."""
    u = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double().unflatten(-1, (-1, GROUP))
    return (words[..., :1].double() * (u + words[..., 1:].double())).flatten(-2)


def size4(codes, words):
    """|s| (u + |z|): what the sums of codes and zeros are made of."""
    return values4(codes, torch.stack([words[..., 0], words[..., 1].abs()], -1)).abs()


def empty_cache4(nb, bs, hkv, d, code=0xff, scale=float("nan")):
    c = {n: torch.full((nb, bs, hkv, d // 2), code, dtype=torch.uint8) for n in "kv"}
    c.update({n + "s": torch.full((nb, hkv, bs, d // GROUP, 2), scale, dtype=torch.bfloat16) for n in "kv"})
    return c


def store4(c, n, slots, rows):
    nb, bs = c[n].shape[:2]
    codes, words = quantise4(rows)
    c[n].view(nb * bs, *c[n].shape[2:])[slots] = codes
    c[n + "s"][slots // bs, :, slots % bs] = words


def take4(c, n, slots):
    """(bytes, words) of the rows in those slots."""
    nb, bs = c[n].shape[:2]
    return c[n].view(nb * bs, *c[n].shape[2:])[slots], c[n + "s"][slots // bs, :, slots % bs]


def rows4(c, n, slots):
    return values4(*take4(c, n, slots))


def cache4(lens, bt, nb, bs, hkv, d, seed, vary=1.0, dtype="bf16", offset=0.0):
    """A cache whose used rows hold quantised random rows (sizes spread over e^+-vary, shifted by `offset` of
    them) and whose other slots hold codes 15 and NaN."""
    import quant_harness as Q
    g = torch.Generator().manual_seed(seed)
    c = empty_cache4(nb, bs, hkv, d)
    for n in "kv":
        for s, L in enumerate(lens):
            if L:
                x = torch.randn(L, hkv, d, generator=g) + offset
                x = x * torch.exp(vary * torch.randn(L, hkv, 1, generator=g))
                store4(c, n, Q.slots_of(bt, s, 0, L, bs), x.to(DT[dtype]))
    return c


# ---------------------------------------------------- norm, rotation, write

def turn(x, positions, freq, interleaved=False, factor=1.0, weight=None, eps=1e-6):
    """Rows [T, H, D] normalised (weight given) and turned, in 64 bits."""
    y = x.double()
    if weight is not None:
        y = y * weight.double() / torch.sqrt(y.square().mean(-1, keepdim=True) + eps)
    n = freq.numel()
    # the angle modulo a turn in exact arithmetic: freq as a fraction, positions as whole numbers
    from fractions import Fraction
    two_pi = Fraction(884279719003555, 140737488355328) + Fraction(9935515200043022, 2 ** 105)   # to 2^-105
    turns = torch.empty(len(positions), n, dtype=torch.float64)
    for i, f in enumerate(freq.tolist()):
        per = Fraction(f) / two_pi
        for t, p in enumerate(positions.tolist()):
            turns[t, i] = float(p * per % 1)
    angle = 2 * np.pi * turns[:, None]
    i = torch.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    out = y.clone()
    c, s = factor * torch.cos(angle), factor * torch.sin(angle)
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def turn_tolerance(x, d, dtype, factor=1.0, weight=None, eps=1e-6):
    """Worst case of the 32-bit steps of turn(), as a bound per element from the pair's size.

    The fraction of a turn and sincospi are off by 2^-24 and two units each, cos and sin by 4 x 2^-24
    in all; the norm sums d squares (d half steps at most) and takes a root of 2 units; products and
    the sum add 4 half steps: (d + 16) 2^-24 of |a| + |b|, then one rounding to dtype."""
    y = x.double()
    if weight is not None:
        y = y * weight.double() / torch.sqrt(y.square().mean(-1, keepdim=True) + eps)
    size = 2 * y.abs().amax(-1, keepdim=True) * max(1.0, abs(factor))
    return size * (d + 16) * 2.0 ** -24, (torch.finfo(DT[dtype]).eps / 2 if dtype != "f32" else 2.0 ** -24)


# ---------------------------------------------------------- block tables

def update(bt, lens, changes, free, count, bs, room):
    """The step on lists: (table, lengths, stack, count, cu, slots, positions)."""
    bt, free = [list(r) for r in bt], list(free)
    new = [max(0, n + c) for n, c in zip(lens, changes)]
    blocks = lambda n: -(-n // bs)   # noqa: E731
    for i in reversed(range(len(lens))):
        for b in reversed(range(blocks(new[i]), blocks(lens[i]))):
            free[count] = bt[i][b]
            count += 1
    cu, slots, pos = [0], [], []
    for i in range(len(lens)):
        for b in range(blocks(lens[i]), blocks(new[i])):
            count -= 1
            bt[i][b] = free[count]
        for p in range(lens[i], new[i]):
            slots.append(bt[i][p // bs] * bs + p % bs)
            pos.append(p)
        cu.append(len(pos))
    return bt, new, free, count, cu, slots + [-1] * (room - len(pos)), pos + [0] * (room - len(pos))
