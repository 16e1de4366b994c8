"""Plain 64-bit forms of the quantised-cache operators and of shared-prefix
decode, and the inputs their tests share (CPU tensors; the tests move them)."""
from __future__ import annotations

import numpy as np
import torch

QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE_DTYPE = {"e4m3": torch.uint8, "int8": torch.int8}
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
FLOOR = np.float32(2.0 ** -60)


def e4m3_values() -> np.ndarray:
    """Values of the 256 e4m3 codes (bias 7, no infinities)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


def round_e4m3(y: np.ndarray) -> np.ndarray:
    """Codes of y (|y| <= 448 up to rounding): nearest value, ties to the even code."""
    grid = e4m3_values()[:127]                       # 0 .. 448, codes 0 .. 126
    a = np.abs(y.astype(np.float64))
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def quantise(x: torch.Tensor, fmt: str):
    """(codes, scales) of rows [..., D] by the definition, each fp32 step rounded once."""
    v = x.float().numpy()
    qmax = np.float32(QMAX[fmt])
    with np.errstate(invalid="ignore", over="ignore"):
        a = np.abs(v).max(-1)
        bad = ~np.isfinite(a)
        a = np.maximum(np.where(bad, np.float32(1), a), FLOOR).astype(np.float32)
        y = (v * (qmax / a)[..., None]).astype(np.float32)
    y = np.where(bad[..., None], np.float32(0), y)
    codes = round_e4m3(y) if fmt == "e4m3" else np.rint(y).astype(np.int8)
    codes = np.where(bad[..., None], codes.dtype.type(0), codes)
    scales = np.where(bad, np.float32(np.nan), a / qmax).astype(np.float32)
    return torch.from_numpy(codes), torch.from_numpy(scales)


def values(codes: torch.Tensor, fmt: str) -> torch.Tensor:
    if fmt == "int8":
        return codes.double()
    return torch.from_numpy(e4m3_values()[codes.numpy()])


def attend(q, k, v, scale):
    """softmax(scale q k^T) v in 64 bits for q [Hq, D], k/v [L, Hkv, D]; zeros for L = 0."""
    hq, d = q.shape
    hkv = k.shape[1]
    if k.shape[0] == 0:
        return torch.zeros(hq, d, dtype=torch.float64)
    x = torch.einsum("hgd,lhd->hgl", q.double().view(hkv, hq // hkv, d), k) * float(np.float32(scale))
    return torch.einsum("hgl,lhd->hgd", torch.softmax(x, -1), v).reshape(hq, d)


def tolerance(ref, vmax, length, d, xmax, out_dtype):
    """Worst case of the kernels' 32-bit steps, as a bound on |out - ref|.

    A logit sums d products in fp32 (d / 2^24 of sum |q k|, which xmax bounds) and
    its exponential is off by that, by the rounding of x log2(e) - m and by 2 ulp
    of the exponential: xmax (d + 4) + 4 half steps.  Weights enter the product
    as two 16-bit parts (2^-17 at the least).  Up to length + 8 fp32 additions
    form the sum of the weights and as many the product (each off by half a step
    of at most the final sum of magnitudes); for int8 codes the product is summed
    with 128 added to each code, which doubles its magnitudes, and the sum of its
    weights taken off again: 4 (length + 8) in all, relative to the largest |v|.
    The output is rounded once more."""
    rel = 2.0 ** -24 * (xmax * (d + 4) + 4 + 4 * (length + 8)) + 2.0 ** -16
    tol = rel * vmax + 1e-30
    if out_dtype != "f32":
        fi = torch.finfo(DT[out_dtype])
        tol = tol + fi.eps / 2 * np.abs(ref) + fi.smallest_normal * fi.eps
    return tol


def tables(lens, bs, seed, extra=5):
    """Block table (int32 [B, max], -7 past a row's end) and pool size."""
    g = np.random.default_rng(seed)
    blocks = [-(-n // bs) for n in lens]
    nb = sum(blocks) + extra
    order = g.permutation(nb).astype(np.int32)
    bt = np.full((len(lens), max(1, max(blocks, default=1))), -7, np.int32)
    at = 0
    for s, n in enumerate(blocks):
        bt[s, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(bt), nb


def slots_of(bt, s, lo, hi, bs):
    p = torch.arange(lo, hi)
    return bt[s, p // bs].long() * bs + p % bs


def quant_cache(lens, bt, nb, bs, hkv, d, fmt, seed, vary=1.0, dtype="bf16"):
    """A cache whose used rows hold quantised random rows (row sizes spread over
    e^+-vary) and whose other slots hold the worst: NaN codes (int8: -128) and NaN scales."""
    g = torch.Generator().manual_seed(seed)
    c = {}
    for n in "kv":
        codes = torch.full((nb * bs, hkv, d), 0x7f if fmt == "e4m3" else -128, dtype=CODE_DTYPE[fmt])
        scales = torch.full((nb * bs, hkv), float("nan"))
        for s, L in enumerate(lens):
            if L == 0:
                continue
            x = torch.randn(L, hkv, d, generator=g) * torch.exp(vary * torch.randn(L, hkv, 1, generator=g))
            sl = slots_of(bt, s, 0, L, bs)
            codes[sl], scales[sl] = quantise(x.to(DT[dtype]), fmt)
        c[n] = codes.view(nb, bs, hkv, d)
        c[n + "s"] = scales.view(nb, bs, hkv)
    return c


def quant_rows(c, n, sl, fmt):
    codes, sc = c[n], c[n + "s"]
    return values(codes.view(-1, *codes.shape[2:])[sl], fmt) * sc.view(-1, sc.shape[2])[sl].double()[..., None]
