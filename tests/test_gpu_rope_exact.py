"""GPU tests of what the rotation with the cache write leaves as it is, and of its angles and bytes where
ordinary sizes cannot show them: far positions, high frequencies, calls of few and of many tokens."""
from fractions import Fraction

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_140_gb300 as pa

import step_harness as S
from test_gpu_rope import KINDS, caches, inputs, rope_write, slots_for, write

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_140_gb300 import _build
    _build.build()


# ------------------------------------------------------ few and many tokens

@pytest.mark.parametrize("interleaved,rot,d", [(False, 64, 64), (True, 32, 128), (False, 128, 128)])
@pytest.mark.parametrize("kind", KINDS + ["half"])
def test_many_normalised_tokens_make_the_bytes_of_few(kind, interleaved, rot, d):
    """One call of 163 tokens of 120 rows, and calls of 20 and less, which take another form of the kernel: a
    token's bytes do not depend on how many others come with it, norms of queries and keys included."""
    T, hq, hkv, bs, nb = 163, 64, 28, 16, 12
    _, dev, pos = inputs(T, hq, hkv, d, "bf16", seed=5)
    g = torch.Generator().manual_seed(2)
    qw, kw = ((1 + 0.3 * torch.randn(d, generator=g)).bfloat16().cuda() for _ in "qk")
    slots = torch.randperm(nb * bs, generator=torch.Generator().manual_seed(0))[:T].cuda()
    pos = pos.cuda()
    freq, _ = pa.rope_frequencies(rot)
    made = []
    for step in (T, 20):
        if kind == "half":
            c = {n: torch.full((nb, bs, hkv, d), 3.0, dtype=torch.bfloat16, device="cuda") for n in "kv"}
        else:
            c = caches(kind, nb, bs, hkv, d)
        out = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
        for t in range(0, T, step):
            part, a, s = [x[t:t + step] for x in dev], out[t:t + step], slots[t:t + step]
            kws = dict(interleaved=interleaved, q_weight=qw, k_weight=kw)
            if kind == "half":
                pa.rope_and_cache(a, *part, c["k"], c["v"], s, pos[t:t + step], freq, **kws)
            else:
                rope_write(kind, a, part, c, s, pos[t:t + step], freq, **kws)
        made.append([out.view(torch.uint8)] + [x.view(torch.uint8) for x in c.values()])
    for a, b in zip(*made):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ angles

def turns_of(position, f):
    """position * f / 2 pi modulo 1, with pi to 2^-380 by Machin's formula."""
    def arctan(n):          # of 1 / n
        t = (1 << 400) // n
        total, k, sign = t, 1, -1
        while t:
            t //= n * n
            k += 2
            total += sign * (t // k)
            sign = -sign
        return total
    pi = Fraction(4 * (4 * arctan(5) - arctan(239)), 1 << 400)
    return float(position * Fraction(f) / (2 * pi) % 1)


FAR = [(p, f) for f in (1.0, 1.9999, 0.3, 10000.0 ** -0.9, 3.7, 977.0, 2.0 ** 19 + 0.123, 2.0 ** 20 - 2.0 ** -30, 2.0 ** -60)
       for p in (1, 12345, 2 ** 22 + 1, 2 ** 30 + 7, 2 ** 40 + 3, 2 ** 45 - 1, 2 ** 50 + 99, 2 ** 62 + 12345, 2 ** 63 - 1)]


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_of_far_positions_and_high_frequencies(interleaved, sign):
    """A key of one element, 1 in the first place of its only pair, turns to (cos, sin) of the angle, and the larger of
    the two stands in the row's scale with 32 bits.

    In units of 2^-24: the angle's fraction of a turn, a 64-bit number within [-1/2, 1/2), is rounded to 24
    bits (half a unit 2^-25 of half a turn: pi / 2 of an angle), which moves the larger of cos and sin by at most
    0.71 of that, 1.12; sincospi is off by two units in the last place of a number in [1/2, 1], 2; the product with
    the factor 1 and the sum with 0 are exact, the scale's division is off by 1/2: below 4.  The angle itself
    may be off by 2^-24 more."""
    n, d, bs = len(FAR), 64, 16
    got = torch.empty(n, dtype=torch.float64)
    for i, (p, f) in enumerate(FAR):
        key = torch.zeros(1, 1, d, dtype=torch.float16, device="cuda")
        key[0, 0, 0] = 1
        freq = torch.zeros(4, dtype=torch.float64, device="cuda")
        freq[0] = f * (-1 if i % 3 == 0 else 1)
        c = caches("int8", 1, bs, 1, d)
        q = torch.zeros(1, 1, d, dtype=torch.float16, device="cuda")
        rope_write("int8", torch.empty_like(q), [q, key, key], c, torch.zeros(1, dtype=torch.int64, device="cuda"),
                   torch.tensor([sign * p], device="cuda"), freq, interleaved=interleaved)
        got[i] = c["ks"].view(-1)[0].double().item() * 127
        codes = c["k"].view(-1, d)[0, [0, 1 if interleaved else 4]].double().cpu()
        want = 2 * np.pi * turns_of(sign * p, freq[0].item())
        pair = torch.tensor([np.cos(want), np.sin(want)], dtype=torch.float64)
        assert abs(got[i] - pair.abs().max()) <= 5 * 2.0 ** -24, (p, f, (got[i] - pair.abs().max()) * 2 ** 24)
        # both signs and the smaller one: to half a code
        assert ((codes * got[i] / 127 - pair).abs() <= 0.5 / 127 + 2.0 ** -20).all(), (p, f)


@pytest.mark.parametrize("kind", ["int8", "half"])
def test_near_and_far_positions_in_one_call(kind):
    """Tokens of ordinary and of far positions, negative ones too, and frequencies on both sides of 2: the bytes that
    each has in a call of its own."""
    T, hq, hkv, d, bs, nb = 66, 300, 3, 64, 16, 5
    _, dev, pos = inputs(T, hq, hkv, d, "bf16", seed=5)
    pos[1::2] = 2 ** 31 + pos[1::2] * 2 ** 40
    pos[2::4] *= -1
    pos[3::4] *= -1
    pos[4], pos[5], pos[6] = 2 ** 31 - 1, -2 ** 31, -2 ** 31 - 1
    pos = pos.cuda()
    freq, _ = pa.rope_frequencies(d)
    freq[3:6] = torch.tensor([2.0, -3.5, 1.9999], device="cuda", dtype=torch.float64)
    slots = torch.randperm(nb * bs, generator=torch.Generator().manual_seed(0))[:T].cuda()
    made = []
    for step in (T, 1):
        c = caches(kind, nb, bs, hkv, d) if kind == "int8" else \
            {n: torch.full((nb, bs, hkv, d), 3.0, dtype=torch.bfloat16, device="cuda") for n in "kv"}
        out = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
        for t in range(0, T, step):
            part = [x[t:t + step] for x in dev]
            scales = dict(k_scales=c["ks"], v_scales=c["vs"]) if kind == "int8" else {}
            pa.rope_and_cache(out[t:t + step], *part, c["k"], c["v"], slots[t:t + step], pos[t:t + step], freq, **scales)
        made.append([out.view(torch.uint8)] + [x.view(torch.uint8) for x in c.values()])
    for a, b in zip(*made):
        assert torch.equal(a, b)


# ------------------------------------------------------------ bytes as they are

@pytest.mark.parametrize("T", [5, 1100])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_values_go_into_a_16_bit_cache_bit_for_bit(dtype, T):
    """Every one of the 65,536 numbers of the type (of 5 tokens, some), NaNs of any bits among them."""
    hkv, d, bs = 1, 64, 16
    (q, k, v), dev, pos = inputs(T, 32, hkv, d, dtype, wide=False)
    bits = torch.arange(T * d) if T * d >= 65536 else torch.arange(65536 - T * d, 65536)
    dev[2] = (bits % 65536).to(torch.int32).to(torch.int16).view(S.DT[dtype]).view(T, hkv, d).cuda()
    slots = slots_for(T, T // bs + 3, bs, skip=False).cuda()
    freq, _ = pa.rope_frequencies(d)
    made = []
    for rope in (True, False):
        kc, vc = (torch.full((T // bs + 3, bs, hkv, d), 3.0, dtype=S.DT[dtype], device="cuda") for _ in "kv")
        if rope:
            pa.rope_and_cache(torch.empty_like(dev[0]), *dev, kc, vc, slots, pos.cuda(), freq)
        else:
            pa.reshape_and_cache(dev[1], dev[2], kc, vc, slots)
        made.append(vc.view(torch.int16))
    assert torch.equal(*made)


@pytest.mark.parametrize("d", [64, 128])
def test_one_scale_per_tensor_makes_the_bytes_of_the_write(d):
    """Keys at position 0 and values, saturated ones, infinities and NaN among them, for either head size."""
    T, hq, hkv, bs = 70, 3, 5, 16
    _, dev, pos = inputs(T, hq, hkv, d, "bf16")
    for t in dev[1:]:      # (beyond the 16 elements that are turned: infinity times a sine of 0 is no number)
        t[3, 1] = 0
        t[4, 2, 37], t[5, 0, 39], t[6, 1, 32] = float("inf"), float("nan"), float("-inf")
        t[7] *= 1000
    slots = slots_for(T, 8, bs).cuda()
    got, want = caches("tensor", 8, bs, hkv, d), caches("tensor", 8, bs, hkv, d)
    freq, _ = pa.rope_frequencies(16)
    rope_write("tensor", torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda"), dev, got, slots, 0 * pos.cuda(), freq)
    write("tensor", dev[1].contiguous(), dev[2].contiguous(), want, slots)
    for n in got:
        assert torch.equal(got[n], want[n]), n
