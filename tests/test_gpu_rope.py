"""GPU tests of the norm, rotation and cache write in one pass, against 64 bits and
against the calls that it stands for."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_140_gb300 as pa

import quant_harness as Q
import step_harness as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_140_gb300 import _build
    _build.build()


def inputs(T, hq, hkv, d, dtype, seed=0, wide=True, far=100000):
    g = torch.Generator().manual_seed(seed)
    rows = torch.randn(T, (hq + 2 * hkv), d, generator=g) * torch.exp(torch.randn(T, hq + 2 * hkv, 1, generator=g))
    rows = rows.to(S.DT[dtype])
    q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    pos = torch.randint(0, far, (T,), generator=g)
    if wide:      # slices of one projection's output, with a gap behind
        buf = torch.zeros(T, (hq + 2 * hkv) * d + 40, dtype=S.DT[dtype], device="cuda")
        buf[:, :(hq + 2 * hkv) * d] = rows.reshape(T, -1).cuda()
        dev = [buf[:, a * d:b * d].view(T, b - a, d) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv))]
    else:
        dev = [t.contiguous().cuda() for t in (q, k, v)]
    return (q, k, v), dev, pos


def slots_for(T, nb, bs, seed=0, skip=True):
    g = np.random.default_rng(seed)
    slots = g.permutation(nb * bs)[:T].astype(np.int64)
    if skip and T > 2:
        slots[g.random(T) < 0.1] = -1
    return torch.from_numpy(slots)


def check(T, hq, hkv, d, bs, dtype, rot=None, interleaved=False, norm="both", factor=1.0, scaling=None, seed=0, wide=True,
          far=100000, eps=1e-6, base=10000.0, inplace=False):
    rot = rot or d
    (q, k, v), dev, pos = inputs(T, hq, hkv, d, dtype, seed, wide, far)
    freq, _ = pa.rope_frequencies(rot, base=base, scaling=scaling, scale=8.0 if scaling else 1.0)
    g = torch.Generator().manual_seed(seed + 1)
    qw, kw = ((1 + 0.3 * torch.randn(d, generator=g)).to(S.DT[dtype]) for _ in "qk")
    qw, kw = (qw if norm in ("both", "q") else None), (kw if norm in ("both", "k") else None)
    nb = T // bs + 3
    slots = slots_for(T, nb, bs, seed)
    kc, vc = (torch.full((nb, bs, hkv, d), 3.0, dtype=S.DT[dtype], device="cuda") for _ in "kv")
    out = dev[0] if inplace else torch.full((T, hq, d), float("nan"), dtype=S.DT[dtype], device="cuda")
    err = pa.new_err_flag()
    pa.rope_and_cache(out, *dev, kc, vc, slots.cuda(), pos.cuda(), freq, interleaved=interleaved, factor=factor,
                      q_weight=None if qw is None else qw.cuda(), k_weight=None if kw is None else kw.cuda(), eps=eps,
                      err_flag=err)
    assert pa.read_err_flag(err) == 0
    keep = slots >= 0
    for name, x, w, got in (("q", q, qw, out.cpu()),
                            ("k", k[keep], kw, kc.cpu().view(nb * bs, hkv, d)[slots[keep]])):
        p = pos if name == "q" else pos[keep]
        ref = S.turn(x, p, freq.cpu(), interleaved, factor, w, eps)
        tol, half = S.turn_tolerance(x, d, dtype, factor, w, eps)
        bad = (got.double() - ref).abs() - (tol + half * ref.abs() + torch.finfo(S.DT[dtype]).smallest_normal)
        assert bad.max() <= 0, (name, bad.max())
    want = torch.full((nb * bs, hkv, d), 3.0, dtype=S.DT[dtype])
    want[slots[keep]] = v[keep]
    assert torch.equal(vc.cpu().view(nb * bs, hkv, d), want)
    rest = torch.ones(nb * bs, dtype=torch.bool)
    rest[slots[keep]] = False
    assert torch.all(kc.cpu().view(nb * bs, hkv, d)[rest] == 3)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,hq,hkv,d,rot", [(1, 1, 1, 64, 64), (3, 4, 4, 64, 16), (7, 5, 1, 128, 128), (19, 8, 2, 128, 32),
                                            (5, 40, 40, 128, 128), (2, 3, 3, 128, 8), (33, 6, 3, 64, 56), (4, 2, 1, 128, 120)])
def test_rows(T, hq, hkv, d, rot, dtype, interleaved):
    check(T, hq, hkv, d, 16, dtype, rot, interleaved)


@pytest.mark.parametrize("norm", ["none", "q", "k"])
def test_norms_of_either(norm):
    check(9, 4, 2, 128, 16, "bf16", norm=norm)


@pytest.mark.parametrize("T,hq,hkv,d", [(2600, 8, 2, 64), (611, 40, 40, 128), (3001, 1, 1, 128)])
def test_many_tokens(T, hq, hkv, d):
    check(T, hq, hkv, d, 32, "bf16", rot=32, far=4096)


@pytest.mark.parametrize("scaling", ["linear", "base", "parts"])
def test_scalings_and_far_positions(scaling):
    check(6, 4, 2, 128, 16, "f16", scaling=scaling, far=1 << 40, factor=1.2, norm="none")


def test_in_place():
    check(5, 4, 2, 128, 16, "bf16", wide=False, inplace=True)
    check(300, 4, 2, 64, 16, "f16", wide=False, inplace=True, interleaved=True, rot=32)


def test_negative_positions_turn_back():
    (q, k, v), dev, pos = inputs(4, 2, 1, 64, "f16", wide=False)
    freq, _ = pa.rope_frequencies(64)
    kc, vc = (torch.zeros(1, 16, 1, 64, dtype=torch.float16, device="cuda") for _ in "kv")
    out = torch.empty_like(dev[0])
    pa.rope_and_cache(out, *dev, kc, vc, torch.arange(4, device="cuda"), -pos.cuda(), freq)
    ref = S.turn(q, -pos, freq.cpu())
    tol, half = S.turn_tolerance(q, 64, "f16")
    assert torch.all((out.cpu().double() - ref).abs() <= tol + half * ref.abs() + 1e-7)


def test_zero_rows_and_no_numbers():
    """A row of zeros stays zeros under a norm; a NaN stays in its row."""
    (q, k, v), dev, pos = inputs(3, 2, 1, 128, "bf16", wide=False)
    dev[0][0, 0] = 0
    dev[0][1, 1, 5] = float("nan")
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    freq, _ = pa.rope_frequencies(128)
    kc, vc = (torch.zeros(1, 16, 1, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    out = torch.empty_like(dev[0])
    pa.rope_and_cache(out, *dev, kc, vc, torch.arange(3, device="cuda"), pos.cuda(), freq, q_weight=w)
    assert torch.all(out[0, 0] == 0) and torch.all(out[1, 1].isnan())
    assert torch.all(out[0, 1].isfinite()) and torch.all(out[1, 0].isfinite()) and torch.all(out[2].isfinite())


def test_bad_slot_is_skipped_and_reported():
    (q, k, v), dev, pos = inputs(3, 2, 1, 64, "f16", wide=False)
    freq, _ = pa.rope_frequencies(64)
    kc, vc = (torch.zeros(2, 16, 1, 64, dtype=torch.float16, device="cuda") for _ in "kv")
    err = pa.new_err_flag()
    out = torch.empty_like(dev[0])
    pa.rope_and_cache(out, *dev, kc, vc, torch.tensor([32, 7, 10 ** 12], device="cuda"), pos.cuda(), freq, err_flag=err)
    assert pa.read_err_flag(err) == pa.FLAG_BAD_SLOT
    assert (vc.view(32, -1) != 0).any(-1).nonzero().flatten().tolist() == [7]
    assert torch.all(out.isfinite())


# ------------------------------------------------- caches of codes

KINDS = ["tensor", "e4m3", "int8", "int4"]


def caches(kind, nb, bs, hkv, d):
    if kind == "int4":
        c = {n: t.cuda() for n, t in S.empty_cache4(nb, bs, hkv, d, 3, 5.0).items()}
    else:
        c = {n: torch.full((nb, bs, hkv, d), 3, dtype=Q.CODE_DTYPE["int8" if kind == "int8" else "e4m3"], device="cuda")
             for n in "kv"}
        if kind != "tensor":
            c.update({n + "s": torch.full((nb, bs, hkv), 5.0, device="cuda") for n in "kv"})
    return c


def write(kind, key, value, c, slots):
    if kind == "tensor":
        pa.reshape_and_cache(key, value, c["k"], c["v"], slots, k_scale=0.06, v_scale=0.03)
    else:
        f = pa.int4_reshape_and_cache if kind == "int4" else pa.quant_reshape_and_cache
        f(key, value, c["k"], c["v"], c["ks"], c["vs"], slots)


def rope_write(kind, out, dev, c, slots, pos, freq, **kw):
    scales = dict(k_scale=0.06, v_scale=0.03) if kind == "tensor" else dict(k_scales=c["ks"], v_scales=c["vs"])
    pa.rope_and_cache(out, *dev, c["k"], c["v"], slots, pos, freq, **scales, **kw)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", KINDS)
def test_values_and_unturned_keys_are_the_same_bytes_as_the_write_makes(kind, d):
    """Position 0 turns nothing: keys and values as the cache's own write makes them, bit for bit."""
    T, hq, hkv, bs = 70, 3, 5, 16
    _, dev, pos = inputs(T, hq, hkv, d, "bf16")
    dev[1][3, 1] = 0
    dev[2][4, 2, 7] = float("inf")
    dev[2][5, 0, 9] = float("nan")
    slots = slots_for(T, 8, bs).cuda()
    got, want = caches(kind, 8, bs, hkv, d), caches(kind, 8, bs, hkv, d)
    freq, _ = pa.rope_frequencies(16)
    out = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
    if kind == "tensor" and d == 64:     # pa.reshape_and_cache takes such caches for D 128 only; the codes are the same
        one = caches(kind, 8, bs, hkv, d)
        rope_write(kind, out, dev, one, slots, 0 * pos.cuda(), freq)
        keep = (slots >= 0).nonzero().flatten()
        codes = one["v"].view(-1, hkv, d)[slots[keep]].view(torch.float8_e4m3fn).float()
        # a true division in 32 bits, as the cache's scale is defined (a scalar divisor is a product on the GPU)
        x = torch.from_numpy(dev[2][keep].float().cpu().numpy() / np.float32(0.03))
        ok = x.abs() < 448
        assert torch.equal(codes.cpu()[ok], x.to(torch.float8_e4m3fn).float()[ok])
        return
    rope_write(kind, out, dev, got, slots, 0 * pos.cuda(), freq)
    write(kind, dev[1].contiguous(), dev[2].contiguous(), want, slots)
    for n in got:
        a, b = (t.view(torch.uint8) if t.dtype in (torch.uint8, torch.int8) else t for t in (got[n], want[n]))
        assert torch.equal(a.float().nan_to_num(7.0), b.float().nan_to_num(7.0)), n


@pytest.mark.parametrize("interleaved,rot", [(False, 128), (False, 32), (True, 64), (True, 128), (False, 72)])
@pytest.mark.parametrize("kind", KINDS)
def test_turned_keys_as_codes(kind, interleaved, rot):
    """Codes stand for the turned row to within half a step, and its 32-bit error."""
    T, hq, hkv, d, bs = 40, 2, 3, 128, 16
    (q, k, v), dev, pos = inputs(T, hq, hkv, d, "bf16", seed=3)
    slots = torch.randperm(64, generator=torch.Generator().manual_seed(0))[:T]
    c = caches(kind, 4, bs, hkv, d)
    freq, _ = pa.rope_frequencies(rot)
    w = (1 + 0.3 * torch.randn(d)).bfloat16()
    out = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
    rope_write(kind, out, dev, c, slots.cuda(), pos.cuda(), freq, interleaved=interleaved, k_weight=w.cuda())
    ref = S.turn(k, pos, freq.cpu(), interleaved, 1.0, w)
    tol, _ = S.turn_tolerance(k, d, "f32", weight=w)
    if kind == "int4":
        c = {n: t.cpu() for n, t in c.items()}
        got = S.rows4(c, "k", slots)
        step = c["ks"][slots // bs, :, slots % bs][..., 0].double().repeat_interleave(64, -1)
        zero = c["ks"][slots // bs, :, slots % bs][..., 1].double().abs().repeat_interleave(64, -1)
        # half a code, what s lacks of a fifteenth of the range (2^-8 of 15 codes), the rounding of z (2^-8 of it)
        bound = step * (0.5 + 15 * 2.0 ** -8 + zero * 2.0 ** -8) + 2 * tol
    else:
        codes = c["k"].cpu().view(-1, hkv, d)[slots]
        val = Q.values(codes, "int8" if kind == "int8" else "e4m3")
        sc = torch.tensor(0.06, dtype=torch.float32).double().expand(T, hkv, 1) if kind == "tensor" else \
            c["ks"].cpu().view(-1, hkv)[slots].double()[..., None]
        got = val * sc
        half = 0.5 * sc if kind == "int8" else torch.maximum(ref.abs() * 2.0 ** -4, sc * 2.0 ** -10)
        bound = half * (1 + 1e-5) + 2 * tol
        if kind == "tensor":     # beyond 448 codes saturate
            inside = ref.abs() < 440 * sc
            got, ref, bound = torch.where(inside, got, ref), ref, bound
    assert torch.all((got - ref).abs() <= bound), ((got - ref).abs() / bound).max()


@pytest.mark.parametrize("interleaved,rot,d", [(False, 64, 64), (True, 32, 128), (False, 128, 128)])
@pytest.mark.parametrize("kind", KINDS + ["half"])
def test_many_tokens_make_the_bytes_of_few(kind, interleaved, rot, d):
    """One call of 163 tokens of 120 rows, four tokens at a time, and calls of 20 and less, one by one: the same
    operations on every element, so the same bytes."""
    T, hq, hkv, bs, nb = 163, 64, 28, 16, 12
    _, dev, pos = inputs(T, hq, hkv, d, "bf16", seed=5)
    dev[1][11, 3, 7] = float("inf")
    dev[2][161, 27, d - 1] = float("nan")
    slots = torch.randperm(nb * bs, generator=torch.Generator().manual_seed(0))[:T]
    slots[::17] = -1
    slots, pos = slots.cuda(), pos.cuda()
    freq, _ = pa.rope_frequencies(rot)
    made = []
    for step in (T, 20):
        if kind == "half":
            c = {n: torch.full((nb, bs, hkv, d), 3.0, dtype=torch.bfloat16, device="cuda") for n in "kv"}
        else:
            c = caches(kind, nb, bs, hkv, d)
        out = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
        for t in range(0, T, step):
            part = [x[t:t + step] for x in dev]
            if kind == "half":
                pa.rope_and_cache(out[t:t + step], *part, c["k"], c["v"], slots[t:t + step], pos[t:t + step], freq,
                                  interleaved=interleaved)
            else:
                rope_write(kind, out[t:t + step], part, c, slots[t:t + step], pos[t:t + step], freq, interleaved=interleaved)
        made.append([out.view(torch.uint8)] + [x.view(torch.uint8) for x in c.values()])
    for a, b in zip(*made):
        assert torch.equal(a, b)
