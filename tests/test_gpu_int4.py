"""GPU tests of the cache of 4-bit codes: write and read-back bit for bit, decode
against its 64-bit plain form, and a run of them together."""
import threading

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


def same(a, b):
    """Equal values, NaN where NaN."""
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())


# ------------------------------------------------------------------ write

def hard_rows(T, hkv, d, dtype, seed):
    """Random rows with the awkward ones among them: constant ones, far from zero, the type's
    smallest and largest values, exact ties, infinities and NaN."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, hkv, d, generator=g) * torch.exp(2 * torch.randn(T, hkv, 1, generator=g))).to(S.DT[dtype])
    flat = x.view(-1, d)
    fi = torch.finfo(S.DT[dtype])
    one = torch.randn(d, generator=g)
    special = [torch.zeros(d), torch.full((d,), -3.7), 100 + 0.1 * one, torch.full((d,), fi.max), one.sign() * fi.max,
               torch.full((d,), fi.smallest_normal * fi.eps * 3), torch.arange(d).float() % 31 / 2, -one.abs()]
    for bad in (float("inf"), float("-inf"), float("nan")):
        r = one.clone()
        r[d - 3] = bad
        special.append(r)
    special.append(torch.where(torch.arange(d) % 2 == 0, float("inf"), float("-inf")))
    for i, r in enumerate(special):
        if i * 2 < flat.shape[0]:
            flat[i * 2] = r.to(S.DT[dtype])
    return x


def check_write(T, hkv, d, bs, dtype, seed=0, strided=False):
    key, value = hard_rows(T, hkv, d, dtype, seed), hard_rows(T, hkv, d, dtype, seed + 1).flip(0)
    nb = T // bs + 3
    g = np.random.default_rng(seed)
    slots = g.permutation(nb * bs)[:T].astype(np.int64)
    slots[g.random(T) < 0.1] = -1
    c = S.empty_cache4(nb, bs, hkv, d, 3, 5.0)
    dev = {n: t.cuda() for n, t in c.items()}
    kk, vv = key.cuda(), value.cuda()
    if strided:   # slices of a wider projection output
        wide = torch.zeros(T, hkv * d * 2 + 24, dtype=S.DT[dtype], device="cuda")
        wide[:, 8:8 + hkv * d] = kk.view(T, -1)
        wide[:, 16 + hkv * d:16 + 2 * hkv * d] = vv.view(T, -1)
        kk = wide[:, 8:8 + hkv * d].view(T, hkv, d)
        vv = wide[:, 16 + hkv * d:16 + 2 * hkv * d].view(T, hkv, d)
    err = pa.new_err_flag()
    pa.int4_reshape_and_cache(kk, vv, dev["k"], dev["v"], dev["ks"], dev["vs"], torch.from_numpy(slots).cuda(),
                              err_flag=err)
    assert pa.read_err_flag(err) == 0
    keep = slots >= 0
    for n, x in (("k", key), ("v", value)):
        S.store4(c, n, torch.from_numpy(slots[keep]), x[keep])
        assert torch.equal(dev[n].cpu(), c[n]), f"{n} codes"
        assert same(dev[n + "s"].cpu(), c[n + "s"]), f"{n} scales"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,hkv,d,bs", [(1, 1, 64, 8), (1, 1, 128, 16), (37, 3, 64, 16), (64, 8, 128, 32), (5, 40, 128, 16),
                                        (3001, 20, 128, 48)])
def test_write(T, hkv, d, bs, dtype):
    check_write(T, hkv, d, bs, dtype)


@pytest.mark.parametrize("T,hkv,d", [(1, 2, 64), (19, 5, 128)])
def test_write_strided(T, hkv, d):
    check_write(T, hkv, d, 16, "f16", seed=2, strided=True)


def test_write_bad_slot_is_skipped_and_reported():
    hkv, d, bs, nb = 2, 64, 16, 4
    x = torch.randn(3, hkv, d, device="cuda").half()
    c = {n: t.cuda() for n, t in S.empty_cache4(nb, bs, hkv, d, 0, 0.0).items()}
    err = pa.new_err_flag()
    slots = torch.tensor([nb * bs, 5, nb * bs + 10 ** 12], device="cuda")
    pa.int4_reshape_and_cache(x, x, c["k"], c["v"], c["ks"], c["vs"], slots, err_flag=err)
    assert pa.read_err_flag(err) == pa.FLAG_BAD_SLOT
    want = S.empty_cache4(nb, bs, hkv, d, 0, 0.0)
    for n in "kv":
        S.store4(want, n, torch.tensor([5]), x[1:2].cpu())
    assert all(torch.equal(c[n].cpu(), want[n]) for n in c)


# --------------------------------------------------------------- read-back

@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("hkv,d,bs", [(1, 64, 8), (3, 128, 16), (8, 128, 48)])
def test_gather(hkv, d, bs, out):
    lens, starts = [0, 1, 50, 0, 17, 33, 0], [0, 4, 13, 2, 0, 100, 9]
    full = [s + n for s, n in zip(starts, lens)]
    bt, nb = Q.tables(full, bs, 3)
    c = S.cache4(full, bt, nb, bs, hkv, d, 5)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1]) + 3
    o = [torch.full((T, hkv, d), 9.0, dtype=S.DT[out], device="cuda") for _ in range(2)]
    err = pa.new_err_flag()
    pa.int4_gather(o[0], o[1], c["k"].cuda(), c["v"].cuda(), c["ks"].cuda(), c["vs"].cuda(), bt.cuda(),
                   torch.from_numpy(cu).cuda(), torch.tensor(starts, dtype=torch.int32).cuda(), err_flag=err)
    assert pa.read_err_flag(err) == 0
    for n, got in zip("kv", o):
        want = torch.full((T, hkv, d), 9.0, dtype=S.DT[out])
        for s, L in enumerate(lens):
            codes, w = S.take4(c, n, Q.slots_of(bt, s, starts[s], starts[s] + L, bs))
            u = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, 64))
            want[cu[s]:cu[s] + L] = ((u + w[..., 1:].float()) * w[..., :1].float()).flatten(-2).to(S.DT[out])
        assert torch.equal(got.cpu(), want), n    # two fp32 steps, one rounding: the same bits


def test_gather_reports_bad_ids_and_positions():
    hkv, d, bs = 2, 64, 16
    bt, nb = Q.tables([32, 32, 32], bs, 1)
    c = S.cache4([32, 32, 32], bt, nb, bs, hkv, d, 2)
    bad = bt.clone()
    bad[1, 1] = nb + 3
    cu = torch.tensor([0, 32, 64, 96], dtype=torch.int32)
    o = [torch.full((100, hkv, d), 9.0, device="cuda") for _ in range(2)]
    args = [c[n].cuda() for n in ("k", "v", "ks", "vs")]
    err = pa.new_err_flag()
    pa.int4_gather(*o, *args, bad.cuda(), cu.cuda(), err_flag=err)
    assert pa.read_err_flag(err) == pa.FLAG_BAD_BLOCK_ID
    got = o[0].cpu()
    assert torch.equal(got[48:64], torch.zeros(16, hkv, d)) and torch.all(got[96:] == 9)
    starts = torch.tensor([0, 0, 16], dtype=torch.int32)
    pa.int4_gather(*o, *args, bt.cuda(), cu.cuda(), starts.cuda(), err_flag=err)
    assert pa.read_err_flag(err) == pa.FLAG_BAD_CONTEXT_LEN
    assert torch.equal(o[1][80:96].cpu(), torch.zeros(16, hkv, d))


# ------------------------------------------------------------------ decode

LENS = [0, 1, 15, 16, 17, 255, 256, 257, 700, 33]


def run_decode(c, q, bt, lens, out="f32", scale=None, err=None, **kw):
    d = q.shape[2]
    o = torch.full(q.shape, float("nan"), dtype=S.DT[out], device="cuda")
    e = err if err is not None else pa.new_err_flag()
    pa.int4_decode(o, q.cuda(), c["k"].cuda(), c["v"].cuda(), c["ks"].cuda(), c["vs"].cuda(), bt.cuda(),
                   torch.tensor(lens, dtype=torch.int32).cuda(), scale if scale is not None else d ** -0.5, err_flag=e, **kw)
    if err is None:
        assert pa.read_err_flag(e) == 0
    return o


def compare(got, c, q, bt, lens, bs, scale, out):
    """Within what 32-bit steps can differ by.  Sums run over codes and zeros apart, so they are taken relative
    to sums of s (u + |z|), not of |s (u + z)|; otherwise the bound of the 8-bit cache."""
    hkv, d = c["k"].shape[2], 2 * c["k"].shape[3]
    hq = q.shape[1]
    o = got.cpu().double()
    for s, L in enumerate(lens):
        sl = Q.slots_of(bt, s, 0, L, bs)
        k, v = S.rows4(c, "k", sl), S.rows4(c, "v", sl)
        ref = Q.attend(q[s], k, v, scale)
        if L == 0:
            assert torch.equal(o[s], ref)
            continue
        kmag, vmag = S.size4(*S.take4(c, "k", sl)), S.size4(*S.take4(c, "v", sl))
        vmax = vmag.amax((0, 2)).repeat_interleave(hq // hkv)[:, None].numpy()
        xs = torch.einsum("hgd,lhd->hgl", q[s].double().abs().view(hkv, hq // hkv, d), kmag) * abs(scale)
        tol = Q.tolerance(ref.numpy(), vmax, L, d, xs.reshape(hq, -1).amax(-1)[:, None].numpy(), out)
        err = (o[s] - ref).abs().numpy()
        assert np.all(np.isfinite(o[s].numpy())), f"sequence {s}"
        assert np.all(err <= tol), f"sequence {s} (length {L}): {np.max(err / tol):.2f} of the bound"


def check_decode(lens, hq, hkv, d, bs, qdt, out="f32", seed=0, vary=1.0, qsize=1.0, offset=0.0, **kw):
    bt, nb = Q.tables(lens, bs, seed)
    c = S.cache4(lens, bt, nb, bs, hkv, d, seed, vary=vary, offset=offset)
    g = torch.Generator().manual_seed(seed + 9)
    q = (qsize * torch.randn(len(lens), hq, d, generator=g)).to(S.DT[qdt])
    scale = float(np.float32(d ** -0.5 / qsize))
    got = run_decode(c, q, bt, lens, out, scale, **kw)
    compare(got, c, q, bt, lens, bs, scale, out)
    return got


@pytest.mark.parametrize("hq,hkv,d,bs,qdt", [
    (4, 4, 64, 16, "f16"), (8, 8, 128, 16, "bf16"), (1, 1, 128, 8, "f16"), (8, 1, 64, 8, "bf16"), (2, 2, 64, 8, "f16"),
    (6, 3, 128, 32, "bf16"), (16, 4, 128, 16, "f16"), (32, 8, 64, 64, "bf16"), (64, 8, 128, 16, "f16"), (2, 2, 128, 16, "f16"),
    (10, 10, 128, 48, "bf16"), (12, 12, 64, 256, "f16"), (8, 2, 128, 128, "f16"), (16, 16, 128, 8, "bf16")])
def test_decode(hq, hkv, d, bs, qdt):
    check_decode(LENS, hq, hkv, d, bs, qdt)


@pytest.mark.parametrize("out", ["f16", "bf16"])
def test_decode_half_outputs(out):
    check_decode(LENS, 8, 8, 128, 16, out, out=out)


@pytest.mark.parametrize("P", [16, 48, 512])
@pytest.mark.parametrize("hkv", [1, 4, 8])
def test_decode_partitions(P, hkv):
    check_decode([0, 1, 48, 49, 511, 513, 2050], hkv * 2, hkv, 128, 16, "bf16", partition_size=P)


@pytest.mark.parametrize("hq,hkv,n,hi,P", [(8, 8, 60, 900, 128), (32, 8, 70, 1000, 256), (4, 1, 60, 3000, 512),
                                           (4, 4, 90, 1200, 0), (6, 3, 80, 2000, 512)])
def test_decode_enough_work_for_items_to_be_cut_between_sms(hq, hkv, n, hi, P):
    rng = np.random.default_rng(n)
    lens = rng.integers(1, hi, n).tolist()
    lens[3], lens[7], lens[n - 1] = 0, hi, 0
    check_decode(lens, hq, hkv, 64, 32, "bf16", seed=n, partition_size=P)


@pytest.mark.parametrize("hkv", [2, 8])
def test_decode_long_context(hkv):
    check_decode([9001, 4500], hkv * 4, hkv, 128, 32, "bf16", seed=3)


def test_decode_more_sequences_than_one_launch_takes():
    lens = np.random.default_rng(7).integers(0, 40, 2300).tolist()
    lens[-1] = 40
    check_decode(lens, 2, 1, 64, 16, "f16")


def test_decode_rows_of_very_different_sizes():
    check_decode([40, 300, 1000], 8, 8, 128, 16, "bf16", vary=3.0)


@pytest.mark.parametrize("offset", [-3.0, 40.0])
def test_decode_rows_far_from_zero(offset):
    check_decode([40, 300, 1000], 8, 4, 128, 16, "bf16", offset=offset, vary=0.3)


@pytest.mark.parametrize("qsize", [2.0 ** -40, 2.0 ** 40])
def test_decode_queries_beyond_binary16(qsize):
    check_decode([5, 100, 300], 8, 4, 64, 16, "bf16", qsize=qsize)


def test_decode_rising_keys_zero_rows_and_zero_queries():
    """Logits that rise with the position move the reference in every slot; rows of zeros have the floor's scale."""
    lens, hkv, d, bs = [700, 64, 50], 8, 128, 16
    bt, nb = Q.tables(lens, bs, 1)
    c = S.cache4(lens, bt, nb, bs, hkv, d, 1)
    q = torch.ones(3, hkv, d).half()
    q[2] = 0
    for s, L in enumerate(lens):
        sl = Q.slots_of(bt, s, 0, L, bs)
        x = torch.randn(L, hkv, d, generator=torch.Generator().manual_seed(s)) + torch.arange(L)[:, None, None] / 20
        S.store4(c, "k", sl, x.bfloat16())
        S.store4(c, "v", sl[::3], torch.zeros(len(sl[::3]), hkv, d).bfloat16())
    compare(run_decode(c, q, bt, lens), c, q, bt, lens, bs, float(np.float32(d ** -0.5)), "f32")
    S.store4(c, "v", torch.arange(nb * bs), torch.zeros(nb * bs, hkv, d).bfloat16())
    assert torch.all(run_decode(c, q, bt, lens) == 0)


def test_decode_many_tokens_of_little_weight_count():
    """One token of weight 1 and 20,000 of 2^-24.6 each: their share, 2^-10.3, must not be rounded away."""
    L, hkv, d, bs = 20001, 8, 64, 32
    bt, nb = Q.tables([L], bs, 1)
    c = S.cache4([1], bt, nb, bs, hkv, d, 1)
    q = torch.zeros(1, hkv, d).half()
    q[..., 0] = 1.0
    k = torch.zeros(L, hkv, d)
    k[0, :, 0], k[1:, :, 0] = 17.05 / 2, -17.05 / 2
    v = torch.ones(L, hkv, d)
    v[0] = 0.0
    sl = Q.slots_of(bt, 0, 0, L, bs)
    S.store4(c, "k", sl, k.half())
    S.store4(c, "v", sl, v.half())
    got = run_decode(c, q, bt, [L], scale=1.0)[0].cpu().double()
    ref = Q.attend(q[0], S.rows4(c, "k", sl), S.rows4(c, "v", sl), 1.0)
    # 32-bit sums of 20,001 terms: 20,001 half steps of 2^-24, 1.2e-3, relative to the sum at most
    assert 2e-4 < ref.min() and ((got - ref).abs() / ref).max() < 1.2e-3


def test_decode_poisoned_groups_reach_their_sequence_and_head_only():
    lens, hkv, d, bs = [100, 300, 100], 8, 128, 16
    bt, nb = Q.tables(lens, bs, 1)
    q = torch.randn(3, hkv, d, generator=torch.Generator().manual_seed(0)).half()
    at = Q.slots_of(bt, 1, 77, 78, bs)
    for n in ("ks", "vs"):
        c = S.cache4(lens, bt, nb, bs, hkv, d, 1)
        clean = run_decode(c, q, bt, lens)
        c[n][at // bs, 5, at % bs, 1, 0] = float("nan")
        got = run_decode(c, q, bt, lens)
        first = 0 if n == "ks" else 64          # a V group: its own elements
        assert torch.all(got[1, 5, first:].isnan())
        got[1, 5, first:] = clean[1, 5, first:]
        assert torch.equal(got, clean)


@pytest.mark.parametrize("hkv", [1, 8])
def test_decode_bad_block_ids_leave_their_tokens_out(hkv):
    lens, d, bs = [100, 300], 64, 8
    bt, nb = Q.tables(lens, bs, 1)
    c = S.cache4(lens, bt, nb, bs, hkv, d, 1)
    q = torch.randn(2, hkv, d, generator=torch.Generator().manual_seed(0)).half()
    bad = bt.clone()
    bad[1, 3], bad[1, 20] = -2, nb
    err = pa.new_err_flag()
    got = run_decode(c, q, bad, lens, err=err).cpu().double()
    assert pa.read_err_flag(err) == pa.FLAG_BAD_BLOCK_ID
    keep = torch.cat([Q.slots_of(bt, 1, a, b, bs) for a, b in ((0, 24), (32, 160), (168, 300))])
    ref = Q.attend(q[1], S.rows4(c, "k", keep), S.rows4(c, "v", keep), d ** -0.5)
    assert (got[1] - ref).abs().max() < 1e-3


def test_decode_bad_context_length_gives_a_zero_row():
    lens, hkv, d, bs = [100, 60, 40], 4, 128, 16
    bt, nb = Q.tables(lens, bs, 1)
    c = S.cache4(lens, bt, nb, bs, hkv, d, 1)
    q = torch.randn(3, hkv, d).half()
    clean = run_decode(c, q, bt, lens)
    for bad in (-1, 113):
        err = pa.new_err_flag()
        got = run_decode(c, q, bt, [100, bad, 40], err=err)
        assert pa.read_err_flag(err) == pa.FLAG_BAD_CONTEXT_LEN
        assert torch.all(got[1] == 0) and torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])


def test_decode_is_reproducible_and_block_ids_do_not_matter():
    lens = [0, 33, 1000, 257]
    a = check_decode(lens, 16, 8, 128, 16, "bf16", seed=5)
    bt, nb = Q.tables(lens, 16, 5)
    c = S.cache4(lens, bt, nb, 16, 8, 128, 5)
    perm = torch.randperm(nb)
    inv = torch.argsort(perm)
    bt2 = torch.where(bt >= 0, inv[bt.clamp(min=0).long()].int(), bt)
    q = torch.randn(4, 16, 128, generator=torch.Generator().manual_seed(14)).bfloat16()
    scale = float(np.float32(128 ** -0.5))
    assert torch.equal(a, run_decode({n: t[perm] for n, t in c.items()}, q, bt2, lens, scale=scale))


def test_tensors_on_16_byte_boundaries():
    """Tensors that start 16 bytes past a 32-byte boundary."""
    hkv, d, bs, L = 2, 64, 16, 21
    bt, nb = Q.tables([L], bs, 3)
    c = S.cache4([L], bt, nb, bs, hkv, d, 5)

    def off(t):
        n = 16 // t.element_size()
        wide = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")
        wide[n:] = t.flatten().cuda()
        return wide[n:].view(t.shape)
    t = {n: off(x) for n, x in c.items()}
    sl = Q.slots_of(bt, 0, 0, L, bs)
    key = torch.randn(L, hkv, d).half()
    pa.int4_reshape_and_cache(off(key), off(key), t["k"], t["v"], t["ks"], t["vs"], sl.cuda())
    o = [off(torch.zeros(L, hkv, d).half()) for _ in range(2)]
    pa.int4_gather(*o, t["k"], t["v"], t["ks"], t["vs"], bt.cuda(), torch.tensor([0, L], dtype=torch.int32).cuda())
    rows = S.values4(*S.quantise4(key))
    assert torch.equal(o[0].cpu(), rows.float().half()) and torch.equal(o[1].cpu(), o[0].cpu())
    q = torch.randn(1, 4, d).half()
    out = off(torch.zeros(1, 4, d).half())
    pa.int4_decode(out, off(q), t["k"], t["v"], t["ks"], t["vs"], bt.cuda(), torch.tensor([L], dtype=torch.int32).cuda(),
                   0.125)
    assert (out[0].cpu().double() - Q.attend(q[0], rows, rows, 0.125)).abs().max() < 4e-3


# ------------------------------------------------- a run of them together

def test_chunk_then_decode_copied_swapped_and_captured():
    """A prompt written and read back, its blocks copied and swapped out and in as bytes, then decode steps that append
    a row each, eagerly and replayed from one graph, on two threads' streams."""
    hq, hkv, d, bs, B, steps = 8, 4, 128, 16, 3, 4
    g = torch.Generator().manual_seed(3)
    prompt = [37, 16, 90]
    total = [n + steps for n in prompt]
    bt, nb = Q.tables(total, bs, 1, extra=12)
    rows = [[torch.randn(n, hkv, d, generator=g).bfloat16() for n in total] for _ in "kv"]
    want = S.empty_cache4(nb, bs, hkv, d, 0, 1.0)
    c = {n: t.cuda() for n, t in want.items()}
    pool = {n: torch.empty_like(t, device="cpu").pin_memory() for n, t in c.items()}

    def raw(t):
        return t.view(torch.uint8).reshape(nb, 1, 1, -1)
    sl = [Q.slots_of(bt, s, 0, n, bs) for s, n in enumerate(prompt)]
    k, v = (torch.cat([r[s][:n] for s, n in enumerate(prompt)]).cuda() for r in rows)
    pa.int4_reshape_and_cache(k, v, c["k"], c["v"], c["ks"], c["vs"], torch.cat(sl).cuda())
    # sequence 2's blocks go elsewhere, by way of a copy and of host memory
    free = sorted(set(range(nb)) - set(bt[bt >= 0].tolist()))
    mine = bt[2][bt[2] >= 0].tolist()
    pairs = torch.tensor(list(zip(mine, free[:len(mine)])), device="cuda")
    pa.copy_blocks(raw(c["k"]), raw(c["v"]), pairs)
    pa.copy_blocks(raw(c["ks"]), raw(c["vs"]), pairs)
    there = torch.tensor([[b, b] for b in free[:len(mine)]], device="cuda")
    for a, b in (("k", "v"), ("ks", "vs")):
        pa.swap_blocks(raw(c[a]), raw(c[b]), raw(pool[a]), raw(pool[b]), there)
        for n in (a, b):
            raw(c[n])[there[:, 0]] = 0x7f
        pa.swap_blocks(raw(pool[a]), raw(pool[b]), raw(c[a]), raw(c[b]), there)
    bt[2, :len(mine)] = torch.tensor(free[:len(mine)], dtype=torch.int32)
    tables = bt.cuda()
    o = [torch.empty(sum(prompt), hkv, d, device="cuda") for _ in range(2)]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(prompt)]), dtype=torch.int32).cuda()
    pa.int4_gather(*o, c["k"], c["v"], c["ks"], c["vs"], tables, cu)
    for got, x in zip(o, (k, v)):
        assert torch.equal(got.cpu(), S.values4(*S.quantise4(x.cpu())).float())

    queries = torch.randn(steps, B, hq, d, generator=g).bfloat16()
    failures = []

    def serve(captured):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                cc = {n: t.clone() for n, t in c.items()}
                q, kk, vv = (torch.zeros(B, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
                slots = torch.zeros(B, dtype=torch.int64, device="cuda")
                ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
                out = torch.empty(B, hq, d, device="cuda")

                def step():
                    pa.int4_reshape_and_cache(kk, vv, cc["k"], cc["v"], cc["ks"], cc["vs"], slots)
                    pa.int4_decode(out, q, cc["k"], cc["v"], cc["ks"], cc["vs"], tables, ctx, 0.1, partition_size=32)
                slots.fill_(-1)
                graph = pa.StepGraph(step) if captured else None
                for i in range(steps):
                    at = [n + i for n in prompt]
                    q.copy_(queries[i])
                    for t, r in ((kk, rows[0]), (vv, rows[1])):
                        t.copy_(torch.stack([r[s][p] for s, p in enumerate(at)]))
                    slots.copy_(torch.cat([Q.slots_of(bt, s, p, p + 1, bs) for s, p in enumerate(at)]))
                    ctx.copy_(torch.tensor([p + 1 for p in at]))
                    graph.replay() if captured else step()
                    got = out.cpu().double()
                    for s, p in enumerate(at):
                        kr, vr = (S.values4(*S.quantise4(r[s][:p + 1])) for r in rows)
                        ref = Q.attend(queries[i, s], kr, vr, 0.1)
                        # 32-bit steps over at most 94 tokens of |v| < 6: 2^-24 (94 x 4 + |x| (d + 4)) 6 < 1e-4
                        assert (got[s] - ref).abs().max() < 1e-4, (captured, i, s)
        except BaseException as e:     # noqa: BLE001 - handed to the main thread
            failures.append(e)
    serve(True)
    threads = [threading.Thread(target=serve, args=(False,)) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures[0]
