"""GPU tests of the quantised cache: write, read-back and decode against their
64-bit plain forms (codes and scales bit for bit), and runs of them together."""
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_140_gb300 as pa

import quant_harness as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_140_gb300 import _build
    _build.build()


# ------------------------------------------------------------------ write

def hard_rows(T, hkv, d, dtype, seed):
    """Random rows with the awkward ones among them: zeros, the type's smallest
    and largest values, rows of exact code ties, infinities and NaN."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, hkv, d, generator=g) * torch.exp(2 * torch.randn(T, hkv, 1, generator=g))
    x = x.to(Q.DT[dtype])
    flat = x.view(-1, d)
    fi = torch.finfo(Q.DT[dtype])
    special = [torch.zeros(d), torch.full((d,), fi.max), torch.full((d,), fi.smallest_normal * fi.eps * 3),
               torch.arange(d).float() - d / 2, 7.0 * (torch.arange(d) % 65).float() / 64]
    one = torch.randn(d, generator=g)
    for bad in (float("inf"), float("-inf"), float("nan")):
        r = one.clone()
        r[d - 3] = bad
        special.append(r)
    for i, r in enumerate(special):
        if i * 2 < flat.shape[0]:
            flat[i * 2] = r.to(Q.DT[dtype])
    return x


def check_write(T, hkv, d, bs, dtype, fmt, seed=0, strided=False):
    key, value = hard_rows(T, hkv, d, dtype, seed), hard_rows(T, hkv, d, dtype, seed + 1).flip(0)
    nb = T // bs + 3
    g = np.random.default_rng(seed)
    slots = g.permutation(nb * bs)[:T].astype(np.int64)
    slots[g.random(T) < 0.1] = -1
    c = {n: torch.full((nb, bs, hkv, d), 3, dtype=Q.CODE_DTYPE[fmt]) for n in "kv"}
    c.update({n + "s": torch.full((nb, bs, hkv), 5.0) for n in "kv"})
    dev = {n: t.cuda() for n, t in c.items()}
    if strided:   # slices of a wider projection output
        wide = torch.zeros(T, hkv * d * 2 + 24, dtype=Q.DT[dtype], device="cuda")
        wide[:, 8:8 + hkv * d] = key.view(T, -1).cuda()
        wide[:, 16 + hkv * d:16 + 2 * hkv * d] = value.view(T, -1).cuda()
        kk = wide[:, 8:8 + hkv * d].view(T, hkv, d)
        vv = wide[:, 16 + hkv * d:16 + 2 * hkv * d].view(T, hkv, d)
    else:
        kk, vv = key.cuda(), value.cuda()
    err = pa.new_err_flag()
    pa.quant_reshape_and_cache(kk, vv, dev["k"], dev["v"], dev["ks"], dev["vs"], torch.from_numpy(slots).cuda(),
                               err_flag=err)
    assert pa.read_err_flag(err) == 0
    keep = slots >= 0
    for n, x in (("k", key), ("v", value)):
        codes, scales = Q.quantise(x[keep], fmt)
        c[n].view(nb * bs, hkv, d)[slots[keep]] = codes
        c[n + "s"].view(nb * bs, hkv)[slots[keep]] = scales
        assert torch.equal(dev[n].cpu(), c[n]), f"{n} codes"
        got, want = dev[n + "s"].cpu(), c[n + "s"]
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num()), f"{n} scales"


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,hkv,d,bs", [(1, 1, 64, 8), (1, 1, 128, 16), (37, 3, 64, 16), (64, 8, 128, 32), (5, 40, 128, 16)])
def test_write(T, hkv, d, bs, dtype, fmt):
    check_write(T, hkv, d, bs, dtype, fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
def test_write_many_rows(d, fmt):
    check_write(3001, 20, d, 16, "bf16", fmt, seed=4)     # several rows per thread, a ragged last block


@pytest.mark.parametrize("T,hkv,d", [(1, 2, 64), (19, 5, 128)])
def test_write_strided(T, hkv, d):
    check_write(T, hkv, d, 16, "f16", "int8", seed=2, strided=True)


def test_write_bad_slot_is_skipped_and_reported():
    hkv, d, bs, nb = 2, 64, 16, 4
    x = torch.randn(3, hkv, d, device="cuda").half()
    codes = torch.zeros(nb, bs, hkv, d, dtype=torch.int8, device="cuda")
    c2 = codes.clone()
    s1, s2 = torch.zeros(nb, bs, hkv, device="cuda"), torch.zeros(nb, bs, hkv, device="cuda")
    err = pa.new_err_flag()
    slots = torch.tensor([nb * bs, 5, nb * bs + 10 ** 12], device="cuda")
    pa.quant_reshape_and_cache(x, x, codes, c2, s1, s2, slots, err_flag=err)
    assert pa.read_err_flag(err) == pa.FLAG_BAD_SLOT
    touched = (s1.view(-1, hkv) != 0).any(-1).nonzero().flatten().tolist()
    assert touched == [5] and torch.equal(codes, c2)


# --------------------------------------------------------------- read-back

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("hkv,d,bs", [(1, 64, 8), (3, 128, 16), (8, 128, 48)])
def test_gather(hkv, d, bs, out, fmt):
    lens, starts = [0, 1, 50, 0, 17, 33, 0], [0, 4, 13, 2, 0, 100, 9]
    full = [s + n for s, n in zip(starts, lens)]
    bt, nb = Q.tables(full, bs, 3)
    c = Q.quant_cache(full, bt, nb, bs, hkv, d, fmt, 5)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1]) + 3
    o = [torch.full((T, hkv, d), 9.0, dtype=Q.DT[out], device="cuda") for _ in range(2)]
    err = pa.new_err_flag()
    pa.quant_gather(o[0], o[1], c["k"].cuda(), c["v"].cuda(), c["ks"].cuda(), c["vs"].cuda(), bt.cuda(),
                    torch.from_numpy(cu).cuda(), torch.tensor(starts, dtype=torch.int32).cuda(), err_flag=err)
    assert pa.read_err_flag(err) == 0
    for n, got in zip("kv", o):
        want = torch.full((T, hkv, d), 9.0, dtype=Q.DT[out])
        for s, L in enumerate(lens):
            sl = Q.slots_of(bt, s, starts[s], starts[s] + L, bs)
            codes, sc = c[n].view(-1, hkv, d)[sl], c[n + "s"].view(-1, hkv)[sl]
            want[cu[s]:cu[s] + L] = (Q.values(codes, fmt).float() * sc[..., None]).to(Q.DT[out])
        assert torch.equal(got.cpu(), want), n    # one fp32 product, one rounding: the same bits


def test_gather_into_rows_on_16_byte_boundaries():
    """Outputs that start 16 bytes past a 32-byte boundary, and caches and rows of write that do."""
    hkv, d, bs, L = 2, 64, 16, 21
    bt, nb = Q.tables([L], bs, 3)
    c = Q.quant_cache([L], bt, nb, bs, hkv, d, "int8", 5)

    def off(t):
        n = 16 // t.element_size()
        wide = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")
        wide[n:] = t.flatten().cuda()
        return wide[n:].view(t.shape)
    o = [off(torch.zeros(L, hkv, d).half()) for _ in range(2)]
    pa.quant_gather(*o, off(c["k"]), off(c["v"]), off(c["ks"]), off(c["vs"]), bt.cuda(),
                    torch.tensor([0, L], dtype=torch.int32).cuda())
    sl = Q.slots_of(bt, 0, 0, L, bs)
    for n, got in zip("kv", o):
        assert torch.equal(got.cpu(), Q.quant_rows(c, n, sl, "int8").float().half())
    key = torch.randn(L, hkv, d).half()
    t = {n: off(x) for n, x in c.items()}
    pa.quant_reshape_and_cache(off(key), off(key), t["k"], t["v"], t["ks"], t["vs"], sl.cuda())
    codes, scales = Q.quantise(key, "int8")
    assert torch.equal(t["v"].view(-1, hkv, d)[sl.cuda()].cpu(), codes)
    assert torch.equal(t["vs"].view(-1, hkv)[sl.cuda()].cpu(), scales)
    q = torch.randn(1, 4, d).half()
    out = off(torch.zeros(1, 4, d).half())
    pa.quant_decode(out, off(q), t["k"], t["v"], t["ks"], t["vs"], bt.cuda(), torch.tensor([L], dtype=torch.int32).cuda(),
                    0.125)
    ref = Q.attend(q[0], *[Q.values(codes, "int8") * scales.double()[..., None]] * 2, 0.125)
    assert (out[0].cpu().double() - ref).abs().max() < 4e-3


def test_gather_without_starts_and_many_sequences():
    hkv, d, bs = 1, 64, 16
    g = np.random.default_rng(0)
    lens = g.integers(0, 4, 1500).tolist()        # more sequences than a block keeps in shared memory
    bt, nb = Q.tables(lens, bs, 1)
    c = Q.quant_cache(lens, bt, nb, bs, hkv, d, "int8", 2)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    o = [torch.zeros(int(cu[-1]), hkv, d, device="cuda") for _ in range(2)]
    err = pa.new_err_flag()
    pa.quant_gather(*o, c["k"].cuda(), c["v"].cuda(), c["ks"].cuda(), c["vs"].cuda(), bt.cuda(), cu.cuda(), err_flag=err)
    assert pa.read_err_flag(err) == 0
    sl = torch.cat([Q.slots_of(bt, s, 0, L, bs) for s, L in enumerate(lens)])
    for n, got in zip("kv", o):
        assert torch.equal(got.cpu(), Q.quant_rows(c, n, sl, "int8").float())


def test_gather_reports_bad_ids_and_positions():
    hkv, d, bs = 2, 64, 16
    bt, nb = Q.tables([32, 32, 32], bs, 1)
    c = Q.quant_cache([32, 32, 32], bt, nb, bs, hkv, d, "e4m3", 2)
    bad = bt.clone()
    bad[1, 1] = nb + 3
    cu = torch.tensor([0, 32, 64, 96], dtype=torch.int32)
    o = [torch.full((100, hkv, d), 9.0, device="cuda") for _ in range(2)]
    args = [c[n].cuda() for n in ("k", "v", "ks", "vs")]
    err = pa.new_err_flag()
    pa.quant_gather(*o, *args, bad.cuda(), cu.cuda(), err_flag=err)
    assert pa.read_err_flag(err) == pa.FLAG_BAD_BLOCK_ID
    got = o[0].cpu()
    assert torch.equal(got[48:64], torch.zeros(16, hkv, d)) and torch.all(got[96:] == 9)
    assert torch.equal(got[64:96], Q.quant_rows(c, "k", Q.slots_of(bt, 2, 0, 32, bs), "e4m3").float())
    # positions outside the table: zeros; the last sequence starts 16 too late
    starts = torch.tensor([0, 0, 16], dtype=torch.int32)
    pa.quant_gather(*o, *args, bt.cuda(), cu.cuda(), starts.cuda(), err_flag=err)
    assert pa.read_err_flag(err) == pa.FLAG_BAD_CONTEXT_LEN
    assert torch.equal(o[1][80:96].cpu(), torch.zeros(16, hkv, d))
    # bounds that reach past the output: reported, nothing outside is written
    pa.quant_gather(*o, *args, bt.cuda(), torch.tensor([0, 32, 64, 200], dtype=torch.int32).cuda(), err_flag=err)
    assert pa.read_err_flag(err) & pa.FLAG_BAD_CONTEXT_LEN


# ------------------------------------------------------------------ decode

LENS = [0, 1, 15, 16, 17, 255, 256, 257, 700, 33]


def run_decode(c, q, bt, lens, out="f32", scale=None, err=None, **kw):
    d = q.shape[2]
    o = torch.full(q.shape, float("nan"), dtype=Q.DT[out], device="cuda")
    e = err if err is not None else pa.new_err_flag()
    pa.quant_decode(o, q.cuda(), c["k"].cuda(), c["v"].cuda(), c["ks"].cuda(), c["vs"].cuda(), bt.cuda(),
                    torch.tensor(lens, dtype=torch.int32).cuda(), scale if scale is not None else d ** -0.5, err_flag=e,
                    **kw)
    if err is None:
        assert pa.read_err_flag(e) == 0
    return o


def check_decode(lens, hq, hkv, d, bs, fmt, qdt, out="f32", seed=0, vary=1.0, qsize=1.0, **kw):
    bt, nb = Q.tables(lens, bs, seed)
    c = Q.quant_cache(lens, bt, nb, bs, hkv, d, fmt, seed, vary=vary)
    g = torch.Generator().manual_seed(seed + 9)
    q = (qsize * torch.randn(len(lens), hq, d, generator=g)).to(Q.DT[qdt])
    scale = float(np.float32(d ** -0.5 / qsize))
    got = run_decode(c, q, bt, lens, out, scale, **kw)
    compare(got, c, q, bt, lens, bs, fmt, scale, out)
    return got


def compare(got, c, q, bt, lens, bs, fmt, scale, out):
    hkv, d = c["k"].shape[2:]
    hq = q.shape[1]
    o = got.cpu().double()
    for s, L in enumerate(lens):
        sl = Q.slots_of(bt, s, 0, L, bs)
        k, v = Q.quant_rows(c, "k", sl, fmt), Q.quant_rows(c, "v", sl, fmt)
        ref = Q.attend(q[s], k, v, scale)
        if L == 0:
            assert torch.equal(o[s], ref)
            continue
        vmax = v.abs().amax((0, 2)).repeat_interleave(hq // hkv)[:, None].numpy()
        xs = torch.einsum("hgd,lhd->hgl", q[s].double().abs().view(hkv, hq // hkv, d), k.abs()) * abs(scale)
        tol = Q.tolerance(ref.numpy(), vmax, L, d, xs.reshape(hq, -1).amax(-1)[:, None].numpy(), out)
        err = (o[s] - ref).abs().numpy()
        assert np.all(np.isfinite(o[s].numpy())), f"sequence {s}"
        assert np.all(err <= tol), f"sequence {s} (length {L}): {np.max(err / tol):.2f} of the bound"


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("hq,hkv,d,bs,qdt", [
    (4, 4, 64, 16, "f16"), (8, 8, 128, 16, "bf16"), (1, 1, 128, 8, "f16"), (8, 1, 64, 8, "bf16"),
    (6, 3, 128, 32, "bf16"), (16, 4, 128, 16, "f16"), (32, 8, 64, 64, "bf16"), (64, 8, 128, 16, "f16"),
    (10, 10, 128, 48, "bf16"), (12, 12, 64, 256, "f16"), (8, 2, 128, 128, "f16")])
def test_decode(hq, hkv, d, bs, qdt, fmt):
    check_decode(LENS, hq, hkv, d, bs, fmt, qdt)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("out", ["f16", "bf16"])
def test_decode_half_outputs(out, fmt):
    check_decode(LENS, 8, 8, 128, 16, fmt, out, out=out)


@pytest.mark.parametrize("P", [16, 48, 128, 512])
@pytest.mark.parametrize("hkv", [1, 4, 8])
def test_decode_partitions(P, hkv):
    check_decode([0, 1, 48, 49, 511, 513, 2050], hkv * 2, hkv, 128, 16, "e4m3", "bf16", partition_size=P)


@pytest.mark.parametrize("hq,hkv,n,hi,P", [(8, 8, 60, 900, 128), (16, 16, 50, 700, 0), (32, 8, 70, 1000, 256),
                                           (4, 1, 60, 3000, 512), (4, 4, 90, 1200, 0), (6, 3, 80, 2000, 512)])
def test_decode_enough_work_for_items_to_be_cut_between_sms(hq, hkv, n, hi, P):
    rng = np.random.default_rng(n)
    lens = rng.integers(1, hi, n).tolist()
    lens[3], lens[7], lens[n - 1] = 0, hi, 0
    check_decode(lens, hq, hkv, 64, 32, "e4m3" if hkv % 3 else "int8", "bf16", seed=n, partition_size=P)


def test_decode_launches_of_many_sequences_cut_items_apart():
    """Two launches of a long batch, both with items cut between SMs."""
    rng = np.random.default_rng(3)
    lens = rng.integers(1, 120, 4000).tolist()
    check_decode(lens, 8, 8, 64, 16, "int8", "f16", seed=3, partition_size=64)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("hkv", [2, 8])
def test_decode_long_context(hkv, fmt):
    check_decode([9001, 4500], hkv * 4, hkv, 128, 32, fmt, "bf16", seed=3)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_decode_rows_of_very_different_sizes(fmt):
    """Row sizes spread over e^+-6: V scales of many powers of two in one sum."""
    check_decode([40, 300, 1000], 8, 8, 128, 16, fmt, "bf16", vary=3.0)


@pytest.mark.parametrize("qsize", [2.0 ** -40, 2.0 ** 40])
def test_decode_queries_beyond_binary16(qsize):
    check_decode([5, 100, 300], 8, 4, 64, 16, "int8", "bf16", qsize=qsize)


def test_decode_rising_keys_and_zero_rows():
    """Logits that rise with the position move the reference in every slot; zero V rows have the floor's scale."""
    lens, hkv, d, bs = [700, 64], 8, 128, 16
    bt, nb = Q.tables(lens, bs, 1)
    c = Q.quant_cache(lens, bt, nb, bs, hkv, d, "e4m3", 1)
    q = torch.ones(2, hkv, d).half()
    for s, L in enumerate(lens):
        sl = Q.slots_of(bt, s, 0, L, bs)
        x = torch.randn(L, hkv, d, generator=torch.Generator().manual_seed(s)) + torch.arange(L)[:, None, None] / 20
        codes, sc = Q.quantise(x.bfloat16(), "e4m3")
        c["k"].view(-1, hkv, d)[sl] = codes
        c["ks"].view(-1, hkv)[sl] = sc
        z = sl[::3]
        zc, zs = Q.quantise(torch.zeros(len(z), hkv, d).bfloat16(), "e4m3")
        c["v"].view(-1, hkv, d)[z] = zc
        c["vs"].view(-1, hkv)[z] = zs
    got = run_decode(c, q, bt, lens)
    compare(got, c, q, bt, lens, bs, "e4m3", float(np.float32(d ** -0.5)), "f32")
    # V rows that are all zero: a zero output
    zc, zs = Q.quantise(torch.zeros(nb * bs, hkv, d).bfloat16(), "e4m3")
    c["v"], c["vs"] = zc.view(nb, bs, hkv, d), zs.view(nb, bs, hkv)
    assert torch.all(run_decode(c, q, bt, lens) == 0)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_decode_many_tokens_of_little_weight_count(fmt):
    """One token of weight 1 and 20,000 of 2^-24.6 each: their share, 2^-10.3, must not be rounded away."""
    L, hkv, d, bs = 20001, 8, 64, 32
    bt, nb = Q.tables([L], bs, 1)
    c = Q.quant_cache([1], bt, nb, bs, hkv, d, fmt, 1)
    q = torch.zeros(1, hkv, d).half()
    q[..., 0] = 1.0
    scale = 1.0
    k = torch.zeros(L, hkv, d)
    k[0, :, 0] = 17.05 / 2          # the others: -17.05 / 2, so e^-17.05 = 2^-24.6 of the first's weight
    k[1:, :, 0] = -17.05 / 2
    v = torch.ones(L, hkv, d)
    v[0] = 0.0
    for n, x in (("k", k), ("v", v)):
        codes, sc = Q.quantise(x.half(), fmt)
        sl = Q.slots_of(bt, 0, 0, L, bs)
        c[n].view(-1, hkv, d)[sl] = codes
        c[n + "s"].view(-1, hkv)[sl] = sc
    got = run_decode(c, q, bt, [L], scale=scale)[0].cpu().double()
    sl = Q.slots_of(bt, 0, 0, L, bs)
    ref = Q.attend(q[0], Q.quant_rows(c, "k", sl, fmt), Q.quant_rows(c, "v", sl, fmt), scale)
    assert 5e-4 < ref.min() and ((got - ref).abs() / ref).max() < 1e-3


def test_decode_poisoned_row_reaches_its_sequence_and_head_only():
    lens, hkv, d, bs = [100, 300, 100], 8, 64, 16
    bt, nb = Q.tables(lens, bs, 1)
    for n in ("ks", "vs"):
        c = Q.quant_cache(lens, bt, nb, bs, hkv, d, "int8", 1)
        q = torch.randn(3, hkv, d, generator=torch.Generator().manual_seed(0)).half()
        clean = run_decode(c, q, bt, lens)
        c[n].view(-1, hkv)[Q.slots_of(bt, 1, 77, 78, bs), 5] = float("nan")
        got = run_decode(c, q, bt, lens)
        assert torch.all(got[1, 5].isnan())
        got[1, 5] = clean[1, 5]
        assert torch.equal(got, clean)


@pytest.mark.parametrize("hkv", [1, 8])
def test_decode_bad_block_ids_leave_their_tokens_out(hkv):
    lens, d, bs = [100, 300], 64, 8
    bt, nb = Q.tables(lens, bs, 1)
    c = Q.quant_cache(lens, bt, nb, bs, hkv, d, "e4m3", 1)
    q = torch.randn(2, hkv, d, generator=torch.Generator().manual_seed(0)).half()
    bad = bt.clone()
    bad[1, 3], bad[1, 20] = -2, nb
    err = pa.new_err_flag()
    got = run_decode(c, q, bad, lens, err=err).cpu().double()
    assert pa.read_err_flag(err) == pa.FLAG_BAD_BLOCK_ID
    keep = torch.cat([Q.slots_of(bt, 1, a, b, bs) for a, b in ((0, 24), (32, 160), (168, 300))])
    ref = Q.attend(q[1], Q.quant_rows(c, "k", keep, "e4m3"), Q.quant_rows(c, "v", keep, "e4m3"), d ** -0.5)
    assert (got[1] - ref).abs().max() < 1e-3


def test_decode_bad_context_length_gives_a_zero_row():
    lens, hkv, d, bs = [100, 60, 40], 4, 128, 16
    bt, nb = Q.tables(lens, bs, 1)
    c = Q.quant_cache(lens, bt, nb, bs, hkv, d, "int8", 1)
    q = torch.randn(3, hkv, d).half()
    clean = run_decode(c, q, bt, lens)
    for bad in (-1, 113):
        err = pa.new_err_flag()
        got = run_decode(c, q, bt, [100, bad, 40], err=err)
        assert pa.read_err_flag(err) == pa.FLAG_BAD_CONTEXT_LEN
        assert torch.all(got[1] == 0) and torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])


def test_decode_more_sequences_than_one_launch_takes():
    g = np.random.default_rng(7)
    lens = g.integers(0, 40, 2300).tolist()
    lens[-1] = 40
    check_decode(lens, 2, 1, 64, 16, "int8", "f16")


def test_decode_is_reproducible_and_block_ids_do_not_matter():
    lens = [0, 33, 1000, 257]
    a = check_decode(lens, 16, 8, 128, 16, "e4m3", "bf16", seed=5)
    b = check_decode(lens, 16, 8, 128, 16, "e4m3", "bf16", seed=5)
    assert torch.equal(a, b)
    bt, nb = Q.tables(lens, 16, 5)
    c = Q.quant_cache(lens, bt, nb, 16, 8, 128, "e4m3", 5)
    perm = torch.randperm(nb)
    inv = torch.argsort(perm)
    moved = {n: t[perm] for n, t in c.items()}
    bt2 = torch.where(bt >= 0, inv[bt.clamp(min=0).long()].int(), bt)
    q = torch.randn(4, 16, 128, generator=torch.Generator().manual_seed(14)).bfloat16()
    assert torch.equal(run_decode(c, q, bt, lens), run_decode(moved, q, bt2, lens))


# ----------------------------------------------------- runs of them together

def test_write_share_read_prefill_and_decode_together():
    """A prompt is written quantised, its blocks are copied for a second sequence
    (codes and scales), read back to 16 bits for a prefill of the tail, and both
    sequences decode over their caches."""
    hkv, hq, d, bs, n0, new = 2, 4, 128, 16, 40, 9
    g = torch.Generator().manual_seed(1)
    L = n0 + new
    nb = 16
    kc = torch.zeros(nb, bs, hkv, d, dtype=torch.int8, device="cuda")
    vc, ks = kc.clone(), torch.zeros(nb, bs, hkv, device="cuda")
    vs = ks.clone()
    rows = [torch.randn(L, hkv, d, generator=g).bfloat16() for _ in range(2)]
    bt = torch.tensor([[3, 9, 1, 5], [3, 9, 7, 2]], dtype=torch.int32)
    sl = Q.slots_of(bt, 0, 0, L, bs).cuda()
    pa.quant_reshape_and_cache(rows[0].cuda(), rows[1].cuda(), kc, vc, ks, vs, sl)
    pairs = torch.tensor([[1, 7], [5, 2]], device="cuda")       # sequence 1 gets blocks of its own from the third on
    pa.copy_blocks(kc.view(torch.uint8), vc.view(torch.uint8), pairs)
    pa.copy_blocks(ks.view(torch.uint8).view(nb, bs, hkv, 4), vs.view(torch.uint8).view(nb, bs, hkv, 4), pairs)
    cu = torch.tensor([0, L, 2 * L], dtype=torch.int32, device="cuda")
    dense = [torch.empty(2 * L, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pa.quant_gather(*dense, kc, vc, ks, vs, bt.cuda(), cu)
    for x, y in zip(rows, dense):
        assert torch.equal(y[:L], y[L:])
        # within half a code step of the row's largest value, and a bf16 rounding
        step = x.double().abs().amax(-1, keepdim=True) / 127
        assert torch.all((y[:L].cpu().double() - x.double()).abs() <= 0.5001 * step + x.double().abs() * 2.0 ** -8)
    # prefill of the tail over the dense rows as a 16-bit paged cache
    pk, pv = (torch.zeros(8, bs, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pk.view(-1, hkv, d)[:L], pv.view(-1, hkv, d)[:L] = dense[0][:L], dense[1][:L]
    qn = torch.randn(new, hq, d, generator=g).bfloat16().cuda()
    o = torch.empty(new, hq, d, device="cuda")
    pa.prefill(o, qn, pk, pv, torch.arange(4, dtype=torch.int32, device="cuda")[None].contiguous(),
               torch.tensor([L], dtype=torch.int32, device="cuda"),
               torch.tensor([0, new], dtype=torch.int32, device="cuda"), d ** -0.5, max_q_len=new)
    # decode of the last token over both sequences' quantised caches equals the prefill's last row up to the
    # bf16 rounding of the dense rows
    q2 = qn[-1:].expand(2, hq, d).contiguous()
    od = torch.empty(2, hq, d, device="cuda")
    pa.quant_decode(od, q2, kc, vc, ks, vs, bt.cuda(), torch.tensor([L, L], dtype=torch.int32, device="cuda"), d ** -0.5)
    assert torch.equal(od[0], od[1])
    assert (od[0] - o[-1]).abs().max() < 0.05


def test_captured_steps_replay_on_new_inputs_and_keep_their_own_workspaces():
    """Two captured decode steps with split contexts, replayed on two streams at
    once, after larger eager calls; each equals its eager result."""
    hkv, d, bs = 8, 128, 16
    cases = []
    for seed, lens in ((1, [900, 700]), (2, [1200, 300, 1500])):
        bt, nb = Q.tables(lens, bs, seed)
        c = {n: t.cuda() for n, t in Q.quant_cache(lens, bt, nb, bs, hkv, d, "e4m3", seed).items()}
        st = dict(c=c, bt=bt.cuda(), ctx=torch.tensor(lens, dtype=torch.int32).cuda(),
                  q=torch.randn(len(lens), hkv, d, device="cuda").bfloat16(),
                  new=torch.randn(2, len(lens), hkv, d, device="cuda").bfloat16(),
                  slots=torch.stack([Q.slots_of(bt, s, L - 1, L, bs)[0] for s, L in enumerate(lens)]).cuda())
        st["out"] = torch.empty(len(lens), hkv, d, device="cuda")

        def step(st=st):
            c = st["c"]
            pa.quant_reshape_and_cache(st["new"][0], st["new"][1], c["k"], c["v"], c["ks"], c["vs"], st["slots"])
            pa.quant_decode(st["out"], st["q"], c["k"], c["v"], c["ks"], c["vs"], st["bt"], st["ctx"], d ** -0.5)
        st["step"], st["graph"] = step, pa.StepGraph(step)
        cases.append(st)
    big_lens = [6000] * 8
    check_decode(big_lens, 8, 8, 64, 16, "int8", "f16")
    streams = [torch.cuda.Stream() for _ in cases]
    for rep in range(3):
        want = []
        for st in cases:
            st["q"].normal_()
            st["new"].normal_()
            st["step"]()
            want.append(st["out"].clone())
            st["out"].zero_()
        torch.cuda.synchronize()
        for st, s in zip(cases, streams):
            with torch.cuda.stream(s):
                st["graph"].replay()
        torch.cuda.synchronize()
        for st, w in zip(cases, want):
            assert torch.equal(st["out"], w)


def test_calls_on_two_streams_at_once():
    lens, hkv, d, bs = [3000, 2500], 8, 128, 16
    bt, nb = Q.tables(lens, bs, 1)
    c = {n: t.cuda() for n, t in Q.quant_cache(lens, bt, nb, bs, hkv, d, "int8", 1).items()}
    ctx = torch.tensor(lens, dtype=torch.int32).cuda()
    qs = [torch.randn(2, hkv, d, device="cuda").half() for _ in range(2)]
    outs = [torch.empty(2, hkv, d, device="cuda") for _ in range(2)]
    want = []
    bt = bt.cuda()
    for q in qs:
        o = torch.empty(2, hkv, d, device="cuda")
        pa.quant_decode(o, q, c["k"], c["v"], c["ks"], c["vs"], bt, ctx, 0.1)
        want.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for q, o, s in zip(qs, outs, streams):
            with torch.cuda.stream(s):
                pa.quant_decode(o, q, c["k"], c["v"], c["ks"], c["vs"], bt, ctx, 0.1)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_threads_on_one_stream():
    """Calls of several launches, made by threads on the same stream with the default workspaces."""
    hkv, d, bs = 8, 128, 16
    work = []
    for i, lens in enumerate(([5000, 2500, 17], [700] * 40, [9000])):
        bt, nb = Q.tables(lens, bs, i)
        c = {n: t.cuda() for n, t in Q.quant_cache(lens, bt, nb, bs, hkv, d, "e4m3", i).items()}
        q = torch.randn(len(lens), hkv, d, device="cuda").half()
        work.append((q, c, bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), max(lens)))

    def call(w):
        q, c, bt, ctx, most = w
        o = torch.empty(q.shape, device="cuda")
        pa.quant_decode(o, q, c["k"], c["v"], c["ks"], c["vs"], bt, ctx, 0.1, max_context_len=most)
        return o
    want = [call(w) for w in work]
    torch.cuda.synchronize()
    wrong = torch.zeros(len(work), dtype=torch.int32, device="cuda")

    def loop(i):
        for _ in range(200):
            wrong[i] += (call(work[i]) != want[i]).any()
    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert wrong.tolist() == [0] * len(work)


def test_cache_slots_past_two_to_the_thirty_one_bytes():
    """Rows whose byte offset passes 2^32 in a cache of 5 GB of codes."""
    hkv, d, bs = 8, 128, 16
    nb = 330_000
    codes = [torch.zeros(nb, bs, hkv, d, dtype=torch.int8, device="cuda") for _ in range(2)]
    sc = [torch.zeros(nb, bs, hkv, device="cuda") for _ in range(2)]
    L = 40
    bt = torch.tensor([[nb - 1, 7, nb - 3]], dtype=torch.int32)
    sl = Q.slots_of(bt, 0, 0, L, bs)
    g = torch.Generator().manual_seed(0)
    k, v = (torch.randn(L, hkv, d, generator=g).half() for _ in range(2))
    pa.quant_reshape_and_cache(k.cuda(), v.cuda(), *codes, *sc, sl.cuda())
    o = [torch.empty(L, hkv, d, device="cuda") for _ in range(2)]
    pa.quant_gather(*o, *codes, *sc, bt.cuda(), torch.tensor([0, L], dtype=torch.int32).cuda())
    ref = {}
    for n, x, got in (("k", k, o[0]), ("v", v, o[1])):
        cc, s = Q.quantise(x, "int8")
        ref[n] = Q.values(cc, "int8") * s.double()[..., None]
        assert torch.equal(got.cpu(), ref[n].float())
    q = torch.randn(1, hkv, d, generator=g).half()
    out = torch.empty(1, hkv, d, device="cuda")
    pa.quant_decode(out, q.cuda(), *codes, *sc, bt.cuda(), torch.tensor([L], dtype=torch.int32).cuda(), d ** -0.5)
    assert (out[0].cpu().double() - Q.attend(q[0], ref["k"], ref["v"], d ** -0.5)).abs().max() < 1e-4


def test_refusals():
    kc = torch.zeros(4, 16, 2, 64, dtype=torch.int8, device="cuda")
    sc = torch.zeros(4, 16, 2, device="cuda")
    x = torch.zeros(3, 2, 64, dtype=torch.float16, device="cuda")
    sl = torch.zeros(3, dtype=torch.int64, device="cuda")
    ok = dict(key=x, value=x, k_cache=kc, v_cache=kc.clone(), k_scales=sc, v_scales=sc.clone(), slot_mapping=sl)
    for name, bad in [("k_scales", sc.half()), ("k_scales", sc[:, :, :1].contiguous()), ("slot_mapping", sl.int()),
                      ("key", x.transpose(0, 1)), ("key", x.cpu()), ("v_cache", kc.view(torch.uint8)),
                      ("k_scales", sc.cpu()), ("slot_mapping", sl[:2])]:
        with pytest.raises((ValueError, TypeError)):
            pa.quant_reshape_and_cache(**{**ok, name: bad})
    wide = torch.zeros(3, 2 * 64 + 4, dtype=torch.float16, device="cuda")[:, :128].view(3, 2, 64)
    with pytest.raises(pa.PagedAttentionError):          # a token stride that is no multiple of 8
        pa.quant_reshape_and_cache(**{**ok, "key": wide})
    q = torch.zeros(1, 2, 64, dtype=torch.float16, device="cuda")
    dec = dict(out=q.clone(), query=q, k_cache=kc, v_cache=kc.clone(), k_scales=sc, v_scales=sc.clone(),
               block_tables=torch.zeros(1, 4, dtype=torch.int32, device="cuda"),
               context_lens=torch.ones(1, dtype=torch.int32, device="cuda"), scale=0.1)
    for name, bad in [("query", q.float()), ("k_cache", kc.half()), ("block_tables", dec["block_tables"].long()),
                      ("out", q[:, :1].contiguous()), ("partition_size", 24), ("max_context_len", -1)]:
        with pytest.raises((ValueError, TypeError)):
            pa.quant_decode(**{**dec, name: bad})
    with pytest.raises(pa.PagedAttentionError):          # a bound beyond the table
        pa.quant_decode(**dec, max_context_len=65)
    with pytest.raises(pa.PagedAttentionError):          # a workspace that is too small
        pa.quant_decode(**{**dec, "block_tables": torch.zeros(1, 100, dtype=torch.int32, device="cuda")},
                        workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
