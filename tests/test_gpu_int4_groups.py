"""GPU tests of decode over the 4-bit cache where the two 64-element groups of a V row differ in
size: each group's elements against 64 bits, within what is right for that group alone."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_140_gb300 as pa

import quant_harness as Q
import step_harness as S

pytestmark = pytest.mark.gpu

D, BS = 128, 16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_140_gb300 import _build
    _build.build()


def case(lens, hq, hkv, v_of, seed=0, rising=0.0):
    """Tables, a cache with V rows v_of(random rows [L, hkv, 128]) and K rows whose logits rise, and queries."""
    bt, nb = Q.tables(lens, BS, seed)
    c = S.cache4(lens, bt, nb, BS, hkv, D, seed, vary=0.0)
    for s, L in enumerate(lens):
        if L == 0:
            continue
        sl = Q.slots_of(bt, s, 0, L, BS)
        g = torch.Generator().manual_seed(100 * seed + s)
        S.store4(c, "v", sl, v_of(torch.randn(L, hkv, D, generator=g)).bfloat16())
        if rising:
            S.store4(c, "k", sl, (torch.randn(L, hkv, D, generator=g) + torch.arange(L)[:, None, None] * rising).bfloat16())
    q = torch.randn(len(lens), hq, D, generator=torch.Generator().manual_seed(seed + 9)).bfloat16()
    return bt, c, q.abs() if rising else q


def decode(bt, c, q, lens, **kw):
    out = torch.full(q.shape, float("nan"), device="cuda")
    err = pa.new_err_flag()
    pa.int4_decode(out, q.cuda(), c["k"].cuda(), c["v"].cuda(), c["ks"].cuda(), c["vs"].cuda(), bt.cuda(),
                   torch.tensor(lens, dtype=torch.int32).cuda(), float(np.float32(D ** -0.5)), err_flag=err, **kw)
    assert pa.read_err_flag(err) == 0
    return out.cpu().double()


def compare(got, bt, c, q, lens, groups=(0, 1)):
    """Each group against the bound of 32-bit steps relative to the largest s (u + |z|) of that group alone.

    Q.tolerance, whose 2^-16 holds the weights' parts: a group's largest weight is kept above 2^6 and a weight
    loses less than 2^-24 where its low part ends, 2^-30 of the largest; over the 2,100 tokens here at most 2^-18.9."""
    scale = float(np.float32(D ** -0.5))
    hq, hkv = q.shape[1], c["k"].shape[2]
    for s, L in enumerate(lens):
        sl = Q.slots_of(bt, s, 0, L, BS)
        ref = Q.attend(q[s], S.rows4(c, "k", sl), S.rows4(c, "v", sl), scale)
        if L == 0:
            assert torch.equal(got[s], ref)
            continue
        kmag, vmag = S.size4(*S.take4(c, "k", sl)), S.size4(*S.take4(c, "v", sl))
        xs = torch.einsum("hgd,lhd->hgl", q[s].double().abs().view(hkv, hq // hkv, D), kmag) * scale
        xmax = xs.reshape(hq, -1).amax(-1)[:, None].numpy()
        for a in (64 * g for g in groups):
            vmax = vmag[..., a:a + 64].amax((0, 2)).repeat_interleave(hq // hkv)[:, None].numpy()
            tol = Q.tolerance(ref[:, a:a + 64].numpy(), vmax, L, D, xmax, "f32")
            err = (got[s, :, a:a + 64] - ref[:, a:a + 64]).abs().numpy()
            assert np.all(err <= tol), f"sequence {s} (length {L}), group {a // 64}: {np.max(err / tol):.2f} of the bound"


HEADS = [(8, 8), (16, 8), (32, 8), (64, 8), (2, 2), (2, 1), (4, 1), (8, 1)]


@pytest.mark.parametrize("small", [0, 1])
@pytest.mark.parametrize("bits", [8, 16, 24, 40, 100])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_a_group_much_smaller_than_its_neighbour(hq, hkv, bits, small):
    """Down to 2^-50 beside 2^50 (the last of `bits`), by either group."""
    def v_of(x):
        x = x * 2.0 ** (bits // 2 if bits == 100 else 0)
        x[..., 64 * small:64 * small + 64] *= 2.0 ** -bits
        return x
    lens = [1, 0, 17, 300, 700]
    bt, c, q = case(lens, hq, hkv, v_of, seed=bits + small)
    compare(decode(bt, c, q, lens), bt, c, q, lens)


@pytest.mark.parametrize("P", [0, 48])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_groups_of_changing_sizes(hq, hkv, P):
    """One token of very large values in one group, late and early; groups large in turn from token to token; logits
    that rise with the position, so that every group's weights pass their references again and again."""
    def one(x):
        if len(x) > 20:
            x[len(x) - 9, :, :64] *= 2.0 ** 30
            x[11, :, 64:] *= 2.0 ** 20
        return x

    def turns(x):
        x[0::2, :, :64] *= 2.0 ** -20
        x[1::2, :, 64:] *= 2.0 ** -20
        return x

    def grow(x):
        n = len(x)
        x[..., :64] *= torch.exp2(torch.linspace(0, 40, n))[:, None, None]
        x[..., 64:] *= torch.exp2(torch.linspace(10, -30, n))[:, None, None]
        return x
    lens = [5, 64, 333, 2100]
    for i, (v_of, rising) in enumerate(((one, 0.0), (turns, 0.0), (turns, 0.02), (grow, 0.0), (grow, 0.02))):
        bt, c, q = case(lens, hq, hkv, v_of, seed=i, rising=rising)
        compare(decode(bt, c, q, lens, partition_size=P), bt, c, q, lens)


@pytest.mark.parametrize("hq,hkv", HEADS)
def test_items_cut_between_sms(hq, hkv):
    """Enough work for shares that end inside an item: its parts are joined by a launch of their own."""
    def v_of(x):
        x[..., 64:] *= 2.0 ** -24
        return x
    lens = np.random.default_rng(hq).integers(1, 1500, 60 if hkv > 2 else 120).tolist()
    bt, c, q = case(lens, hq, hkv, v_of, seed=hq)
    compare(decode(bt, c, q, lens, partition_size=256), bt, c, q, lens)


@pytest.mark.parametrize("hq,hkv", HEADS)
def test_a_group_of_zeros_beside_one_of_values(hq, hkv):
    """Zeros answer nothing that could be seen beside the smallest value of the format, 2^-60: codes 0 and zeros 0
    enter turned, as -15 and 15 of that unit, in sums that are right to 2^-18.  (compare() knows no such
    terms: it takes a group of zeros to have sums of nothing.)"""
    lens = [1, 2, 333]

    def v_of(x):
        x[..., 64:] = 0
        return x
    bt, c, q = case(lens, hq, hkv, v_of)
    got = decode(bt, c, q, lens)
    assert torch.all(got[..., 64:].abs() <= 15 * 2.0 ** -78)
    compare(got, bt, c, q, lens, groups=(0,))


@pytest.mark.parametrize("group", [0, 1])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_a_group_that_is_no_number_leaves_its_neighbour_right(hq, hkv, group):
    """A V scale that is NaN: its head's elements of that group are NaN, all others as right as ever."""
    lens = [100, 300, 100]
    bt, c, q = case(lens, hq, hkv, lambda x: x, rising=0.05)
    at = Q.slots_of(bt, 1, 177, 178, BS)
    c["vs"][at // BS, 0, at % BS, group, 0] = float("nan")
    got = decode(bt, c, q, lens)
    a, r = 64 * group, hq // hkv
    assert torch.all(got[1, :r, a:a + 64].isnan())
    c["vs"][at // BS, 0, at % BS, group, 0] = 0.0          # something finite to compare the others by
    ref = Q.attend(q[1], *(S.rows4(c, n, Q.slots_of(bt, 1, 0, 300, BS)) for n in "kv"), float(np.float32(D ** -0.5)))
    got[1, :r, a:a + 64] = ref[:r, a:a + 64]
    compare(got, bt, c, q, lens)


@pytest.mark.parametrize("hq,hkv", [(8, 8), (32, 8), (2, 1)])
def test_tables_wider_than_any_context(hq, hkv):
    """A captured step's tables have room for the longest context there may be: the same bytes as of narrow ones."""
    lens = [1, 0, 17, 300, 700]
    bt, c, q = case(lens, hq, hkv, lambda x: x)
    wide = torch.full((len(lens), 4096), -7, dtype=torch.int32)
    wide[:, :bt.shape[1]] = bt
    kw = dict(max_context_len=700, partition_size=64)
    assert torch.equal(decode(bt, c, q, lens, **kw), decode(wide, c, q, lens, **kw))
