"""GPU tests of partitions that start inside a block and hold up to 32 of them:
automatic lengths near the limit at block sizes above 32, and the longest legal
requests.  The caches are small pools that every sequence's table goes through
in a random order of its own, so neighbouring blocks always differ."""
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


def pool_tables(n, width, nb, seed):
    g = np.random.default_rng(seed)
    return torch.from_numpy(np.stack([np.concatenate([g.permutation(nb) for _ in range(-(-width // nb))])[:width]
                                      for _ in range(n)]).astype(np.int32))


def compare(got, q, rows, bt, lens, bs, scale, out="f32", extra=0.0, only=None):
    """got [B, Hq, D] against the 64-bit form over rows(name, slots) [L, Hkv, D], for the sequences of ``only``."""
    hq, d = q.shape[1:]
    for s in only if only is not None else range(len(lens)):
        L = lens[s]
        sl = Q.slots_of(bt, s, 0, L, bs)
        k, v = rows("k", sl), rows("v", sl)
        hkv = k.shape[1]
        ref = Q.attend(q[s], k, v, scale)
        vmax = v.abs().amax((0, 2)).repeat_interleave(hq // hkv)[:, None].numpy() if L else np.zeros((hq, 1))
        xs = torch.einsum("hgd,lhd->hgl", q[s].double().abs().view(hkv, hq // hkv, d), k.abs()) * scale
        xmax = xs.reshape(hq, -1).amax(-1)[:, None].numpy() if L else 0.0
        tol = Q.tolerance(ref.numpy(), vmax, L, d, xmax, out) + extra * vmax
        err = (got[s].cpu().double() - ref).abs().numpy()
        assert np.all(err <= tol), f"sequence {s} (length {L}): {np.max(err / tol):.2f} of the bound"


def quant_case(lens, width, hq, hkv, d, bs, fmt, seed, **kw):
    nb = 70
    bt = pool_tables(len(lens), width, nb, seed)
    g = torch.Generator().manual_seed(seed)
    c = {}
    for n in "kv":
        x = torch.randn(nb, bs, hkv, d, generator=g)
        c[n], c[n + "s"] = Q.quantise(x.half(), fmt)
    q = (3 * torch.randn(len(lens), hq, d, generator=g)).half()
    out = torch.empty(q.shape, device="cuda")
    err = pa.new_err_flag()
    pa.quant_decode(out, q.cuda(), c["k"].cuda(), c["v"].cuda(), c["ks"].cuda(), c["vs"].cuda(), bt.cuda(),
                    torch.tensor(lens, dtype=torch.int32).cuda(), d ** -0.5, err_flag=err, **kw)
    assert pa.read_err_flag(err) == 0
    compare(out, q, lambda n, sl: Q.quant_rows(c, n, sl, fmt), bt, lens, bs, d ** -0.5)


def shared_case(members, shared, private, width, hq, hkv, d, bs, dtype, seed, only=None, extra=0.0, **kw):
    """Groups over a pool: a group's tables start with the same whole prefix blocks
    (the prefixes are whole blocks here)."""
    nb = 70
    group = [i for i, m in enumerate(members) for _ in range(m)]
    lens = [shared[i] + p for i, p in zip(group, private)]
    bt = pool_tables(len(group), width, nb, seed)
    first = np.concatenate([[0], np.cumsum(members)])
    for s, i in enumerate(group):
        assert shared[i] % bs == 0
        bt[s, :shared[i] // bs] = bt[first[i], :shared[i] // bs]
    g = torch.Generator().manual_seed(seed)
    c = {n: torch.randn(nb, bs, hkv, d, generator=g).to(Q.DT[dtype]) for n in "kv"}
    q = (3 * torch.randn(len(group), hq, d, generator=g)).to(Q.DT[dtype])
    out = torch.empty(q.shape, device="cuda")
    err = pa.new_err_flag()
    pa.decode_shared(out, q.cuda(), c["k"].cuda(), c["v"].cuda(), bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                     torch.tensor(first, dtype=torch.int32).cuda(),
                     torch.tensor([shared[i] for i in group], dtype=torch.int32).cuda(), d ** -0.5, err_flag=err, **kw)
    assert pa.read_err_flag(err) == 0
    compare(out, q, lambda n, sl: c[n].view(-1, hkv, d)[sl].double(), bt, lens, bs, d ** -0.5, extra=extra, only=only)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_automatic_partitions_of_a_quantised_cache_with_128_token_blocks(fmt):
    """19 sequences on 8 KV heads under a bound of 81,280 tokens: partitions just below 32 blocks."""
    quant_case([9000, 8100, 4064, 4065, 12200, 0, 1] + [30] * 12, 635, 8, 8, 64, 128, fmt, 1, max_context_len=81280)


@pytest.mark.parametrize("bs,n,bound", [(256, 64, 48400), (96, 19, 60800)])
def test_automatic_partitions_of_other_block_sizes(bs, n, bound):
    quant_case([9000, 17000, 40] + [3] * (n - 3), -(-bound // bs), 8, 8, 64, bs, "int8", 2, max_context_len=bound)


def test_automatic_partitions_without_a_prefix():
    """190 sequences under a bound of 4,080 tokens in blocks of 64, one pass."""
    lens = [4080, 4064, 4033, 4032, 2033] + [50] * 185
    shared_case([1] * 190, [0] * 190, lens, 64, 8, 8, 64, 64, "f16", 3, only=range(8), max_context_len=4080, max_shared_len=0)


@pytest.mark.parametrize("members", [[2] * 95, [60] + [1] * 130])
def test_automatic_partitions_behind_a_prefix(members):
    """The private parts of a batch with one shared prefix of 640 tokens, the longest of 4,064."""
    n = sum(members)
    private = [4064, 4050] + [50] * (n - 3) + [4064]
    shared_case(members, [640] + [0] * (len(members) - 1), private, 74, 8, 8, 64, 64, "bf16", 4,
                only=[0, 1, 2, n - 2, n - 1], max_context_len=640 + 4064, max_shared_len=640, max_group_size=max(members))


def test_private_parts_longer_than_the_bounds_let_expect():
    """Bounds that differ by 2,020 tokens, and private parts of twice that in groups without a prefix."""
    n = 400
    private = [2020, 2020] + [50] * (n - 4) + [4040, 4060]
    shared_case([4] + [1] * (n - 4), [1984] + [0] * (n - 4), private, 64, 8, 8, 64, 64, "f16", 5,
                only=[0, 1, 2, n - 2, n - 1], max_context_len=4060, max_shared_len=2040, max_group_size=4)


@pytest.mark.parametrize("bs,n,longest", [(64, 126, 6144), (256, 189, 16384)])
def test_automatic_partitions_of_prefixes_on_the_split_kernel(bs, n, longest):
    """Prefixes of groups of two, of which the longest fill their bound."""
    shared = [longest, longest - 2 * bs] + [bs] * (n - 2)
    shared_case([2] * n, shared, [1, 20] * n, longest // bs + 1, 8, 8, 64, bs, "f16", 6, only=[0, 1, 2, 3, 2 * n - 1],
                max_context_len=longest + 20, max_shared_len=longest, max_group_size=2)


@pytest.mark.parametrize("bs", [32, 48, 64, 128])
def test_the_longest_requests_that_start_inside_blocks(bs):
    P = 31 * bs + 16
    lens = [3 * P + 5, 2 * P, P + 1, 40, 0, 5 * P - 1]
    quant_case(lens, -(-5 * P // bs), 8, 4, 64, bs, "e4m3", 7, partition_size=P)
    shared_case([1] * 6, [0] * 6, lens, -(-5 * P // bs), 8, 4, 64, bs, "bf16", 8, partition_size=P, max_shared_len=0)


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 128), (4, 2, 64)])
@pytest.mark.parametrize("bs,P", [(64, 2032), (128, 4064), (48, 1520), (64, 2000)])
def test_decode_with_long_requests_that_start_inside_blocks(bs, P, hq, hkv, d):
    """pa.decode on the cooperative (d = 128) and the per-warp kernel."""
    lens = [3 * P + 5, 2 * P, P + 1, P, 40, 1]
    nb, width = 70, -(-(3 * P + 5) // bs)
    bt = pool_tables(len(lens), width, nb, 9)
    g = torch.Generator().manual_seed(9)
    c = {n: torch.randn(nb, bs, hkv, d, generator=g).bfloat16() for n in "kv"}
    q = (2 * torch.randn(len(lens), hq, d, generator=g)).bfloat16()
    out = torch.empty(q.shape, device="cuda")
    err = pa.new_err_flag()
    args = (bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), d ** -0.5)
    pa.decode(out, q.cuda(), c["k"].cuda(), c["v"].cuda(), *args, partition_size=P, err_flag=err)
    assert pa.read_err_flag(err) == 0
    compare(out, q, lambda n, sl: c[n].view(-1, hkv, d)[sl].double(), bt, lens, bs, d ** -0.5)
