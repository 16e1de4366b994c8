"""GPU tests of how accurately quantised decode sums V: errors in proportion to each
output's own sum of magnitudes, not to the row's largest value."""
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


def decode(q, k, v, fmt, bs, **kw):
    """(output [1, Hq, D], quantised K and V in 64 bits) of one sequence of rows k, v [L, Hkv, D]."""
    L, hkv, d = k.shape
    bt, nb = Q.tables([L], bs, 3)
    c = Q.quant_cache([1], bt, nb, bs, hkv, d, fmt, 1)
    sl = Q.slots_of(bt, 0, 0, L, bs)
    for n, x in (("k", k), ("v", v)):
        codes, sc = Q.quantise(x, fmt)
        c[n].view(-1, hkv, d)[sl] = codes
        c[n + "s"].view(-1, hkv)[sl] = sc
    out = torch.empty(q.shape, device="cuda")
    pa.quant_decode(out, q.cuda(), c["k"].cuda(), c["v"].cuda(), c["ks"].cuda(), c["vs"].cuda(), bt.cuda(),
                    torch.tensor([L], dtype=torch.int32).cuda(), 1.0, **kw)
    return out.cpu().double(), Q.quant_rows(c, "k", sl, fmt), Q.quant_rows(c, "v", sl, fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("hq,hkv,d,L", [(8, 8, 128, 5000), (4, 1, 64, 3000), (16, 2, 128, 777), (8, 8, 64, 16)])
def test_dims_without_a_value_come_out_as_zero(hq, hkv, d, L, fmt):
    g = torch.Generator().manual_seed(L)
    q, k = torch.randn(1, hq, d, generator=g).half() / 4, torch.randn(L, hkv, d, generator=g).half()
    v = torch.zeros(L, hkv, d)
    v[..., 5] = torch.randn(L, hkv, generator=g)
    out, _, _ = decode(q, k, v.half(), fmt, 32)
    keep = torch.arange(d) != 5
    assert torch.all(out[..., keep] == 0) and torch.all(out[..., 5] != 0)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("hq,hkv,d,bs,L,P", [(8, 8, 128, 128, 8000, 4096), (4, 4, 64, 32, 8000, 1024), (8, 1, 128, 256, 8192, 8192),
                                             (8, 8, 128, 16, 300, 0)])
def test_sums_of_few_values_among_many_tokens(hq, hkv, d, bs, L, P, fmt):
    """Flat weights over a long partition; every row holds one large value, in dim 0, and
    each other dim a value in three tokens only.

    A dim's sum has three terms that are not 0, so its numerator takes at most three
    products (weights as two binary16 parts, 2^-22 each; the scale and the exponential 2
    ulp) and additions; the sum of the weights takes L additions, L 2^-24 at most.  All
    relative to sum p |v| of that dim: (L + 64) 2^-24."""
    g = torch.Generator().manual_seed(L + P)
    q, k = torch.zeros(1, hq, d).half(), torch.randn(L, hkv, d, generator=g).half()
    v = torch.zeros(L, hkv, d)
    v[..., 0] = 1.0 + torch.rand(L, hkv, generator=g)
    for i in range(1, d):
        v[torch.randperm(L, generator=g)[:3], :, i] = torch.randn(3, hkv, generator=g)
    out, _, vq = decode(q, k, v.half(), fmt, bs, partition_size=P)
    rep = hq // hkv
    ref = vq.mean(0).repeat_interleave(rep, 0)
    size = vq.abs().mean(0).repeat_interleave(rep, 0)
    err = (out[0] - ref).abs()
    assert torch.all(err <= (L + 64) * 2.0 ** -24 * size), (err / size.clamp(min=1e-30)).max().item() * 2 ** 24
