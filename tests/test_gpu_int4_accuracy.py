"""GPU tests of how accurately decode over the 4-bit cache sums V: in proportion to the sum itself,
not to its terms."""
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


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 128), (16, 8, 128), (32, 8, 128), (64, 8, 128), (8, 8, 64), (64, 8, 64)])
def test_sums_of_values_of_both_signs(hq, hkv, d):
    """Flat weights over 32,000 tokens whose values cancel, so that a sum grows as its terms' random walk does.

    32,000 tokens by 8 heads are cut into one share for each of 152 SMs at least, of 224 tokens
    and a slot of 32 at either end: 288.  A product of 16 tokens may cut one unit, 2^-23, off its
    accumulator, twice where weights come as two products.  If accumulators follow the walk too,
    36 cuts of 2^-23 sqrt(i / 18) of the sum, both ways, make (2/3) 36 2^-23 = 2^-18.4 of it; shares'
    errors add up as the shares do at worst.  The zeros' sums (16 lanes, 18 additions each of
    up to 7.5 (18) of the weight, half a unit 2^-24 of that: random, 16 x 9 x 7.5 x sqrt(18) 2^-24 / 4 of a
    weight against a sum of 4 sqrt(288)) 2^-20, the weights' two parts (2^-22), the exponential and the scale
    2^-22 each: below 2^-17 in all."""
    L, bs = 32000, 32
    bt, nb = Q.tables([L], bs, 3)
    c = S.cache4([L], bt, nb, bs, hkv, d, 5, vary=0.0)
    sl = Q.slots_of(bt, 0, 0, L, bs)
    S.store4(c, "k", sl, torch.zeros(L, hkv, d).bfloat16())
    q = torch.randn(1, hq, d, generator=torch.Generator().manual_seed(1)).half()
    out = torch.empty(q.shape, device="cuda")
    pa.int4_decode(out, q.cuda(), c["k"].cuda(), c["v"].cuda(), c["ks"].cuda(), c["vs"].cuda(), bt.cuda(),
                   torch.tensor([L], dtype=torch.int32).cuda(), float(np.float32(d ** -0.5)))
    ref = S.rows4(c, "v", sl).mean(0).repeat_interleave(hq // hkv, 0)
    err = ((out[0].cpu().double() - ref).norm() / ref.norm()).item()
    assert err <= 2.0 ** -17, err


@pytest.mark.parametrize("hq", [8, 64])
def test_heads_without_a_value_beside_heads_with_values(hq):
    """Rows of zeros in one head, values of both signs, of one sign, and a single token in the others:
    a head of zeros answers nothing that could be seen beside the smallest value of the format, 2^-60."""
    hkv, d, bs, lens = 8, 128, 16, [1, 2, 333]
    bt, nb = Q.tables(lens, bs, 3)
    c = S.cache4(lens, bt, nb, bs, hkv, d, 5)
    q = torch.randn(3, hq, d, generator=torch.Generator().manual_seed(1)).half()
    for s, L in enumerate(lens):
        sl = Q.slots_of(bt, s, 0, L, bs)
        x = torch.randn(L, hkv, d, generator=torch.Generator().manual_seed(s))
        x[:, 1] = 0
        x[:, 2] = x[:, 2].abs() + 1
        x[:, 3] = -x[:, 3].abs() - 1
        S.store4(c, "v", sl, x.bfloat16())
    out = torch.empty(q.shape, device="cuda")
    pa.int4_decode(out, q.cuda(), c["k"].cuda(), c["v"].cuda(), c["ks"].cuda(), c["vs"].cuda(), bt.cuda(),
                   torch.tensor(lens, dtype=torch.int32).cuda(), float(np.float32(d ** -0.5)))
    r = hq // hkv
    got = out.cpu().double()
    # 15 units of 2^-60, in sums that are right to 2^-18
    assert torch.all(got[:, r:2 * r].abs() <= 15 * 2.0 ** -78)
    assert torch.all(got[:, 2 * r:3 * r] > 0) and torch.all(got[:, 3 * r:4 * r] < 0)
