"""Host-side checks of the 4-bit cache, table update and rotation calls: refusals that
return before any CUDA call, planning, helpers, and the tests' own 64-bit forms."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import step_harness as S


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_140_gb300 import _build, _lib
    _build.build()
    return _lib.load()


NUL = ctypes.c_void_p(0)
BAD = ctypes.c_size_t(-1).value


def test_int4_write_and_read_refusals(lib):
    from paged_kv_cache_140_gb300 import _lib as L

    def write(T=3, ks=256, vs=256, nb=8, bs=16, hkv=4, d=64, dt=0):
        return lib.pa_int4_reshape_and_cache(NUL, NUL, ks, vs, NUL, NUL, NUL, NUL, NUL, T, nb, bs, hkv, d, dt, NUL, NUL)
    assert write(T=0) == L.PA_OK
    assert write() == L.PA_ERR_INVALID_ARG                   # null tensors
    for kw in (dict(T=-1), dict(dt=2), dict(ks=255), dict(vs=260), dict(nb=0), dict(bs=0)):
        assert write(**{"T": 0, **kw}) == L.PA_ERR_INVALID_ARG, kw
    for kw in (dict(d=96), dict(nb=1 << 28), dict(nb=1 << 30, bs=1, hkv=4)):
        assert write(**{"T": 0, "ks": 1 << 12, "vs": 1 << 12, **kw}) == L.PA_ERR_UNSUPPORTED, kw

    def gather(T=3, B=2, odt=2, d=64, maxnb=4, bs=16, nb=8):
        return lib.pa_int4_gather(NUL, NUL, odt, NUL, NUL, NUL, NUL, NUL, maxnb, NUL, NUL, B, T, 4, d, bs, nb, NUL, NUL)
    assert gather(T=0) == L.PA_OK and gather(B=0) == L.PA_OK
    assert gather() == L.PA_ERR_INVALID_ARG
    assert gather(T=0, odt=3) == L.PA_ERR_INVALID_ARG
    assert gather(T=0, maxnb=0) == L.PA_ERR_INVALID_ARG
    assert gather(T=0, d=80) == L.PA_ERR_UNSUPPORTED
    assert gather(T=1 << 31) == L.PA_ERR_UNSUPPORTED
    assert gather(T=0, nb=1 << 29) == L.PA_ERR_UNSUPPORTED


def test_int4_decode_refusals_and_planning(lib):
    from paged_kv_cache_140_gb300 import _lib as L

    def dec(B=0, hq=8, hkv=8, d=64, bs=16, maxnb=8, ctx=100, qdt=0, odt=2, scale=0.1, P=0, nb=64):
        return lib.pa_int4_decode(NUL, odt, NUL, qdt, NUL, NUL, NUL, NUL, NUL, maxnb, NUL, ctx, B, hq, hkv, d, bs, nb, scale,
                                  P, NUL, 0, NUL, NUL)
    assert dec() == L.PA_OK
    assert dec(B=2) == L.PA_ERR_INVALID_ARG                  # null tensors
    for kw in (dict(qdt=2), dict(odt=4), dict(hq=9), dict(ctx=129), dict(scale=float("nan")), dict(P=24), dict(P=1024),
               dict(B=-1), dict(ctx=-1), dict(scale=float("inf"))):
        assert dec(**kw) == L.PA_ERR_INVALID_ARG, kw
    for kw in (dict(hq=24), dict(d=96), dict(bs=12), dict(nb=1 << 30)):
        assert dec(**kw) == L.PA_ERR_UNSUPPORTED, kw
    ws = lib.pa_int4_decode_workspace_size
    assert ws(4, 4, 4, 64, 16, 100, 0) == 0
    assert ws(256, 40, 40, 128, 16, 2048, 0) >= 256 * 40 * 4 * 132 * 4
    # every half of up to 256 CTAs may leave rows of an item it continues
    assert ws(1, 8, 8, 128, 16, 8192, 0) - lib.pa_quant_decode_workspace_size(1, 8, 8, 128, 16, 8192, 0) >= 256 * 8 * 132 * 4
    assert ws(1, 8, 8, 128, 16, 8192, 8192) == BAD and ws(1, 12, 8, 128, 16, 100, 0) == BAD


def test_update_tables_refusals(lib):
    from paged_kv_cache_140_gb300 import _lib as L
    one = ctypes.c_void_p(0x1000)

    def up(bt=one, maxnb=8, lens=one, ch=one, out=one, B=2, free=one, cap=10, cnt=one, outc=one, nb=10, bs=16, cu=one,
           slots=one, pos=one, T=4):
        return lib.pa_update_tables(bt, maxnb, lens, ch, out, B, free, cap, cnt, outc, nb, bs, cu, slots, pos, T, NUL, NUL)
    for kw in (dict(bt=NUL), dict(lens=NUL), dict(ch=NUL), dict(out=NUL), dict(free=NUL), dict(cnt=NUL), dict(outc=NUL),
               dict(cu=NUL), dict(slots=NUL), dict(pos=NUL), dict(B=-1), dict(maxnb=0), dict(cap=-1), dict(nb=0), dict(bs=0),
               dict(T=-1)):
        assert up(**kw) == L.PA_ERR_INVALID_ARG, kw
    for kw in (dict(B=8193), dict(maxnb=1 << 27), dict(T=(1 << 30) + 1), dict(cap=1 << 31), dict(nb=1 << 31)):
        assert up(**kw) == L.PA_ERR_UNSUPPORTED, kw


def test_rope_refusals(lib):
    from paged_kv_cache_140_gb300 import _lib as L
    one, odd = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)

    def rope(T=0, hq=4, hkv=2, d=64, dt=0, cdt=0, qs=256, ks=128, vs=128, rot=64, factor=1.0, eps=1e-6, nb=8, bs=16,
             scales=(NUL, NUL), ksc=1.0, vsc=1.0, out=one, q=one, kc=one):
        return lib.pa_rope_and_cache(out, q, one, one, qs, ks, vs, kc, one, cdt, scales[0], scales[1], ksc, vsc, one, one,
                                     one, rot, 0, factor, NUL, NUL, eps, T, hq, hkv, d, dt, nb, bs, NUL, NUL)
    assert rope() == L.PA_OK
    assert rope(cdt=3) == L.PA_OK                            # e4m3, one scale per tensor
    assert rope(cdt=4, scales=(one, one)) == L.PA_OK and rope(cdt=5, scales=(one, one)) == L.PA_OK
    for kw in (dict(T=-1), dict(hq=0), dict(dt=2), dict(rot=0), dict(rot=12), dict(rot=72), dict(factor=float("nan")),
               dict(eps=-1.0), dict(eps=float("nan")), dict(qs=255), dict(qs=260), dict(ks=120), dict(vs=130), dict(cdt=2),
               dict(cdt=3, ksc=0.0), dict(cdt=3, vsc=float("inf")), dict(T=1, cdt=4), dict(T=1, cdt=5, scales=(one, NUL)),
               dict(T=1, out=NUL), dict(T=1, kc=odd), dict(T=1, out=odd), dict(T=1, qs=512)):
        assert rope(**kw) == L.PA_ERR_INVALID_ARG, kw
    for kw in (dict(d=96, qs=4096, ks=4096, vs=4096), dict(cdt=1), dict(T=1 << 31),
               dict(cdt=5, scales=(one, one), nb=1 << 28)):
        assert rope(**kw) == L.PA_ERR_UNSUPPORTED, kw


def test_frequencies():
    import paged_kv_cache_140_gb300 as pa
    f, m = pa.rope_frequencies(128, device="cpu")
    assert m == 1.0 and f.dtype == torch.float64 and f.numel() == 64
    assert f[0] == 1.0 and abs(f[1].item() - 10000.0 ** (-1 / 64)) < 1e-15
    lin, _ = pa.rope_frequencies(128, scaling="linear", scale=4.0, device="cpu")
    assert torch.allclose(lin * 4, f, rtol=1e-15)
    b, _ = pa.rope_frequencies(128, scaling="base", scale=4.0, device="cpu")
    assert b[0] == 1.0 and abs(b[-1].item() * 4 / f[-1].item() - 1) < 1e-12
    p, m = pa.rope_frequencies(128, scaling="parts", scale=32.0, device="cpu")
    assert abs(m - (0.1 * math.log(32) + 1)) < 1e-15
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(p[turns >= 32], f[turns >= 32])
    assert torch.allclose(p[turns <= 1], f[turns <= 1] / 32, rtol=1e-15)
    assert torch.all(p[1:] <= p[:-1])
    for bad in (dict(rot_dim=12), dict(rot_dim=0), dict(rot_dim=64, base=1.0), dict(rot_dim=64, scaling="none"),
                dict(rot_dim=64, scaling="parts", fast_turns=1.0), dict(rot_dim=64, scaling="linear", scale=0.5)):
        with pytest.raises(ValueError):
            pa.rope_frequencies(device="cpu", **bad)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("offset", [0.0, 3.0, 300.0])
def test_plain_4bit_codes_are_within_half_a_step(dtype, offset):
    x = ((torch.randn(50, 3, 128, generator=torch.Generator().manual_seed(1)) + offset) *
         torch.exp(2 * torch.randn(50, 3, 1, generator=torch.Generator().manual_seed(2)))).to(dtype)
    codes, words = S.quantise4(x)
    back = S.values4(codes, words)
    g = x.double().unflatten(-1, (-1, 64))
    s, z = words[..., 0].double(), words[..., 1].double()
    # half a code; s and z are rounded to bf16, each off by up to 2^-8 of itself (8 significant bits: half a last
    # place is 2^-8 of a number at the bottom of its binade): a range of 15 codes that falls short by 2^-8, and z; 32-bit steps
    bound = s * (0.5 + 15 * 2.0 ** -8 + z.abs() * 2.0 ** -8 + (z.abs() + 16) * 2.0 ** -22)
    # (some f16 rows come out infinite: their groups have the scale NaN, and no codes to look at)
    ok = torch.isfinite(g).all(-1)
    assert torch.equal(s.isnan(), ~ok) and torch.all(codes.unflatten(-1, (-1, 32))[~ok] == 0)
    assert torch.all(((back.unflatten(-1, (-1, 64)) - g).abs() <= bound[..., None])[ok])
    # s is a fifteenth of the range, or 2^-8 of the largest value, to bf16, so |min / s| is at most
    # 2^8 (1 + 2^-8 + 2^-15) = 257.01, which bf16 (a last place of 2 there) rounds to 258 at most
    assert torch.all(((s * 15 >= (g.amax(-1) - g.amin(-1)) * (1 - 2.0 ** -8)) & (z.abs() <= 258))[ok])


def test_plain_turn_is_a_rotation():
    x = torch.randn(5, 2, 64, dtype=torch.float64, generator=torch.Generator().manual_seed(0))
    f = torch.tensor([10000.0 ** (-i / 32) for i in range(32)], dtype=torch.float64)
    pos = torch.tensor([0, 1, 7, -7, 123456])
    for inter in (False, True):
        y = S.turn(x, pos, f, inter)
        assert torch.equal(y[0], x[0])
        assert torch.allclose(y.square().sum(-1), x.square().sum(-1), rtol=1e-12)
        # scores of a query and a key depend on the distance alone
        a, b = S.turn(x, pos + 1000, f, inter), S.turn(x.flip(0).contiguous(), pos + 1000, f, inter)
        c, d = S.turn(x, pos, f, inter), S.turn(x.flip(0).contiguous(), pos, f, inter)
        assert torch.allclose((a * b).sum(-1), (c * d).sum(-1), atol=1e-9)


def test_plain_update_is_its_own_undoing():
    bt, free = [[0, 1, -1], [2, -1, -1]], [3, 4, 5, -1, -1, -1]
    new = S.update(bt, [20, 3], [16, 30], free, 3, 16, 46)
    assert new[0] == [[0, 1, 5], [2, 4, 3]] and new[1] == [36, 33] and new[3] == 0
    back = S.update(*new[:2], [-16, -30], new[2], new[3], 16, 0)
    assert back[1] == [20, 3] and back[2] == free and back[3] == 3
