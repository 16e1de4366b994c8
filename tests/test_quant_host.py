"""Host-side checks of the quantised-cache and shared-prefix calls: refusals
that return before any CUDA call, planning, and the tests' own 64-bit forms."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quant_harness as Q


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_140_gb300 import _build, _lib
    _build.build()
    return _lib.load()


NUL = ctypes.c_void_p(0)
BAD = ctypes.c_size_t(-1).value


def test_write_and_read_refusals(lib):
    from paged_kv_cache_140_gb300 import _lib as L

    def write(T=3, ks=256, vs=256, nb=8, bs=16, hkv=4, d=64, dt=0, cdt=4):
        return lib.pa_quant_reshape_and_cache(NUL, NUL, ks, vs, NUL, NUL, NUL, NUL, NUL, T, nb, bs, hkv, d, dt, cdt, NUL,
                                              NUL)
    assert write(T=0) == L.PA_OK
    assert write() == L.PA_ERR_INVALID_ARG                   # null tensors
    assert write(T=-1) == L.PA_ERR_INVALID_ARG
    assert write(T=0, cdt=0) == L.PA_ERR_INVALID_ARG         # not a quantised cache
    assert write(T=0, dt=2) == L.PA_ERR_INVALID_ARG          # f32 rows
    assert write(T=0, d=96) == L.PA_ERR_UNSUPPORTED
    assert write(T=0, ks=255) == L.PA_ERR_INVALID_ARG        # stride below a row
    assert write(T=0, vs=260) == L.PA_ERR_INVALID_ARG        # stride no multiple of 8

    def gather(T=3, B=2, odt=2, cdt=3, d=64, maxnb=4, bs=16):
        return lib.pa_quant_gather(NUL, NUL, odt, NUL, NUL, cdt, NUL, NUL, NUL, maxnb, NUL, NUL, B, T, 4, d, bs, 8, NUL,
                                   NUL)
    assert gather(T=0) == L.PA_OK and gather(B=0) == L.PA_OK
    assert gather() == L.PA_ERR_INVALID_ARG
    assert gather(T=0, cdt=1) == L.PA_ERR_INVALID_ARG
    assert gather(T=0, odt=3) == L.PA_ERR_INVALID_ARG
    assert gather(T=0, d=80) == L.PA_ERR_UNSUPPORTED
    assert gather(T=1 << 31) == L.PA_ERR_UNSUPPORTED
    assert gather(T=0, maxnb=0) == L.PA_ERR_INVALID_ARG


def test_decode_refusals(lib):
    from paged_kv_cache_140_gb300 import _lib as L

    def dec(B=2, hq=8, hkv=8, d=64, bs=16, maxnb=8, ctx=100, qdt=0, cdt=4, odt=2, scale=0.1, P=0, nb=64):
        return lib.pa_quant_decode(NUL, odt, NUL, qdt, NUL, NUL, cdt, NUL, NUL, NUL, maxnb, NUL, ctx, B, hq, hkv, d, bs,
                                   nb, scale, P, NUL, 0, NUL, NUL)
    assert dec(B=0) == L.PA_OK
    assert dec() == L.PA_ERR_INVALID_ARG
    for kw in (dict(cdt=0), dict(qdt=2), dict(odt=4), dict(hq=9), dict(ctx=129), dict(scale=float("nan")), dict(P=24),
               dict(P=1024), dict(B=-1), dict(ctx=-1), dict(scale=float("inf"))):
        assert dec(**{"B": 0, **kw}) == L.PA_ERR_INVALID_ARG, kw
    for kw in (dict(hq=24), dict(d=96), dict(bs=12), dict(nb=1 << 30)):
        assert dec(**{"B": 0, **kw}) == L.PA_ERR_UNSUPPORTED, kw
    # a partition whose 33 blocks would not fit a warp's lanes
    assert dec(B=0, bs=64, maxnb=100, ctx=6000, P=2032) == L.PA_ERR_INVALID_ARG
    assert dec(B=0, bs=64, maxnb=100, ctx=6000, P=2048) == L.PA_OK
    assert dec(B=0, bs=64, maxnb=100, ctx=6000, P=2000) == L.PA_OK


def test_shared_refusals(lib):
    from paged_kv_cache_140_gb300 import _lib as L

    def dec(B=0, ng=0, mg=0, ms=50, hq=8, hkv=8, d=64, bs=16, maxnb=8, ctx=100, dt=0, odt=2, P=0, scale=0.1):
        return lib.pa_decode_shared(NUL, odt, NUL, NUL, NUL, dt, NUL, maxnb, NUL, ctx, NUL, ng, mg, NUL, ms, B, hq, hkv,
                                    d, bs, 64, scale, P, NUL, 0, NUL, NUL)
    assert dec() == L.PA_OK
    assert dec(B=4, ng=2, mg=2) == L.PA_ERR_INVALID_ARG      # null tensors
    for kw in (dict(ms=101), dict(ms=-1), dict(ng=-1), dict(mg=-1), dict(dt=4), dict(dt=3), dict(odt=3),
               dict(B=4, ng=1, mg=3), dict(P=8), dict(scale=-0.1), dict(scale=float("nan"))):
        assert dec(**kw) == L.PA_ERR_INVALID_ARG, kw
    for kw in (dict(hq=24), dict(d=32), dict(bs=24)):
        assert dec(**kw) == L.PA_ERR_UNSUPPORTED, kw


def test_planning(lib):
    ws = lib.pa_quant_decode_workspace_size
    assert ws(4, 4, 4, 64, 16, 256, 0) == 0                  # a few ring slots are not cut
    assert ws(256, 40, 40, 128, 16, 256, 0) == 0             # nor are lists that fill the GPU
    assert ws(4, 8, 8, 128, 16, 256, 0) > 0
    assert ws(256, 40, 40, 128, 16, 2048, 0) >= 256 * 40 * 4 * 132 * 4
    # few sequences: finer partitions, more partials per row
    assert ws(1, 8, 8, 128, 16, 8192, 0) >= 8 * 64 * 132 * 4
    assert ws(1, 8, 8, 128, 16, 8192, 8192) == BAD           # more than 32 blocks
    assert ws(1, 12, 8, 128, 16, 100, 0) == BAD
    sh = lib.pa_decode_shared_workspace_size
    assert sh(8, 2, 4, 8, 8, 128, 16, 2000, 1000, 0) > 0
    assert sh(4, 1, 4, 4, 4, 64, 16, 100, 64, 0) == 0        # small: one pass, nothing to join
    assert sh(8, 2, 500, 8, 8, 128, 16, 2000, 1000, 0) == sh(8, 2, 8, 8, 8, 128, 16, 2000, 1000, 0)   # at most the batch
    assert sh(8, 2, 4, 8, 8, 128, 16, 2000, 2001, 0) == BAD
    assert sh(8, 2, 4, 8, 8, 128, 12, 2000, 1000, 0) == BAD


def test_plain_rounding_to_e4m3_is_torch_conversion():
    y = torch.cat([torch.linspace(-448, 448, 20011), torch.randn(20000) * 2.0 ** torch.randint(-12, 8, (20000,))])
    y = y.clamp(-448, 448)
    want = y.to(torch.float8_e4m3fn).view(torch.uint8)
    assert np.array_equal(Q.round_e4m3(y.numpy()), want.numpy())
    v = Q.e4m3_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(v, t, equal_nan=True)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_plain_quantisation_is_within_half_a_step(fmt):
    x = (torch.randn(50, 3, 64) * torch.exp(3 * torch.randn(50, 3, 1))).bfloat16()
    codes, scales = Q.quantise(x, fmt)
    back = Q.values(codes, fmt) * scales.double()[..., None]
    err = (back - x.double()).abs()
    step = scales.double()[..., None]
    # int8: half a step; e4m3: half a relative step, or half the subnormal spacing (plus the fp32 roundings)
    bound = 0.5 * step if fmt == "int8" else torch.maximum(x.double().abs() * 2.0 ** -4, 2.0 ** -10 * step)
    assert torch.all(err <= bound * (1 + 1e-6) + 127 * 2.0 ** -22 * step)
