"""Refusals of the Python calls of a serving step (4-bit cache, block tables, rotation with the cache
write), without a GPU: CPU tensors stand for the device's, and the library must not be reached."""
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_140_gb300 as pa

B16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
I32, I64, U8, I8 = torch.int32, torch.int64, torch.uint8, torch.int8


class Reached(Exception):
    """A call went as far as the library."""


class _Library:
    def __getattr__(self, name):
        if name.endswith("_workspace_size"):
            return lambda *a: 0

        def call(*a):
            raise Reached(name)
        return call


@pytest.fixture(autouse=True)
def on_the_host(monkeypatch):
    """get_device() of a CPU tensor is -1, and so the current device here."""
    from paged_kv_cache_140_gb300 import _build
    _build.build()
    rt = pa._Runtime()
    rt.lib, rt.current_device, rt.stream, rt.capturing = _Library(), lambda: -1, lambda dev: 0, lambda: False
    monkeypatch.setattr(pa, "_rt", rt)
    monkeypatch.setattr(pa, "int4_decode_workspace_size", lambda *a: 0)


def refused(call, good, changes, errors=(ValueError, TypeError)):
    """`good` goes through to the library; with any one of `changes` (a dict of arguments) it does not."""
    with pytest.raises(Reached):
        call(**good)
    for i, ch in enumerate(changes):
        with pytest.raises(errors):
            call(**{**good, **ch})
            pytest.fail(f"change {i} ({list(ch)}) was taken")


def cache4(nb=4, bs=16, hkv=2, d=128):
    c = {n + "_cache": torch.zeros(nb, bs, hkv, d // 2, dtype=U8) for n in "kv"}
    c.update({n + "_scales": torch.zeros(nb, hkv, bs, d // 64, 2, dtype=B16) for n in "kv"})
    return c


BAD_CACHES4 = [
    {"k_cache": torch.zeros(4, 16, 2, 64, dtype=I8)}, {"v_cache": torch.zeros(4, 16, 2, 64, dtype=I8)},
    {"v_cache": torch.zeros(5, 16, 2, 64, dtype=U8)}, {"k_cache": torch.zeros(4, 16, 2, 128, dtype=U8)},
    {"k_cache": torch.zeros(4, 16, 128, dtype=U8), "v_cache": torch.zeros(4, 16, 128, dtype=U8)},
    {"k_cache": torch.zeros(4, 16, 3, 64, dtype=U8), "v_cache": torch.zeros(4, 16, 3, 64, dtype=U8)},
    {"k_cache": torch.zeros(4, 16, 2, 128, dtype=U8)[..., ::2]},
    {"k_scales": torch.zeros(4, 2, 16, 2, 2, dtype=F16)}, {"v_scales": torch.zeros(4, 16, 2, 2, 2, dtype=B16)},
    {"k_scales": torch.zeros(4, 2, 16, 2, dtype=B16)}, {"v_scales": torch.zeros(4, 2, 16, 2, 4, dtype=B16)[..., ::2]}]


def test_int4_reshape_and_cache():
    rows = torch.zeros(3, 2, 128, dtype=F16)
    good = dict(key=rows, value=rows, slot_mapping=torch.zeros(3, dtype=I64), **cache4())
    wide = torch.zeros(3, 6, 128, dtype=F16)
    with pytest.raises(Reached):
        pa.int4_reshape_and_cache(**{**good, "key": wide[:, :2], "value": wide[:, 2:4]})
    refused(pa.int4_reshape_and_cache, good, BAD_CACHES4 + [
        {"key": rows.float(), "value": rows.float()}, {"value": rows.bfloat16()}, {"key": rows[:2]}, {"key": rows[0], "value": rows[0]},
        {"key": wide[:, ::3], "value": wide[:, ::3]}, {"key": torch.zeros(3, 2, 256, dtype=F16)[..., ::2]},
        {"key": torch.zeros(3, 3, 128, dtype=F16), "value": torch.zeros(3, 3, 128, dtype=F16)},
        {"slot_mapping": torch.zeros(3, dtype=I32)}, {"slot_mapping": torch.zeros(4, dtype=I64)},
        {"slot_mapping": torch.zeros(6, dtype=I64)[::2]}, {"err_flag": torch.zeros(1, dtype=I64)}])


def test_int4_gather():
    out = torch.zeros(5, 2, 128, dtype=F32)
    good = dict(out_k=out, out_v=out.clone(), block_tables=torch.zeros(2, 4, dtype=I32), cu_seqlens=torch.zeros(3, dtype=I32),
                **cache4())
    refused(pa.int4_gather, good, BAD_CACHES4 + [
        {"out_k": out.double(), "out_v": out.double()}, {"out_v": out.half()}, {"out_v": out[:4]}, {"out_k": out[0]},
        {"out_k": torch.zeros(5, 3, 128), "out_v": torch.zeros(5, 3, 128)}, {"out_k": torch.zeros(5, 2, 256)[..., ::2]},
        {"block_tables": torch.zeros(2, 4, dtype=I64)}, {"block_tables": torch.zeros(8, dtype=I32)},
        {"block_tables": torch.zeros(2, 8, dtype=I32)[:, ::2]}, {"cu_seqlens": torch.zeros(2, dtype=I32)},
        {"cu_seqlens": torch.zeros(3, dtype=I64)}, {"seq_starts": torch.zeros(3, dtype=I32)},
        {"seq_starts": torch.zeros(2, dtype=I64)}, {"seq_starts": torch.zeros(4, dtype=I32)[::2]}])


def test_int4_decode():
    q = torch.zeros(2, 4, 128, dtype=B16)
    good = dict(out=torch.zeros(2, 4, 128), query=q, block_tables=torch.zeros(2, 4, dtype=I32),
                context_lens=torch.zeros(2, dtype=I32), scale=0.1, **cache4())
    refused(pa.int4_decode, good, BAD_CACHES4[:5] + BAD_CACHES4[6:] + [
        {"query": q.float()}, {"out": q.double()}, {"out": q[:1]}, {"query": q[0], "out": q[0]},
        {"query": torch.zeros(2, 4, 256, dtype=B16)[..., ::2]}, {"out": torch.zeros(2, 4, 256)[..., ::2]},
        {"block_tables": torch.zeros(3, 4, dtype=I32)}, {"block_tables": torch.zeros(2, 4, dtype=I64)},
        {"context_lens": torch.zeros(2, dtype=I64)}, {"context_lens": torch.zeros(3, dtype=I32)},
        {"context_lens": torch.zeros(4, dtype=I32)[::2]}])


def test_update_tables():
    i = lambda n: torch.zeros(n, dtype=I32)            # noqa: E731
    good = dict(block_tables=torch.zeros(2, 4, dtype=I32), context_lens=i(2), changes=i(2), free_blocks=i(9), free_count=i(1),
                slot_mapping=torch.zeros(5, dtype=I64), positions=torch.zeros(5, dtype=I64), cu_seqlens=i(3), block_size=16)
    refused(pa.update_tables, good, [
        {"block_tables": torch.zeros(2, 4, dtype=I64)}, {"block_tables": i(8)}, {"block_tables": torch.zeros(2, 8, dtype=I32)[:, ::2]},
        {"context_lens": i(3)}, {"context_lens": torch.zeros(2, dtype=I64)}, {"context_lens": i(4)[::2]},
        {"changes": i(1)}, {"changes": torch.zeros(2, dtype=I64)}, {"changes": i(4)[::2]},
        {"out_lens": i(3)}, {"out_lens": torch.zeros(2, dtype=I64)}, {"out_lens": i(4)[::2]},
        {"free_blocks": torch.zeros(9, dtype=I64)}, {"free_blocks": i(18)[::2]}, {"free_count": i(2)},
        {"free_count": torch.zeros(1, dtype=I64)}, {"out_free_count": i(0)}, {"out_free_count": torch.zeros(1, dtype=I64)},
        {"slot_mapping": torch.zeros(5, dtype=I32)}, {"slot_mapping": torch.zeros(10, dtype=I64)[::2]},
        {"positions": torch.zeros(4, dtype=I64)}, {"positions": torch.zeros(5, dtype=I32)},
        {"positions": torch.zeros(10, dtype=I64)[::2]}, {"cu_seqlens": i(2)}, {"cu_seqlens": torch.zeros(3, dtype=I64)},
        {"cu_seqlens": i(6)[::2]}, {"err_flag": torch.zeros(1, dtype=I64)}])


def test_rope_and_cache():
    def z(*shape, dtype=B16):
        return torch.zeros(*shape, dtype=dtype)
    half = dict(k_cache=z(4, 16, 2, 128), v_cache=z(4, 16, 2, 128))
    good = dict(out_q=z(3, 4, 128), query=z(3, 4, 128), key=z(3, 2, 128), value=z(3, 2, 128), slot_mapping=z(3, dtype=I64),
                positions=z(3, dtype=I64), inv_freq=z(32, dtype=F64), **half)
    rows = dict(k_scales=z(4, 16, 2, dtype=F32), v_scales=z(4, 16, 2, dtype=F32))
    codes = {t: dict(k_cache=z(4, 16, 2, 128, dtype=t), v_cache=z(4, 16, 2, 128, dtype=t)) for t in (I8, U8, torch.float8_e4m3fn)}
    for kind in (codes[U8], codes[torch.float8_e4m3fn], {**codes[I8], **rows}, {**codes[U8], **rows}, cache4()):
        with pytest.raises(Reached):
            pa.rope_and_cache(**{**good, **kind})
    refused(pa.rope_and_cache, good, [
        {"query": z(3, 4, 128, dtype=F32), "out_q": z(3, 4, 128, dtype=F32)}, {"out_q": z(3, 4, 128, dtype=F16)},
        {"out_q": z(2, 4, 128)}, {"out_q": z(3, 4, 256)[..., ::2]}, {"query": z(3, 512), "out_q": z(3, 512)},
        {"query": z(3, 4, 256)[..., ::2]}, {"query": z(3, 8, 128)[:, ::2]}, {"key": z(3, 4, 128)[:, ::2]},
        {"value": z(3, 4, 128)[:, ::2]}, {"key": z(2, 2, 128), "value": z(2, 2, 128)}, {"value": z(3, 3, 128)},
        {"key": z(3, 2, 64), "value": z(3, 2, 64)}, {"key": z(3, 2, 128, dtype=F16), "value": z(3, 2, 128, dtype=F16)},
        {"key": z(3, 3, 128), "value": z(3, 3, 128)}, {"v_cache": z(5, 16, 2, 128)}, {"v_cache": z(4, 16, 2, 128, dtype=F16)},
        {"k_cache": z(4, 16, 2, 64), "v_cache": z(4, 16, 2, 64)}, {"k_cache": z(4, 16, 2, 256)[..., ::2]},
        {"k_cache": z(4, 16, 2, 128, dtype=F16), "v_cache": z(4, 16, 2, 128, dtype=F16)}, codes[I8],
        {**codes[U8], "k_scales": rows["k_scales"]}, rows, {**codes[I8], "k_scales": z(4, 2, 16, dtype=F32), "v_scales": z(4, 2, 16, dtype=F32)},
        {**codes[I8], "k_scales": z(4, 16, 2, dtype=F64), "v_scales": z(4, 16, 2, dtype=F64)},
        {**codes[I8], "k_scales": rows["k_scales"], "v_scales": z(4, 16, 4, dtype=F32)[..., ::2]},
        *[{**cache4(), **ch} for ch in BAD_CACHES4],
        {"slot_mapping": z(3, dtype=I32)}, {"slot_mapping": z(4, dtype=I64)}, {"slot_mapping": z(6, dtype=I64)[::2]},
        {"positions": z(3, dtype=I32)}, {"positions": z(2, dtype=I64)}, {"positions": z(6, dtype=I64)[::2]},
        {"inv_freq": z(32, dtype=F32)}, {"inv_freq": z(64, dtype=F64)[::2]}, {"q_weight": z(64)}, {"k_weight": z(128, dtype=F16)},
        {"q_weight": z(256)[::2]}, {"err_flag": torch.zeros(1, dtype=I64)}])


class Elsewhere:
    """A tensor that says it is on device 3."""

    def __init__(self, t):
        self._t = t

    def __getattr__(self, name):
        return getattr(self._t, name)

    def get_device(self):
        return 3


def test_tensors_of_another_device():
    """One tensor elsewhere than the rest, in turn: the call is refused before the library is reached."""
    q, kv = torch.zeros(3, 4, 128, dtype=B16), torch.zeros(3, 2, 128, dtype=B16)
    i = lambda n: torch.zeros(n, dtype=I32)            # noqa: E731
    slots = torch.zeros(3, dtype=I64)
    calls = [
        (pa.int4_reshape_and_cache, dict(key=kv, value=kv.clone(), slot_mapping=slots, **cache4())),
        (pa.int4_gather, dict(out_k=kv, out_v=kv.clone(), block_tables=torch.zeros(2, 4, dtype=I32), cu_seqlens=i(3),
                              seq_starts=i(2), **cache4())),
        (pa.int4_decode, dict(out=torch.zeros(2, 4, 128), query=q[:2], block_tables=torch.zeros(2, 4, dtype=I32),
                              context_lens=i(2), scale=0.1, **cache4())),
        (pa.update_tables, dict(block_tables=torch.zeros(2, 4, dtype=I32), context_lens=i(2), changes=i(2), free_blocks=i(9),
                                free_count=i(1), slot_mapping=slots, positions=slots.clone(), cu_seqlens=i(3), block_size=16,
                                out_lens=i(2), out_free_count=i(1))),
        (pa.rope_and_cache, dict(out_q=q, query=q.clone(), key=kv, value=kv.clone(), slot_mapping=slots, positions=slots.clone(),
                                 inv_freq=torch.zeros(32, dtype=F64), q_weight=torch.zeros(128, dtype=B16),
                                 k_weight=torch.zeros(128, dtype=B16), **cache4()))]
    for call, good in calls:
        with pytest.raises(Reached):
            call(**good)
        for name, t in good.items():
            if torch.is_tensor(t):
                with pytest.raises(ValueError):
                    call(**{**good, name: Elsewhere(t)})
                    pytest.fail(f"{call.__name__}: {name} was taken")
