"""GPU tests of the default workspaces of the calls that keep one per thread and stream."""
import gc
import threading

import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_140_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_140_gb300 import _build
    _build.build()


def shared_call():
    """A call that needs a workspace of tens of MB, and its result."""
    n, hq, hkv, d, bs, width = 64, 8, 8, 64, 16, 256
    g = torch.Generator(device="cuda").manual_seed(0)
    cache = torch.randn(300, bs, hkv, d, generator=g, device="cuda").half()
    bt = torch.randint(0, 300, (n, width), generator=g, device="cuda").int()
    bt[:, :128] = bt[0, :128]
    args = dict(query=torch.randn(n, hq, d, generator=g, device="cuda").half(), k_cache=cache, v_cache=cache.roll(1, 0),
                block_tables=bt, context_lens=torch.full((n,), 4000, dtype=torch.int32, device="cuda"),
                cu_groups=torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                shared_lens=torch.full((n,), 2048, dtype=torch.int32, device="cuda"), scale=0.125)
    assert pa.decode_shared_workspace_size(n, 1, n, hq, hkv, d, bs, width * bs, width * bs) > 8 << 20

    def call(out):
        pa.decode_shared(out, **args)
    return call, torch.empty(n, hq, d, device="cuda")


def test_workspaces_go_with_their_threads():
    call, out = shared_call()
    call(out)                                   # this thread's own stays
    torch.cuda.synchronize()
    want = out.clone()
    gc.collect()
    held = torch.cuda.memory_allocated()
    during = []

    def work(o):
        for _ in range(3):
            call(o)
        during.append(torch.cuda.memory_allocated())
    outs = [torch.empty_like(out) for _ in range(6)]
    held += sum(-(-o.nbytes // 512) * 512 for o in outs)
    for o in outs:
        t = threading.Thread(target=work, args=(o,))
        t.start()
        t.join()
    torch.cuda.synchronize()
    gc.collect()
    assert max(during) > held + (8 << 20)       # each had one of its own
    assert torch.cuda.memory_allocated() == held
    for o in outs:                              # buffers handed from thread to thread on one stream
        assert torch.equal(o, want)


def test_a_thread_keeps_its_workspace_between_calls():
    call, out = shared_call()
    call(out)
    before = torch.cuda.memory_allocated()
    for _ in range(5):
        call(out)
    assert torch.cuda.memory_allocated() == before


def test_a_replaced_buffer_is_not_handed_out_while_its_last_stream_runs():
    """A workspace made on one stream, used on another and grown there."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    ws, size = pa.DecodeWorkspace("cuda"), 40 << 20
    first, second = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(first):
        old = ws.get(size).data_ptr()
    second.wait_stream(first)
    with torch.cuda.stream(second):
        ws.get(size).zero_()
        torch.cuda._sleep(200_000_000)          # what still uses the buffer
        assert ws.get(2 * size).data_ptr() != old
    with torch.cuda.stream(first):
        fresh = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert not second.query() and fresh.data_ptr() != old
    torch.cuda.synchronize()
