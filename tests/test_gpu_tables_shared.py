"""GPU test of block-table updates for sequences that share their first blocks: how they begin and end."""
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


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("order", [(0, 1, 2), (2, 1, 0), (1, 0, 2)])
def test_sequences_that_share_their_first_blocks(order):
    """A prompt of three blocks, two of which two more sequences take over; all decode, then end one by one.  Each
    block is held by a table or on the stack once, and what the others read stays theirs."""
    hq, hkv, d, bs, pool, shared = 4, 2, 64, 8, 20, 2
    g = torch.Generator().manual_seed(1)
    bt, lens, free, count = i32([[-1] * 6] * 3), i32([0, 0, 0]), i32(list(range(pool))), i32([pool])
    kc, vc = (torch.zeros(pool, bs, hkv, d, dtype=torch.float16, device="cuda") for _ in "kv")
    held = [[], [], []]
    err = pa.new_err_flag()

    def step(changes):
        T = max(1, sum(max(0, c) for c in changes))
        slots, pos = (torch.empty(T, dtype=torch.int64, device="cuda") for _ in range(2))
        pa.update_tables(bt, lens, i32(changes), free, count, slots, pos, i32([0] * 4), bs, err_flag=err)
        assert pa.read_err_flag(err) == 0
        k, v = (torch.randn(T, hkv, d, generator=g).half() for _ in "kv")
        pa.reshape_and_cache(k.cuda(), v.cuda(), kc, vc, slots)
        at = 0
        for s, c in enumerate(changes):
            held[s] = held[s][:max(0, len(held[s]) + c)] if c < 0 else held[s] + list(zip(k[at:at + c], v[at:at + c]))
            at += max(0, c)

    def check(living):
        own = {b for s in living for b in bt[s, :-(-len(held[s]) // bs)].tolist()}
        stack = free[:count.item()].tolist()
        assert len(set(stack)) == len(stack) and not own & set(stack) and len(own) + len(stack) == pool
        q = torch.randn(3, hq, d, generator=g).half()
        out = torch.empty(3, hq, d, device="cuda")
        pa.decode(out, q.cuda(), kc, vc, bt, lens, 0.1)
        for s in range(3):
            assert lens[s].item() == len(held[s])
            if s in living:
                k, v = (torch.stack([r[i] for r in held[s]]).double() for i in (0, 1))
                assert (out[s].cpu().double() - Q.attend(q[s], k, v, 0.1)).abs().max() < 2e-3
    step([20, 0, 0])
    bt[1:, :shared], lens[1:] = bt[0, :shared], shared * bs
    for s in (1, 2):
        held[s] = held[0][:shared * bs]
    step([5, 3, 11])
    check([0, 1, 2])
    living = [0, 1, 2]
    for s in order:
        n, last = len(held[s]), len(living) == 1
        change = [0, 0, 0]
        change[s] = -n if last else shared * bs - n
        step(change)
        if not last:
            lens[s], held[s] = 0, []
        living.remove(s)
        step([1 if x in living else 0 for x in range(3)])
        check(living)
    assert count.item() == pool
