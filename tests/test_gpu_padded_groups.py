"""GPU tests of decode_shared with lists of groups that are padded with empty ones,
as the fixed list of a captured step is."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_140_gb300 as pa

import test_gpu_shared as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_140_gb300 import _build
    _build.build()


def pad(cu, entries, rng):
    """cu with empty groups put in at random places, up to ``entries`` groups."""
    out = list(cu)
    while len(out) - 1 < entries:
        i = int(rng.integers(0, len(out)))
        out.insert(i, out[i])
    return np.asarray(out, np.int32)


def batch(members, shared, hq, hkv, d, dtype, seed, hi=40):
    rng = np.random.default_rng(seed)
    return S.make(members, shared, rng.integers(1, hi, sum(members)).tolist(), hq, hkv, d, 16, dtype, seed=seed)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("members,shared,hq,hkv,d", [
    ([70], [500], 8, 2, 128),                                    # one query tile or a pair, one group
    ([130], [700], 8, 2, 64),
    ([40, 40, 30], [300, 1000, 17], 16, 2, 64),
    # many more groups with a prefix than the list is planned for: CTAs take several units
    ([60] + [3] * 30, [400] + [160 + 16 * i for i in range(30)], 8, 2, 128),
    ([100] + [2] * 20 + [1] * 9, [272] + [128, 1100] * 10 + [0, 500, 64] * 3, 16, 4, 64)])
def test_padded_lists(members, shared, hq, hkv, d, dtype):
    b = batch(members, shared, hq, hkv, d, dtype, 31)
    rng = np.random.default_rng(5)
    n = sum(members)
    first = None
    for entries in (n, n + 44, 700):
        z = {**b, "cu": pad(b["cu"], entries, rng)}
        got = S.check(z)
        assert torch.equal(S.run(z), got)
        if first is not None:
            assert torch.equal(got, first)                       # where the empty groups stand does not matter
        first = got


def test_small_groups_in_padded_lists():
    """The split kernel's prefixes, and batches that take one pass."""
    for members, shared in (([2] * 40, [900] * 40), ([4], [64]), ([1] * 30, [50] * 30)):
        b = batch(members, shared, 4, 4, 128, "bf16", 32)
        S.check({**b, "cu": pad(b["cu"], sum(members) + 9, np.random.default_rng(1))})


def test_a_captured_list_may_hold_other_groups_at_each_replay():
    """One graph, a list of as many entries as sequences; the groups and their prefixes change between replays."""
    n, hq, hkv, d, bs = 96, 8, 2, 128, 16
    batches = [batch(m, s, hq, hkv, d, "bf16", 40 + i) for i, (m, s) in enumerate((
        ([96], [800]), ([48, 48], [800, 320]), ([90] + [1] * 6, [640] + [0] * 6), ([4] * 24, [96 + 16 * i for i in range(24)])))]
    nb, width = max(b["k"].shape[0] for b in batches), max(b["bt"].shape[1] for b in batches)
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")   # noqa: E731
    q, out = z(n, hq, d, t=torch.bfloat16), z(n, hq, d, t=torch.float32)
    kc, vc = z(nb, bs, hkv, d, t=torch.bfloat16), z(nb, bs, hkv, d, t=torch.bfloat16)
    bt, ctx, cu, sh, err = z(n, width), z(n), z(n + 1), z(n), pa.new_err_flag()

    def load(b):
        q.copy_(b["q"])
        kc[:b["k"].shape[0]], vc[:b["v"].shape[0]] = b["k"].cuda(), b["v"].cuda()
        bt[:, :b["bt"].shape[1]] = b["bt"].cuda()
        ctx.copy_(torch.tensor(b["ctx"], dtype=torch.int32))
        cu.copy_(torch.from_numpy(pad(b["cu"], n, np.random.default_rng(2))))
        sh.copy_(torch.from_numpy(b["sh"]))

    def step():
        pa.decode_shared(out, q, kc, vc, bt, ctx, cu, sh, batches[0]["scale"], max_group_size=n, max_shared_len=800,
                         max_context_len=840, err_flag=err)
    load(batches[0])
    graph = pa.StepGraph(step)
    for b in batches + batches[::-1]:
        load(b)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert pa.read_err_flag(err) == 0
        want = S.check(b)
        assert (got - want).abs().max() < 1e-3


@pytest.mark.parametrize("n", [40, 130])
def test_what_breaks_the_rules_in_a_padded_list_is_reported(n):
    b = batch([n - 12, 6, 6], [320, 0, 64], 8, 2, 128, "bf16", 33)
    cu = pad(b["cu"], n + 20, np.random.default_rng(3))
    clean = S.run({**b, "cu": cu})

    def flags(**change):
        err = pa.new_err_flag()
        S.run({**b, "cu": cu, **change}, err=err)
        return pa.read_err_flag(err)
    assert flags() == 0
    s = b["sh"].copy()
    s[n - 9] = 1                                        # one member of the group without a prefix
    assert flags(sh=s) == pa.FLAG_BAD_CONTEXT_LEN
    s = b["sh"].copy()
    s[n - 1] = 48                                       # one of the last group
    assert flags(sh=s) == pa.FLAG_BAD_CONTEXT_LEN
    for at, to in ((0, 1), (len(cu) - 1, n + 1), (len(cu) - 1, n - 1), (len(cu) // 2, -3), (len(cu) // 2, n + 7)):
        c = cu.copy()
        c[at] = to
        assert flags(cu=c) & pa.FLAG_BAD_CONTEXT_LEN, (at, to)
    err = pa.new_err_flag()
    bad = b["bt"].clone()
    bad[0, 3] = b["k"].shape[0]
    got = S.run({**b, "cu": cu, "bt": bad}, err=err)
    assert pa.read_err_flag(err) == pa.FLAG_BAD_BLOCK_ID
    assert torch.equal(got[n - 12:], clean[n - 12:])     # the other groups are untouched
