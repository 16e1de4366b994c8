"""GPU tests of decode with shared prefixes: against the 64-bit plain form and
pa.decode on the same tables, over group shapes, prefix lengths and types."""
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


def make(members, shared, private, hq, hkv, d, bs, dtype, seed=0, ramp=0.0):
    """A batch of groups: members[g] sequences share shared[g] tokens, then have
    private[s] of their own.  Whole prefix blocks are shared; the block where a
    prefix ends is copied per member.  Unused slots hold NaN."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    group = [i for i, m in enumerate(members) for _ in range(m)]
    ctx = [shared[i] + private[s] for s, i in enumerate(group)]
    nshared = [x // bs for x in shared]
    need = sum(nshared) + sum(-(-c // bs) - nshared[i] for c, i in zip(ctx, group))
    nb = need + 4
    order = rng.permutation(nb).astype(np.int32)
    width = max(1, max(-(-c // bs) for c in ctx))
    bt = np.full((len(ctx), width), -3, np.int32)
    at, front = 0, []
    for n in nshared:
        front.append(order[at:at + n])
        at += n
    for s, i in enumerate(group):
        n = -(-ctx[s] // bs) - nshared[i]
        bt[s, :nshared[i]] = front[i]
        bt[s, nshared[i]:nshared[i] + n] = order[at:at + n]
        at += n
    bt = torch.from_numpy(bt)
    cache = {}
    for n in "kv":
        c = torch.full((nb * bs, hkv, d), float("nan")).to(Q.DT[dtype])
        first = {}
        for s, i in enumerate(group):
            rows = torch.randn(ctx[s], hkv, d, generator=g)
            if n == "k":
                rows = rows + ramp * torch.arange(ctx[s])[:, None, None] / max(1, max(ctx))
            rows = rows.to(Q.DT[dtype])
            if i in first:
                rows[:shared[i]] = first[i][:shared[i]]
            else:
                first[i] = rows
            c[Q.slots_of(bt, s, 0, ctx[s], bs)] = rows
        cache[n] = c.view(nb, bs, hkv, d)
    return dict(bt=bt, ctx=ctx, k=cache["k"], v=cache["v"], q=torch.randn(len(ctx), hq, d, generator=g).to(Q.DT[dtype]),
                cu=np.concatenate([[0], np.cumsum(members)]).astype(np.int32),
                sh=np.asarray([shared[i] for i in group], np.int32), bs=bs, scale=float(np.float32(d ** -0.5)),
                mg=max(members), ms=max(shared))


def run(b, out="f32", err=None, bounds=True, **kw):
    o = torch.full(b["q"].shape, float("nan"), dtype=Q.DT[out], device="cuda")
    e = err if err is not None else pa.new_err_flag()
    if bounds:
        kw = dict(max_group_size=b["mg"], max_shared_len=b["ms"], max_context_len=max(b["ctx"]), **kw)
    pa.decode_shared(o, b["q"].cuda(), b["k"].cuda(), b["v"].cuda(), b["bt"].cuda(),
                     torch.tensor(b["ctx"], dtype=torch.int32).cuda(), torch.from_numpy(b["cu"]).cuda(),
                     torch.from_numpy(b["sh"]).cuda(), b["scale"], err_flag=e, **kw)
    if err is None:
        assert pa.read_err_flag(e) == 0
    return o


def check(b, out="f32", **kw):
    got = run(b, out, **kw)
    o = got.cpu().double()
    hq, d = b["q"].shape[1:]
    hkv = b["k"].shape[2]
    for s, L in enumerate(b["ctx"]):
        sl = Q.slots_of(b["bt"], s, 0, L, b["bs"])
        k, v = b["k"].view(-1, hkv, d)[sl].double(), b["v"].view(-1, hkv, d)[sl].double()
        ref = Q.attend(b["q"][s], k, v, b["scale"])
        if L == 0:
            assert torch.equal(o[s], ref)
            continue
        vmax = v.abs().amax((0, 2)).repeat_interleave(hq // hkv)[:, None].numpy()
        xs = torch.einsum("hgd,lhd->hgl", b["q"][s].double().abs().view(hkv, hq // hkv, d), k.abs()) * b["scale"]
        tol = Q.tolerance(ref.numpy(), vmax, L, d, xs.reshape(hq, -1).amax(-1)[:, None].numpy(), out)
        if b["q"].dtype == torch.float16 and b["mg"] * hq // hkv > 16:
            # large groups: the weights of a binary16 prefix are rounded once to
            # binary16 (half a step, 2^-11) before they meet V; the sum uses the rounded ones
            tol = tol + 2.0 ** -11 * vmax
        err = (o[s] - ref).abs().numpy()
        assert np.all(np.isfinite(o[s].numpy())), f"sequence {s}"
        assert np.all(err <= tol), f"sequence {s} (length {L}): {np.max(err / tol):.2f} of the bound"
    return got


SHAPES = [   # members, shared, private
    ([4], [64], [1, 5, 30, 37]),
    ([1, 3, 2], [100, 0, 300], [1, 200, 17, 5, 0, 64]),
    ([1, 1, 1], [0, 16, 1000], [1, 1, 1]),
    ([5, 9], [1000, 33], [1, 2, 3, 0, 300, 1, 1, 20, 30, 40, 50, 60, 70, 1]),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d,bs", [(4, 4, 64, 16), (8, 8, 128, 16), (8, 1, 128, 8), (16, 8, 64, 32), (12, 3, 128, 64),
                                         (16, 2, 64, 128), (6, 6, 128, 48), (32, 8, 128, 256)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_shapes(shape, hq, hkv, d, bs, dtype):
    m, s, p = SHAPES[shape]
    check(make(m, s, p, hq, hkv, d, bs, dtype, seed=shape))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d,bs", [(8, 8, 128, 16), (8, 2, 64, 8), (16, 2, 128, 32), (4, 4, 64, 64)])
@pytest.mark.parametrize("n,shared", [(33, 128), (64, 127), (130, 400), (40, 1031)])
def test_large_groups(n, shared, hq, hkv, d, bs, dtype):
    rng = np.random.default_rng(n)
    check(make([n], [shared], rng.integers(0, 50, n).tolist(), hq, hkv, d, bs, dtype, seed=n))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_groups_of_mixed_sizes(dtype):
    members, shared = [70, 1, 40, 3, 128, 17], [256, 90, 0, 700, 129, 1500]
    rng = np.random.default_rng(1)
    check(make(members, shared, rng.integers(0, 40, sum(members)).tolist(), 16, 4, 128, 16, dtype, seed=5))


@pytest.mark.parametrize("members,hq,hkv", [([9, 30, 4], 16, 8), ([2] * 30, 8, 8), ([60], 16, 2)])
def test_enough_private_tokens_for_items_to_be_cut_between_sms(members, hq, hkv):
    rng = np.random.default_rng(4)
    n = sum(members)
    check(make(members, [300] * len(members), rng.integers(0, 1800, n).tolist(), hq, hkv, 64, 16, "bf16", seed=14))


@pytest.mark.parametrize("n", [20, 60, 140])
def test_private_parts_whose_first_tokens_weigh_nothing(n):
    """Keys of -infinity (all queries positive) before the last private token: where
    an item is cut among them, the part before the cut holds nothing and the part
    behind it the token that outweighs the rest."""
    hkv, d, L, own = 8, 64, 320, 504
    b = make([n], [L], [own] * n, hkv, hkv, d, 16, "bf16", seed=17)
    b["q"] = b["q"].abs() + 0.125
    kf = b["k"].view(-1, hkv, d)
    for s in range(n):
        kf[Q.slots_of(b["bt"], s, L, L + own - 1, 16)] = float("-inf")
        kf[Q.slots_of(b["bt"], s, L + own - 1, L + own, 16)] = 1.0
    out = run(b).cpu().double()
    for s in range(n):
        sl = torch.cat([Q.slots_of(b["bt"], s, 0, L, 16), Q.slots_of(b["bt"], s, L + own - 1, L + own, 16)])
        k, v = kf[sl].double(), b["v"].view(-1, hkv, d)[sl].double()
        ref = Q.attend(b["q"][s], k, v, b["scale"])
        xs = torch.einsum("hgd,lhd->hgl", b["q"][s].double().view(hkv, 1, d), k.abs()) * b["scale"]
        tol = Q.tolerance(ref.numpy(), v.abs().amax((0, 2))[:, None].numpy(), L + own, d,
                          xs.reshape(hkv, -1).amax(-1)[:, None].numpy(), "f32")
        assert np.all((out[s] - ref).abs().numpy() <= tol), f"sequence {s}"


@pytest.mark.parametrize("n,hq,hkv", [(3, 8, 8), (50, 8, 2)])
def test_long_prefix(n, hq, hkv):
    rng = np.random.default_rng(2)
    check(make([n], [9000], rng.integers(0, 300, n).tolist(), hq, hkv, 128, 16, "bf16", seed=2))


@pytest.mark.parametrize("out", ["f16", "bf16"])
@pytest.mark.parametrize("n", [4, 60])
def test_half_outputs(n, out):
    check(make([n], [500], list(range(n)), 8, 4, 128, 16, out, seed=3), out)


@pytest.mark.parametrize("n", [4, 60])
def test_logits_that_rise_with_the_position(n):
    """Keys that grow along the prefix move the running reference throughout."""
    b = make([n], [1500], [7] * n, 4, 2, 128, 16, "bf16", seed=4, ramp=40.0)
    b["q"] = b["q"].abs()
    check(b)


@pytest.mark.parametrize("n", [4, 60])
def test_a_scale_of_zero_averages(n):
    b = make([n], [200], [7] * n, 4, 2, 128, 16, "f16", seed=12)
    b["scale"] = 0.0
    check(b)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_many_tokens_of_little_weight_count(dtype):
    """As for one token of weight 1 in a prefix of 20,000 others of 2^-24.6 each."""
    n, hkv, d, L = 20, 1, 64, 20000
    b = make([n], [L], [1] * n, 1, hkv, d, 16, dtype, seed=13)
    used = torch.cat([Q.slots_of(b["bt"], s, 0, L + 1, 16) for s in range(n)])
    kf, vf = b["k"].view(-1, hkv, d), b["v"].view(-1, hkv, d)
    kf[used], vf[used] = 0.0, 1.0
    kf[used, :, 0] = -8.5
    first = Q.slots_of(b["bt"], 0, 0, 1, 16)
    kf[first, :, 0], vf[first] = 8.5, 0.0
    b["q"][:] = 0.0
    b["q"][..., 0] = 1.0
    b["scale"] = 1.0
    got = run(b)[:, 0, 0].cpu().double()
    share = (L * np.exp(-17.0)) / (1 + L * np.exp(-17.0))
    assert (got - share).abs().max() < 1e-3 * share


@pytest.mark.parametrize("size,groups", [(2, 2100), (9, 250)])
def test_more_sequences_and_groups_than_one_launch_takes(size, groups):
    rng = np.random.default_rng(19)
    check(make([size] * groups, rng.integers(16, 40, groups).tolist(), rng.integers(0, 40, size * groups).tolist(), 4, 4, 64,
               16, "bf16", seed=19))


def test_loose_bounds_and_partition_sizes_agree():
    b = make([3, 20, 1], [300, 513, 40], [9] * 24, 8, 4, 64, 16, "f16", seed=6)
    a = check(b)
    for kw in (dict(bounds=False), dict(partition_size=16), dict(partition_size=512)):
        assert (run(b, **kw) - a).abs().max() < 1e-3
        check(b, **kw)


@pytest.mark.parametrize("n,hq,hkv", [(4, 4, 2), (9, 32, 32), (60, 8, 4)])
def test_empty_groups_and_padded_sequences(n, hq, hkv):
    """Empty groups before, between and behind, more groups than sequences, a bound
    above the batch, and padding sequences of no tokens in a group of their own."""
    b = make([n, 2, 3], [300, 0, 16], [7] * n + [5, 9] + [1] * 3, hq, hkv, 128, 16, "bf16", seed=15)
    want = check(b)
    pad = 3
    z = {k: b[k] for k in ("k", "v", "bs", "scale", "ms")}
    z["q"] = torch.cat([b["q"], torch.randn(pad, hq, 128).bfloat16()])
    z["bt"] = torch.cat([b["bt"], torch.full((pad, b["bt"].shape[1]), -1, dtype=torch.int32)])
    z["ctx"] = b["ctx"] + [0] * pad
    z["sh"] = np.concatenate([b["sh"], np.zeros(pad, np.int32)])
    c = b["cu"].tolist()
    z["cu"] = np.asarray([0, 0, c[1], c[1], c[2], c[3], c[3] + pad] + [c[3] + pad] * 80, np.int32)
    z["mg"] = 1000
    got = run(z)
    assert torch.all(got[-pad:] == 0)
    assert (got[:-pad] - want).abs().max() < 1e-3
    check(z)


def test_context_lengths_may_change_between_replays():
    """A captured step whose contexts grow by a token before each replay, as in a serving loop."""
    n, hkv, d, bs = 40, 4, 64, 16
    b = make([n], [200], [50] * n, 8, hkv, d, bs, "f16", seed=16)
    dev = {k: b[k].cuda() for k in ("q", "k", "v", "bt")}
    ctx = torch.tensor([230] * n, dtype=torch.int32).cuda()
    cu, sh = torch.from_numpy(b["cu"]).cuda(), torch.from_numpy(b["sh"]).cuda()
    out = torch.empty(n, 8, d, device="cuda")

    def step():
        ctx.add_(1)
        pa.decode_shared(out, dev["q"], dev["k"], dev["v"], dev["bt"], ctx, cu, sh, b["scale"], max_group_size=n,
                         max_shared_len=200, max_context_len=250)
    graph = pa.StepGraph(step)
    ctx.fill_(230)
    for i in range(1, 20):
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert ctx[0].item() == 230 + i
        eager = run({**b, "ctx": [230 + i] * n})
        assert (got - eager).abs().max() < 1e-3


def test_matches_decode_on_the_same_tables():
    b = make([4, 4, 30], [1000, 64, 256], [int(x) for x in np.random.default_rng(0).integers(1, 99, 38)], 8, 8, 128, 16,
             "bf16", seed=7)
    got = check(b)
    o = torch.empty_like(got)
    pa.decode(o, b["q"].cuda(), b["k"].cuda(), b["v"].cuda(), b["bt"].cuda(),
              torch.tensor(b["ctx"], dtype=torch.int32).cuda(), b["scale"], max_context_len=max(b["ctx"]))
    assert (o - got).abs().max() < 1e-3
    assert torch.equal(run(b), got)          # the same bits again


@pytest.mark.parametrize("n,hq,hkv", [(5, 4, 4), (12, 32, 32), (60, 4, 4)])
def test_members_tables_may_name_other_blocks_for_the_prefix(n, hq, hkv):
    """Only the first member's table is read for the whole prefix blocks."""
    b = make([n], [256], [10] * n, hq, hkv, 64, 16, "f16", seed=8)
    a = run(b)
    b["bt"][1:, :16] = -9
    assert torch.equal(run(b), a)


@pytest.mark.parametrize("n", [4, 60])
def test_bad_block_ids_and_lengths_are_reported(n):
    b = make([n, 2], [320, 64], [20] * (n + 2), 4, 2, 128, 16, "bf16", seed=9)
    clean = run(b)
    bad = {**b, "bt": b["bt"].clone()}
    bad["bt"][0, 3] = b["k"].shape[0]
    err = pa.new_err_flag()
    got = run(bad, err=err)
    assert pa.read_err_flag(err) == pa.FLAG_BAD_BLOCK_ID
    assert torch.equal(got[n:], clean[n:])                       # the other group is untouched
    for change in (dict(sh=np.where(np.arange(n + 2) == 0, -5, b["sh"]).astype(np.int32)),
                   dict(sh=np.where(np.arange(n + 2) == 1, 300, b["sh"]).astype(np.int32)),
                   dict(cu=np.asarray([0, n + 1, n], np.int32)), dict(cu=np.asarray([0, n, n + 1], np.int32)),
                   dict(cu=np.asarray([-1, n, n + 2], np.int32)),
                   dict(cu=np.asarray([0, n, n + 900], np.int32))):
        err = pa.new_err_flag()
        run({**b, **change}, err=err)
        assert pa.read_err_flag(err) & pa.FLAG_BAD_CONTEXT_LEN, change
    err = pa.new_err_flag()                                       # a context beyond its bound: a zero row
    ctx = list(b["ctx"])
    ctx[n + 1] = -1
    o = run({**b, "ctx": ctx}, err=err)
    assert pa.read_err_flag(err) == pa.FLAG_BAD_CONTEXT_LEN
    assert torch.all(o[n + 1] == 0) and torch.equal(o[:n + 1], clean[:n + 1])


@pytest.mark.parametrize("n,hq,hkv", [(4, 4, 2), (60, 8, 8), (9, 32, 32)])
def test_group_bounds_that_no_sequence_meets_are_reported(n, hq, hkv):
    """Bounds that break the rules where every sequence still finds a group that holds it."""
    b = make([n - 2, 2], [320, 320], [20] * n, hq, hkv, 128, 16, "bf16", seed=18)
    b["mg"] = n
    for cu in ([0, n, n + 1], [0, n - 1, n - 2, n], [1, n], [0, n - 1, n - 1, n + 5], [0, n, -1, n]):
        err = pa.new_err_flag()
        run({**b, "cu": np.asarray(cu, np.int32)}, err=err)
        assert pa.read_err_flag(err) & pa.FLAG_BAD_CONTEXT_LEN, cu


def test_nan_in_one_member_stays_with_it():
    b = make([40], [200], [20] * 40, 4, 4, 128, 16, "bf16", seed=10)
    clean = run(b)
    b["q"][3, 2, 5] = float("nan")
    got = run(b)
    assert torch.all(got[3, 2].isnan())
    got[3, 2] = clean[3, 2]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("n", [4, 60])
def test_captured_steps(n):
    """A decode step over shared prefixes, captured, replayed with new queries and a longer context."""
    b = make([n, 2], [320, 64], [20] * (n + 2), 8, 4, 128, 16, "bf16", seed=11)
    dev = {k: b[k].cuda() for k in ("q", "k", "v", "bt")}
    ctx = torch.tensor(b["ctx"], dtype=torch.int32).cuda()
    cu, sh = torch.from_numpy(b["cu"]).cuda(), torch.from_numpy(b["sh"]).cuda()
    key, value = (torch.randn(n + 2, 4, 128, device="cuda").bfloat16() for _ in range(2))
    slots = torch.stack([Q.slots_of(b["bt"], s, L - 1, L, 16)[0] for s, L in enumerate(b["ctx"])]).cuda()
    out = torch.empty(n + 2, 8, 128, device="cuda")

    def step():
        pa.reshape_and_cache(key, value, dev["k"], dev["v"], slots)
        pa.decode_shared(out, dev["q"], dev["k"], dev["v"], dev["bt"], ctx, cu, sh, b["scale"], max_group_size=n,
                         max_shared_len=320, max_context_len=max(b["ctx"]))
    graph = pa.StepGraph(step)
    for _ in range(3):
        dev["q"].normal_()
        key.normal_()
        value.normal_()
        step()
        want = out.clone()
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_back_to_back_calls_reuse_a_workspace():
    """Calls of different batches behind one another on one stream and workspace."""
    bs = [make([n], [s], [5] * n, 8, 2, 128, 16, "f16", seed=n) for n, s in ((60, 700), (3, 2000), (40, 90))]
    want = [run(b) for b in bs]
    ws = pa.DecodeWorkspace("cuda")
    ws.get(64 << 20)
    dev = [{k: b[k].cuda() for k in ("q", "k", "v", "bt")} | dict(
        ctx=torch.tensor(b["ctx"], dtype=torch.int32).cuda(), cu=torch.from_numpy(b["cu"]).cuda(),
        sh=torch.from_numpy(b["sh"]).cuda(), out=torch.empty(b["q"].shape, device="cuda")) for b in bs]
    torch.cuda.synchronize()
    for _ in range(20):
        for b, t in zip(bs, dev):
            pa.decode_shared(t["out"], t["q"], t["k"], t["v"], t["bt"], t["ctx"], t["cu"], t["sh"], b["scale"],
                             max_group_size=b["mg"], max_shared_len=b["ms"], max_context_len=max(b["ctx"]), workspace=ws)
    torch.cuda.synchronize()
    for t, w in zip(dev, want):
        assert torch.equal(t["out"], w)


def test_refusals():
    b = make([2], [64], [5, 6], 4, 4, 64, 16, "f16")
    t = dict(out=b["q"].cuda(), query=b["q"].cuda(), k_cache=b["k"].cuda(), v_cache=b["v"].cuda(),
             block_tables=b["bt"].cuda(), context_lens=torch.tensor(b["ctx"], dtype=torch.int32).cuda(),
             cu_groups=torch.from_numpy(b["cu"]).cuda(), shared_lens=torch.from_numpy(b["sh"]).cuda(), scale=0.1)
    pa.decode_shared(**t)
    for name, bad in [("cu_groups", t["cu_groups"].long()), ("cu_groups", t["cu_groups"].cpu()),
                      ("shared_lens", t["shared_lens"][:1]), ("query", t["query"].bfloat16()),
                      ("k_cache", t["k_cache"][:, :, :, :32].contiguous()), ("context_lens", t["context_lens"].float()),
                      ("max_shared_len", 4096), ("partition_size", 8), ("err_flag", torch.zeros(1, dtype=torch.int32))]:
        with pytest.raises((ValueError, TypeError)):
            pa.decode_shared(**{**t, name: bad})
    with pytest.raises(pa.PagedAttentionError):          # two sequences in one group of at most one
        pa.decode_shared(**t, max_group_size=1)
    wide = {**t, "block_tables": b["bt"].repeat(1, 300).cuda()}      # bounds under which the call needs a workspace
    with pytest.raises(ValueError):
        pa.decode_shared(**wide, workspace=torch.empty(1 << 28, dtype=torch.uint8))
    with pytest.raises(pa.PagedAttentionError):
        pa.decode_shared(**wide, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
