"""GPU tests of decode_shared where the prefixes get a pass of their own (batches whose
repeated reads would pass 8 MB): every way they are computed, long private parts, and
inputs written by kernels right before the call."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_140_gb300 as pa

import test_gpu_partitions as P
import test_gpu_shared as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_140_gb300 import _build
    _build.build()


def own_pass(members, shared, hkv, d):
    return (sum(members) - len(members)) * max(shared) * hkv * d * 4 > 8 << 20


# A binary16 prefix of more than 8 query rows per KV head has its weights rounded once to
# binary16 (half a step, 2^-11) before they meet V; the sum uses the rounded ones.
def case(members, shared, private, hq, hkv, d, bs, dtype, seed, **kw):
    assert own_pass(members, shared, hkv, d)
    rows = max(members) * hq // hkv
    width = -(-(max(shared) + max(private)) // bs)
    P.shared_case(members, shared, private, width, hq, hkv, d, bs, dtype, seed,
                  extra=2.0 ** -11 if dtype == "f16" and rows > 8 and bs <= 128 else 0.0, max_group_size=max(members),
                  max_shared_len=max(shared), **kw)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,hq,hkv", [(9, 8, 8), (12, 8, 8), (16, 8, 8), (5, 16, 8), (3, 32, 8), (4, 32, 8), (2, 64, 8)])
@pytest.mark.parametrize("d,bs", [(128, 16), (64, 128)])
def test_nine_to_sixteen_rows(n, hq, hkv, d, bs, dtype):
    rng = np.random.default_rng(n)
    case([n], [-(-(3 << 20) // ((n - 1) * hkv * d) // bs) * bs + bs], rng.integers(1, 90, n).tolist(), hq, hkv, d, bs, dtype, 50)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bs", [8, 32, 64, 128])
@pytest.mark.parametrize("members,hq,hkv,d", [([40], 8, 8, 128), ([70, 20], 16, 4, 64), ([150], 8, 4, 128)])
def test_block_sizes_on_the_tensor_cores(members, hq, hkv, d, bs, dtype):
    rng = np.random.default_rng(bs)
    shared = [896 + 128 * i for i in range(len(members))]
    case(members, shared, rng.integers(1, 300, sum(members)).tolist(), hq, hkv, d, bs, dtype, 51)
    # a prefix that ends inside a block, in copies of it
    b = S.make(members, [s + 5 for s in shared], rng.integers(0, 40, sum(members)).tolist(), hq, hkv, d, bs, dtype, seed=52)
    S.check(b)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bs", [48, 80, 256])
@pytest.mark.parametrize("members,hq,hkv", [([7] * 5, 8, 8), ([30], 16, 4), ([3, 9, 20], 4, 1)])
def test_block_sizes_that_the_tensor_core_kernel_does_not_take(members, hq, hkv, bs, dtype):
    rng = np.random.default_rng(bs)
    shared = [bs * (3840 // bs) - i * bs for i in range(len(members))]
    case(members, shared, rng.integers(1, 300, sum(members)).tolist(), hq, hkv, 128, bs, dtype, 53)


@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("members,hq,hkv", [([4] * 12, 8, 8), ([24, 3, 1], 32, 8), ([90], 16, 4)])
def test_long_private_parts(members, hq, hkv, bs):
    rng = np.random.default_rng(7)
    private = rng.integers(1, 3000, sum(members)).tolist()
    private[0], private[-1] = 3000, 0
    case(members, [1024] * len(members), private, hq, hkv, 64, bs, "bf16", 54)


@pytest.mark.parametrize("members", [[2] * 40, [30], [150]])
def test_inputs_written_right_before_the_call(members):
    """Caches, tables, lengths and queries are overwritten by kernels on the stream, and the
    call follows at once; two sets of inputs in turn, nothing waited for in between."""
    hq, hkv, d, bs = 8, 4, 128, 16
    n = sum(members)
    assert own_pass(members, [640], hkv, d)
    rng = np.random.default_rng(n)
    sets = []
    for seed in (60, 61):
        b = S.make(members, [640 if seed == 60 else 512] * len(members), rng.integers(1, 400, n).tolist(), hq, hkv, d, bs, "bf16",
                   seed=seed)
        sets.append((b, S.check(b)))
    nb, width = max(b["k"].shape[0] for b, _ in sets), max(b["bt"].shape[1] for b, _ in sets)
    dev = []
    for b, want in sets:
        bt = torch.zeros(n, width, dtype=torch.int32)
        bt[:, :b["bt"].shape[1]] = b["bt"]
        full = [torch.cat([b[c], b[c][:1].expand(nb - b[c].shape[0], -1, -1, -1)]) for c in "kv"]
        dev.append([t.cuda().contiguous() for t in (b["q"], *full, bt, torch.tensor(b["ctx"], dtype=torch.int32),
                                                    torch.from_numpy(b["sh"]))])
    live = [torch.empty_like(t) for t in dev[0]]
    cu = torch.from_numpy(sets[0][0]["cu"]).cuda()
    kw = dict(max_group_size=max(members), max_shared_len=640, max_context_len=max(max(b["ctx"]) for b, _ in sets))
    outs = [torch.empty(n, hq, d, device="cuda") for _ in range(24)]

    def call(i, order):
        for j in order:
            live[j].copy_(dev[i % 2][j])
        q, k, v, bt, ctx, sh = live
        pa.decode_shared(outs[i], q, k, v, bt, ctx, cu, sh, sets[0][0]["scale"], **kw)
    for i in range(len(outs)):
        # another input is the one written last each time
        call(i, [(j + i // 2) % 6 for j in range(6)])
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, outs[i % 2]) and (o - sets[i % 2][1]).abs().max() < 1e-3, i


def test_calls_on_several_streams_at_once():
    """Prefixes of one query tile, of pairs, of a padded list and a prefill, all of which hold
    tensor memory, on four streams."""
    work = []
    for members, pad in (([12] * 10, 0), ([150], 0), ([30, 20], 60)):
        hq, hkv, d, bs = 8, 4, 128, 16
        assert own_pass(members, [900], hkv, d)
        b = S.make(members, [900] * len(members), [30] * sum(members), hq, hkv, d, bs, "bf16", seed=70)
        cu = np.concatenate([b["cu"], np.full(pad, b["cu"][-1], np.int32)])
        t = [x.cuda() for x in (b["q"], b["k"], b["v"], b["bt"], torch.tensor(b["ctx"], dtype=torch.int32), torch.from_numpy(cu),
                                torch.from_numpy(b["sh"]))]

        def call(out, t=t, b=b):
            pa.decode_shared(out, *t, b["scale"], max_group_size=b["mg"], max_shared_len=900, max_context_len=930)
        work.append((call, torch.empty(b["q"].shape, device="cuda")))
    q = torch.randn(600, 8, 128, device="cuda").bfloat16()
    cache = torch.randn(2, 80, 16, 4, 128, device="cuda").bfloat16()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")       # noqa: E731
    table, ctx, cu_q = torch.arange(75, device="cuda").int()[None].contiguous(), i32([1200]), i32([0, 600])

    def prefill(out):
        pa.prefill(out, q, cache[0], cache[1], table, ctx, cu_q, 128 ** -0.5, max_q_len=600)
    work.append((prefill, torch.empty(q.shape, device="cuda")))
    want = []
    for call, out in work:
        call(out)
        want.append(out.clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    wrong = torch.zeros(len(work), dtype=torch.int32, device="cuda")
    for _ in range(40):
        for i, ((call, out), s) in enumerate(zip(work, streams)):
            with torch.cuda.stream(s):
                call(out)
                wrong[i] += (out != want[i]).any()
    torch.cuda.synchronize()
    assert wrong.tolist() == [0] * len(work)
