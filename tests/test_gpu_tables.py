"""GPU tests of the block tables' update against a stack on the host, and a run of whole
steps: tables, rotation with the cache write, attention."""
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


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Pool:
    """Tables, lengths and stack on the GPU and their copy on the host."""

    def __init__(self, lens, bs, width, pool, seed=0):
        g = np.random.default_rng(seed)
        order = g.permutation(pool).tolist()
        self.bs, self.lens = bs, list(lens)
        self.bt = [[-5] * width for _ in lens]
        at = 0
        for s, n in enumerate(lens):
            for b in range(-(-n // bs)):
                self.bt[s][b] = order[at]
                at += 1
        self.free = order[at:] + [-9] * at
        self.count = pool - at
        self.d = {"bt": i32(self.bt).view(len(lens), width), "lens": i32(self.lens), "free": i32(self.free),
                  "count": i32([self.count])}

    def step(self, changes, room, inplace=True, err=None):
        d = self.d
        slots = torch.full((room,), 77, dtype=torch.int64, device="cuda")
        pos, cu = slots.clone(), i32([99] * (len(self.lens) + 1))
        kw = {} if inplace else dict(out_lens=torch.empty_like(d["lens"]), out_free_count=torch.empty_like(d["count"]))
        e = err if err is not None else pa.new_err_flag()
        pa.update_tables(d["bt"], d["lens"], i32(changes), d["free"], d["count"], slots, pos, cu, self.bs, err_flag=e, **kw)
        if not inplace:
            assert d["lens"].tolist() == self.lens and d["count"].tolist() == [self.count]
            d["lens"], d["count"] = kw["out_lens"], kw["out_free_count"]
        if err is None:
            assert pa.read_err_flag(e) == 0
            self.bt, self.lens, self.free, self.count, *rest = S.update(self.bt, self.lens, changes, self.free, self.count,
                                                                       self.bs, room)
            self.same()
            assert [cu.tolist(), slots.tolist(), pos.tolist()] == list(rest)
        return slots, pos, cu

    def same(self):
        d = self.d
        assert d["bt"].tolist() == self.bt and d["lens"].tolist() == self.lens
        assert d["free"].tolist() == self.free and d["count"].tolist() == [self.count]


@pytest.mark.parametrize("bs", [1, 8, 16, 48])
def test_steps(bs):
    p = Pool([0, 1, bs, bs + 1, 5 * bs - 1, 100, 0], bs, 400 // bs + 2, 7 * (400 // bs + 2))
    p.step([1] * 7, 7)
    p.step([bs, 0, -1, 3 * bs + 1, -200, -3, 0], 4 * bs + 30)
    p.step([-bs, 5, 1, -3 * bs - 1, 17, 3, 2], 40, inplace=False)
    p.step([-2 ** 31, -2 ** 31 + 1, -1000, 0, 1, 0, 0], 1)
    p.step([0] * 7, 0)


def test_undoing_a_step_leaves_the_stack_as_it_was():
    p = Pool([10, 20, 30], 8, 20, 60, seed=3)
    free, count = list(p.free), p.count
    p.step([30, 9, 50], 89)
    p.step([-30, -9, -50], 0)
    assert p.free[:count] == free[:count] and p.count == count


@pytest.mark.parametrize("B,new,room", [(1, 3000, 5000), (1, 1, 1), (700, 40, 14500), (3000, 4, 8000), (8192, 1, 8200)])
def test_many(B, new, room):
    g = np.random.default_rng(B)
    lens = g.integers(0, 200, B).tolist()
    p = Pool(lens, 16, (200 + 3 * new) // 16 + 2, B * 16 + 2 * B * (new // 16 + 2), seed=1)
    for _ in range(2):
        kinds = g.random(B)
        ch = np.where(kinds < 0.2, -g.integers(0, 60, B), g.integers(0, new + 1, B))
        while np.maximum(ch, 0).sum() > room:
            ch //= 2
        p.step(ch.tolist(), room, inplace=bool(B % 2))


def test_no_sequences():
    p = Pool([], 16, 3, 4)
    p.d["bt"] = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    slots, pos, cu = p.step([], 3, err=pa.new_err_flag())
    assert slots.tolist() == [-1] * 3 and pos.tolist() == [0] * 3 and cu.tolist() == [0]


@pytest.mark.parametrize("changes,room,flag", [
    ([40, 100], 200, "blocks"), ([600, 0], 700, "len"), ([10, 10], 19, "len"), ([2 ** 31 - 1, 2 ** 31 - 1], 50, "len")])
def test_what_does_not_fit_changes_nothing(changes, room, flag):
    p = Pool([10, 20], 8, 30, 12)      # 5 blocks held, 7 free
    err = pa.new_err_flag()
    slots, pos, cu = p.step(changes, room, err=err)
    assert pa.read_err_flag(err) == (pa.FLAG_NO_BLOCKS if flag == "blocks" else pa.FLAG_BAD_CONTEXT_LEN)
    p.same()
    assert torch.all(slots == -1) and torch.all(pos == 0) and torch.all(cu == 0)
    p.step([6, 44], 50)                # to 16 and 64 tokens: 2 and 8 blocks, 5 of the 7 that are free
    assert p.count == 2
    p.step([16, 0], 16)                # exactly what is left
    assert p.count == 0


def test_bad_counts_lengths_and_ids():
    err = pa.new_err_flag()
    for count in (-1, 13):
        p = Pool([10, 20], 8, 30, 12)
        p.d["count"].fill_(count)
        p.step([1, 1], 2, err=err)
        assert pa.read_err_flag(err) == pa.FLAG_NO_BLOCKS and p.d["count"].tolist() == [count]
    p = Pool([10, 20], 8, 30, 12)
    p.d["lens"][0] = -3
    p.step([1, 1], 2, err=err)
    assert pa.read_err_flag(err) == pa.FLAG_BAD_CONTEXT_LEN and p.d["lens"].tolist() == [-3, 20]
    # a full stack does not take blocks that it cannot hold
    p = Pool([10, 20], 8, 30, 12)
    p.d["count"].fill_(11)
    p.step([-10, 0], 2, err=err)
    assert pa.read_err_flag(err) == pa.FLAG_NO_BLOCKS
    # an id out of range in the last block, and one on the stack: their tokens have no slot
    p = Pool([10, 20], 8, 30, 12)
    p.d["bt"][0, 1] = 12
    p.d["free"][p.count - 1] = -1
    slots, _, _ = p.step([8, 3], 11, err=err)
    assert pa.read_err_flag(err) == pa.FLAG_BAD_BLOCK_ID
    assert torch.all(slots[:8] == -1) and torch.all(slots[8:] >= 0)


def test_another_stream_and_a_captured_step():
    p = Pool([3, 40, 0], 8, 40, 100)
    changes = i32([0, 0, 0])
    slots = torch.empty(64, dtype=torch.int64, device="cuda")
    pos, cu = torch.empty_like(slots), i32([0] * 4)
    d = p.d
    graph = pa.StepGraph(lambda: pa.update_tables(d["bt"], d["lens"], changes, d["free"], d["count"], slots, pos, cu, 8))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for ch in ([1, 1, 1], [9, -4, 30], [-100, 0, -7], [50, 1, 0]):
            changes.copy_(i32(ch))
            graph.replay()
            p.bt, p.lens, p.free, p.count, c, s, q = S.update(p.bt, p.lens, ch, p.free, p.count, 8, 64)
            p.same()
            assert [cu.tolist(), slots.tolist(), pos.tolist()] == [c, s, q]


# ------------------------------------------------- whole steps together

@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("kind", ["half", "int8", "int4"])
def test_serving_steps(kind, captured):
    """Prompts and then decode steps with drafted tokens taken back and a sequence ended and replaced: tables from the
    changes, queries and keys normalised and turned, rows written, attention; each output against 64 bits over the
    rows that the sequences then hold."""
    hq, hkv, d, bs, B, width, pool_blocks = 8, 2, 128, 16, 3, 12, 24
    g = torch.Generator().manual_seed(1)
    dt = torch.bfloat16
    freq, factor = pa.rope_frequencies(64, scaling="parts", scale=4.0)
    kw_ = (1 + 0.2 * torch.randn(d, generator=g)).to(dt)
    qw_ = (1 + 0.2 * torch.randn(d, generator=g)).to(dt)
    qw, kw = qw_.cuda(), kw_.cuda()
    nb = pool_blocks
    if kind == "half":
        c = {n: torch.zeros(nb, bs, hkv, d, dtype=dt, device="cuda") for n in "kv"}
    elif kind == "int8":
        c = {n: torch.zeros(nb, bs, hkv, d, dtype=torch.int8, device="cuda") for n in "kv"}
        c.update({n + "s": torch.zeros(nb, bs, hkv, device="cuda") for n in "kv"})
    else:
        c = {n: t.cuda() for n, t in S.empty_cache4(nb, bs, hkv, d, 0, 0.0).items()}
    bt, lens = torch.full((B, width), -1, dtype=torch.int32, device="cuda"), i32([0] * B)
    free, count = i32(list(range(nb))), i32([nb])
    changes, cu = i32([0] * B), i32([0] * (B + 1))
    scales = {} if kind == "half" else dict(k_scales=c["ks"], v_scales=c["vs"])

    def buffers(T):
        return dict(qkv=torch.zeros(T, (hq + 2 * hkv) * d, dtype=dt, device="cuda"),
                    q=torch.zeros(T, hq, d, dtype=dt, device="cuda"), slots=torch.zeros(T, dtype=torch.int64, device="cuda"),
                    pos=torch.zeros(T, dtype=torch.int64, device="cuda"), out=torch.zeros(B, hq, d, device="cuda"))

    def front(b):
        pa.update_tables(bt, lens, changes, free, count, b["slots"], b["pos"], cu, bs, err_flag=err)
        T = b["slots"].numel()
        q, k, v = b["qkv"].split([hq * d, hkv * d, hkv * d], 1)
        pa.rope_and_cache(b["q"], q.view(T, hq, d), k.view(T, hkv, d), v.view(T, hkv, d), c["k"], c["v"], b["slots"], b["pos"],
                          freq, factor=factor, q_weight=qw, k_weight=kw, err_flag=err, **scales)

    def attend(b):
        q = b["q"][:B]
        if kind == "half":
            pa.decode(b["out"], q, c["k"], c["v"], bt, lens, 0.09, err_flag=err)
        elif kind == "int8":
            pa.quant_decode(b["out"], q, c["k"], c["v"], c["ks"], c["vs"], bt, lens, 0.09, err_flag=err)
        else:
            pa.int4_decode(b["out"], q, c["k"], c["v"], c["ks"], c["vs"], bt, lens, 0.09, err_flag=err)

    err = pa.new_err_flag()
    chunk, one = buffers(90), buffers(B)

    def step():
        front(one)
        attend(one)
    graph = pa.StepGraph(step) if captured else None
    held = [[] for _ in range(B)]                 # each sequence's (key row, value row), 64 bits

    def as_read(rows):
        """Rows as the cache gives them back."""
        x = torch.stack(rows)
        if kind == "half":
            return x.to(dt).double()
        if kind == "int8":
            codes, sc = Q.quantise(x.float(), "int8")
            return Q.values(codes, "int8") * sc.double()[..., None]
        return S.values4(*S.quantise4(x.float()))

    # prompts, then ordinary steps; -k takes tokens back, a large one ends the sequence
    plan = [[30, 1, 50], [1, 1, 1], [1, 1, 1], [-2, 0, -3], [1, 1, 1], [-1000, 1, 1], [20, 0, 0], [1, 1, 1]]
    for ch in plan:
        gained = sum(max(0, x) for x in ch)
        b = one if ch == [1, 1, 1] else chunk
        qkv = torch.randn(b["slots"].numel(), (hq + 2 * hkv) * d, generator=g).to(dt)
        b["qkv"].copy_(qkv)
        changes.copy_(i32(ch))
        if b is one and captured:
            graph.replay()
        else:
            front(b)
            if b is one:
                attend(b)
        assert pa.read_err_flag(err) == 0
        at, positions = 0, []
        for s, x in enumerate(ch):
            if x < 0:
                held[s] = held[s][:max(0, len(held[s]) + x)]
            for _ in range(max(0, x)):
                positions.append(len(held[s]))
                k, v = qkv[at, hq * d:].split(hkv * d)
                held[s].append((S.turn(k.view(1, hkv, d), torch.tensor([len(held[s])]), freq.cpu(), False, factor, kw_)[0],
                                v.view(hkv, d).double()))
                at += 1
        assert b["pos"].tolist()[:gained] == positions and lens.tolist() == [len(h) for h in held]
        if b is not one:
            continue
        q = S.turn(qkv[:, :hq * d].view(B, hq, d), torch.tensor(positions), freq.cpu(), False, factor, qw_).to(dt)
        for s in range(B):
            k, v = as_read([r[0] for r in held[s]]), as_read([r[1] for r in held[s]])
            ref = Q.attend(q[s], k, v, 0.09)
            # A key's or query's 32-bit error may round an element to the next value of its type or code.  A bf16
            # query element off by one step (2^-8 of itself) moves a logit by 0.09 2^-8 |q k|, one element at a
            # time; norms keep |q| and |k| below 11 (128 elements of about 1, weights and factor of 1.3), so by
            # less than 0.09 2^-8 11 11 / 11 = 0.004, and outputs by that of |v| < 5.  A key code off by one step
            # weighs a fifteenth (int4) of a group's range of 7: 0.09 x 0.5 x |q element| < 3: 0.13 of a logit of one token
            # among 21 or more, 0.13 / 21 x 2 x 5 = 0.06 at the worst.
            assert (b["out"][s].cpu().double() - ref).abs().max() < (0.02 if kind == "half" else 0.06), (ch, s)
