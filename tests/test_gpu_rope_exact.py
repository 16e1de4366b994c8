"""GPU tests of what the rotation with the cache write leaves as it is, and of its angles and bytes where
ordinary sizes cannot show them: far positions, high frequencies, calls of few and of many tokens."""
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_140_gb300 as pa

from test_gpu_rope import KINDS, caches, inputs, rope_write

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_140_gb300 import _build
    _build.build()


# ------------------------------------------------------ few and many tokens

@pytest.mark.parametrize("interleaved,rot,d", [(False, 64, 64), (True, 32, 128), (False, 128, 128)])
@pytest.mark.parametrize("kind", KINDS + ["half"])
def test_many_normalised_tokens_make_the_bytes_of_few(kind, interleaved, rot, d):
    """One call of 163 tokens of 120 rows, and calls of 20 and less, which take another form of the kernel: a
    token's bytes do not depend on how many others come with it, norms of queries and keys included."""
    T, hq, hkv, bs, nb = 163, 64, 28, 16, 12
    _, dev, pos = inputs(T, hq, hkv, d, "bf16", seed=5)
    g = torch.Generator().manual_seed(2)
    qw, kw = ((1 + 0.3 * torch.randn(d, generator=g)).bfloat16().cuda() for _ in "qk")
    slots = torch.randperm(nb * bs, generator=torch.Generator().manual_seed(0))[:T].cuda()
    pos = pos.cuda()
    freq, _ = pa.rope_frequencies(rot)
    made = []
    for step in (T, 20):
        if kind == "half":
            c = {n: torch.full((nb, bs, hkv, d), 3.0, dtype=torch.bfloat16, device="cuda") for n in "kv"}
        else:
            c = caches(kind, nb, bs, hkv, d)
        out = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
        for t in range(0, T, step):
            part, a, s = [x[t:t + step] for x in dev], out[t:t + step], slots[t:t + step]
            kws = dict(interleaved=interleaved, q_weight=qw, k_weight=kw)
            if kind == "half":
                pa.rope_and_cache(a, *part, c["k"], c["v"], s, pos[t:t + step], freq, **kws)
            else:
                rope_write(kind, a, part, c, s, pos[t:t + step], freq, **kws)
        made.append([out.view(torch.uint8)] + [x.view(torch.uint8) for x in c.values()])
    for a, b in zip(*made):
        assert torch.equal(a, b)
