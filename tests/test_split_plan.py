"""The automatic partition length of the split decode kernels, gone over on the
host: a partition's block ids sit in the 32 lanes of one warp, so no partition
may reach into a 33rd block, wherever in a block it starts."""
import ctypes
import math
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHIM = r"""
#include "pa_split_plan.h"
extern "C" int partition(int64_t lists, int64_t boxes, int64_t len, int bs, int slot, int requested) {
    return pa::split_partition(lists, boxes, len, bs, slot, requested);
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "shim.cpp").write_text(SHIM)
    so = d / "shim.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "paged_kv_cache_140_gb300", "csrc"), str(d / "shim.cpp"), "-o", str(so)], check=True)
    fn = ctypes.CDLL(str(so)).partition
    fn.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 3
    return fn


def most_blocks(P, bs):
    """Blocks that a partition of P tokens touches at most, at starts 0, P, 2 P, ..."""
    starts = {k * P % bs for k in range(bs // math.gcd(P, bs))}
    return max((s + P + bs - 1) // bs for s in starts)


BLOCK_SIZES = [8] + list(range(16, 257, 16))
# (boxes, slot): heads per box 8, 4, 2, 1 with 16-bit (8 tiles of 16 tokens) and 8-bit caches (16 tiles)
SLOTS = [(1, 16 * (t >> lg)) for t in (8, 16) for lg in (3, 2, 1, 0)]


@pytest.mark.parametrize("bs", BLOCK_SIZES)
def test_no_automatic_partition_reaches_a_33rd_block(rule, bs):
    cap = 32 * bs
    for boxes, slot in SLOTS + [(5, 16), (5, 32)]:
        # lengths beyond one partition, with as many lists as make an SM's share each whole number of slots
        for slots in range(1, cap // slot + 3):
            for length in (cap + 1, 2 * cap - 32, 40 * cap):
                lists = math.ceil((slots + 0.5) * slot * 152 / (0.4 * length))
                P = rule(lists, boxes, length, bs, slot, 0)
                assert P % 16 == 0 and 16 <= P <= cap and most_blocks(P, bs) <= 32, (boxes, slot, length, lists, P)
        # and lengths that one partition holds (of which private parts may turn out longer)
        for length in range(0, cap + 1):
            P = rule(1 << 20, boxes, length, bs, slot, 0)
            assert P % 16 == 0 and 16 <= P <= cap and most_blocks(P, bs) <= 32, (boxes, slot, length, P)
            if boxes == 1:
                assert P >= length                       # still one partition


@pytest.mark.parametrize("bs", BLOCK_SIZES)
def test_requested_partitions_are_taken_exactly_where_32_blocks_hold_them(rule, bs):
    for P in range(1, 34 * bs, 1 if bs < 64 else 16):
        ok = P % 16 == 0 and most_blocks(P, bs) <= 32 and P <= 32 * bs
        got = rule(100, 1, 100000, bs, 16, P)
        assert got in (0, P)
        if got:
            assert ok, P
        elif ok:                                          # what the rule refuses beyond need: none but long unaligned ones
            assert P % bs != 0 and P > 31 * bs + 16, P


def test_empty_groups_do_not_change_the_plan():
    """256 sequences over one prompt: the workspace (the partial results planned for) of a
    list of groups that is padded is that of the tight one."""
    from paged_kv_cache_140_gb300 import _build, _lib
    _build.build()
    size = _lib.load().pa_decode_shared_workspace_size
    for hkv, d, bs, shared in ((8, 128, 16, 8192), (32, 64, 32, 2000), (4, 64, 128, 4000)):
        tight = size(256, 1, 256, 32, hkv, d, bs, shared + 512, shared, 0)
        for groups in (256, 300):
            assert size(256, groups, 256, 32, hkv, d, bs, shared + 512, shared, 0) == tight, (hkv, groups)
    # nothing shared, and the bounds say so: one pass, as for as many groups as sequences
    assert size(256, 256, 1, 32, 8, 128, 16, 512, 500, 0) == size(256, 300, 1, 32, 8, 128, 16, 512, 500, 0)
    assert size(256, 256, 1, 32, 8, 128, 16, 512, 500, 0) <= size(256, 256, 256, 32, 8, 128, 16, 512, 500, 0)


def test_decode_takes_long_requests_that_start_inside_blocks_as_whole_blocks():
    from paged_kv_cache_140_gb300 import _build, _lib
    _build.build()
    used = _lib.load().pa_decode_partition_size
    for bs in BLOCK_SIZES:
        for P in range(16, 32 * bs + 1, 16):
            got = used(4, 8, 8, 128, bs, 100000, P)
            assert most_blocks(got, bs) <= 32
            assert got == (P if most_blocks(P, bs) <= 32 else P - P % bs), (bs, P)
            assert used(4, 8, 8, 128, bs, P, P) == P         # one partition starts at 0
        assert used(4, 8, 8, 128, bs, 100000, 32 * bs + 16) == 0
