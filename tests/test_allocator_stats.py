"""What BlockAllocator.stats costs, and its slots where holders of a shared
block were cut to different lengths."""
import time

import pytest

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def best(f, n=5):
    out = []
    for _ in range(n):
        t = time.perf_counter()
        f()
        out.append(time.perf_counter() - t)
    return min(out)


def test_cost_does_not_grow_with_shared_tables():
    """2000 forks of a sequence of 2000 blocks: the blocks and the sequences
    are looked at once each, not every table entry (4 million here)."""
    a = pkv.BlockAllocator(4000, 16, seed=1)
    s = a.new_seq()
    a.append(s, 2000 * 16)
    alone = best(a.stats)
    for _ in range(2000):
        a.fork(s)
    assert a.stats()["used_slots"] == 2000 * 16
    assert best(a.stats) < 20 * alone + 200e-6


def test_slots_of_cut_holders():
    """A slot counts while one holder's length covers it."""
    a = pkv.BlockAllocator(16, 16, seed=2)
    s = a.new_seq()
    a.append(s, 48)
    f, h = a.fork(s), a.fork(s)
    a.truncate(f, 20)
    a.truncate(h, 27)
    assert a.stats()["used_slots"] == 48
    a.truncate(s, 18)
    assert a.stats()["used_slots"] == 16 + 11    # the third block has no holder any more
    a.truncate(h, 16)
    assert a.stats()["used_slots"] == 16 + 4
    a.free(f)
    assert a.stats()["used_slots"] == 16 + 2
    a.free(s)
    assert a.stats()["used_slots"] == 16
    a.truncate(h, 3)
    assert a.stats()["used_slots"] == 3
    a.truncate(h, 0)
    assert a.stats() == {"free_blocks": 16, "used_blocks": 0, "used_slots": 0}
    b = pkv.BlockAllocator.load(a.save())
    assert b.stats() == a.stats()
