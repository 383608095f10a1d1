"""select_blocks where a CTA scores several runs of 128 blocks, at d = 256: lists
and counts are equal to the definition's. (A batch does that from 912 runs on,
456 and more are scored one run to a CTA.)"""
import pytest
import torch

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build as pkv_build
from test_gpu_select import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.set_device_check(flag)
    yield flag
    pkv.set_device_check(None)


def spread(n, lo, hi):
    """n lengths from lo to hi, evenly spread, in a scattered order."""
    return [lo + (hi - lo) * (i * 37 % n) // max(1, n - 1) for i in range(n)]


# (lengths, hk, g, block, runs of 128 blocks over all pairs)
SHAPES = [
    (spread(30, 1, 8200), 4, 6, 16, 600),       # one run to a CTA
    (spread(46, 4000, 8192), 4, 2, 16, 736),    # the same, full tables
    (spread(70, 1, 8200), 4, 6, 16, 1400),      # three runs to a CTA, two CTAs
    ([131072, 131041, 100000, 4097, 4096, 33, 70001, 126977], 4, 6, 32, 1024),  # two
    (spread(150, 100, 4100), 8, 1, 16, 3600),   # a whole sequence to a CTA
]


@pytest.mark.parametrize("take,first,last", [(128, 1, 2), (37, 0, 0)])
@pytest.mark.parametrize("lens,hk,g,block,runs", SHAPES)
def test_runs_of_blocks(lens, hk, g, block, runs, take, first, last, _lib):
    most = -(-max(lens) // block)
    assert -(-most // 128) * len(lens) * hk == runs
    c = Case(lens, hk, g, 256, block, seed=runs + take)
    c.verify(c.call(take, first, last), take, first, last)
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0


def test_bad_blocks_of_later_runs(_lib):
    """The best block of each run of 128 has no place in the pool: reported, and
    behind all others."""
    c = Case([8200] * 70, 4, 6, 256, 16, seed=5)
    s = 33
    scores = c.scores(s)
    for at in range(0, 513, 128):
        i = at + int(scores[:, at:at + 128].amax(0).argmax())
        c.tables[s, i] = -1 if at % 256 else c.bounds.shape[0]
        scores[:, i] = -(1 << 40)
    got = c.call(60, 0, 0)
    torch.cuda.synchronize()
    assert int(_lib.item()) == pkv.DEVERR_BLOCK_ID
    _lib.zero_()
    assert got[0][s].tolist() == c.want(s, 60, 0, 0, scores)[0]
    c.verify(got, 60, 0, 0, skip=(s,))
    assert int(_lib.item()) == 0
