"""paged_attention_tree over drafts that no row sees (padding, pruned nodes):
their slots may hold anything, NaN and infinities included."""
import random

import pytest
import torch

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build as pkv_build
from _dense_side import Cache, attend, check, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.set_device_check(flag)
    yield flag
    pkv.set_device_check(None)


def masks_without(n, hidden, rng):
    """n masks of a random tree over the drafts that are not hidden; a hidden
    draft's own row sees some of the others, or nothing."""
    masks, seen = [], []
    for i in range(n):
        m = 0
        if seen and rng.random() < 0.9:
            m = masks[seen[rng.randint(max(0, len(seen) - 4), len(seen) - 1)]]
        if i not in hidden:
            m |= 1 << i
            seen.append(i)
        masks.append(m)
    return masks


def run(c, drafts, hidden, g, seed, flag, poisons):
    """The call with each kind of poison in the hidden drafts' slots, against
    64 bits over the other tokens (the hidden rows of the dense copy are zero:
    no row gives them weight). Bits behind a sequence's drafts are set: they
    name nothing."""
    d, hk = c.d, c.hk
    rng = random.Random(seed)
    start = [0]
    for n in drafts:
        start.append(start[-1] + n)
    masks = [masks_without(n, h, rng) for n, h in zip(drafts, hidden)]
    q = queries(start[-1], hk * g, d, seed)
    words = [m | (~((1 << n) - 1) & ((1 << 64) - 1)) for n, ms in zip(drafts, masks) for m in ms]
    mask = torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64,
                        device="cuda")
    st = torch.tensor(start, dtype=torch.int32, device="cuda")
    for s, h in enumerate(hidden):
        for b in h:
            c.K[s][c.lens[s] - drafts[s] + b] = 0
            c.V[s][c.lens[s] - drafts[s] + b] = 0
    first = None
    for bits in poisons:
        for pool in (c.k, c.v):
            raw = pool if c.fp8 else pool.view(torch.int16)
            for s, h in enumerate(hidden):
                for b in h:
                    t = c.lens[s] - drafts[s] + b
                    raw[int(c.tables[s, t // c.block]), :, t % c.block] = bits
        out = pkv.paged_attention_tree(q, c.k, c.v, c.tables, c.context_lens, st, d ** -0.5,
                                       c.max_context, max(drafts), mask, **c.kw())
        torch.cuda.synchronize()
        assert int(flag.item()) == 0
        for s, n in enumerate(drafts):
            see = torch.ones(n, c.lens[s], dtype=torch.bool)
            for i in range(n):
                for b in range(n):
                    see[i, c.lens[s] - n + b] = bool((masks[s][i] >> b) & 1)
            want, tol = attend(q[start[s]:start[s + 1]], c.K[s], c.V[s], see.cuda(), d ** -0.5)
            check(out[start[s]:start[s + 1]], want, tol, "sequence %d" % s)
        # what a hidden slot holds changes no bit
        first = out if first is None else first
        assert torch.equal(out, first)


BF16 = [0x4000, 0x7FC0, 0x7F80, -0x80]  # 2, NaN, inf, -inf
E4M3 = [0x40, 0x7F, 0xFF]               # 2, NaN, -NaN


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,block", [(128, 16), (128, 32), (256, 16), (256, 32)])
def test_hidden_drafts_hold_anything(d, block, fp8, _lib):
    """Drafts inside one step, over two steps (and, at d = 256, over the two
    halves of a step's V), over the context's end inside a run of 16 tokens;
    everything hidden; nothing committed."""
    shapes = [(70, 20), (135, 12), (1040, 30), (200, 16), (8, 8), (257, 5), (64, 64), (900, 64),
              (128, 9), (129, 9), (333, 40)]
    rng = random.Random(d + block)
    hidden = []
    for i, (_, n) in enumerate(shapes):
        h = {b for b in range(n) if rng.random() < 0.4} | {n - 1}
        hidden.append(set(range(n)) if i == 5 else h)
    c = Cache([a for a, _ in shapes], 2, d, block, fp8, seed=d + block)
    run(c, [n for _, n in shapes], hidden, {128: 3, 256: 6}[d], 7, _lib, E4M3 if fp8 else BF16)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("lens,n", [([3000] * 6, 64), ([700, 711, 725], 40), ([20000], 50)])
def test_several_row_tiles(lens, n, d, fp8, _lib):
    """Up to 512 rows per KV head: every tile loads the hidden rows itself."""
    rng = random.Random(3)
    hidden = [{b for b in range(n) if rng.random() < 0.3} | {0, n - 1} for _ in lens]
    c = Cache(lens, 2, d, 16, fp8, seed=11)
    run(c, [n] * len(lens), hidden, 8, 5, _lib, E4M3 if fp8 else BF16)


@pytest.mark.parametrize("fp8", [False, True])
def test_padded_batch(fp8, _lib):
    """A fixed number of drafts per sequence, as a captured graph has it: the
    padding's slots were never written (a fresh pool) and its bits are clear."""
    lens, real = [50, 300, 129, 77, 515], [3, 0, 8, 1, 5]
    hidden = [set(range(k, 8)) for k in real]
    c = Cache([n + 8 for n in lens], 4, 256, 32, fp8, seed=4)
    run(c, [8] * 5, hidden, 4, 9, _lib, E4M3 if fp8 else BF16)
