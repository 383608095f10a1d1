"""paged_attention_tree against 64-bit attention over a dense copy of the
cache: chains and trees of drafts, ragged batches, rows that see nothing."""
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


def tree_masks(drafts, seed, kind):
    """Per row a mask: `tree` random parents, `any` random bits (bits behind
    the drafts set too, self not always seen)."""
    rng = random.Random(seed)
    out = []
    for n in drafts:
        mine = []
        for i in range(n):
            if kind == "any":
                mine.append(rng.getrandbits(64) if rng.random() < 0.8 else 0)
            else:
                mine.append((mine[rng.randint(max(0, i - 4), i - 1)] if i else 0) | (1 << i))
        out += mine
    return out


def to_mask(masks):
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64,
                        device="cuda")


def starts(drafts, first=0):
    out = [first]
    for n in drafts:
        out.append(out[-1] + n)
    return out


def verify(c, q, start, drafts, masks, out, scale, what):
    for s, n in enumerate(drafts):
        if n == 0:
            continue
        ctx = c.lens[s]
        see = torch.ones(n, ctx, dtype=torch.bool)
        for i in range(n):
            m = (2 << i) - 1 if masks is None else masks[start[s] - start[0] + i]
            for b in range(n):
                see[i, ctx - n + b] = bool((m >> b) & 1)
        want, tol = attend(q[start[s]:start[s] + n], c.K[s], c.V[s], see.cuda(), scale)
        check(out[start[s]:start[s] + n], want, tol, "%s sequence %d" % (what, s))


def call(c, q, start, drafts, mask, scale, max_draft=None, **kw):
    return pkv.paged_attention_tree(
        q, c.k, c.v, c.tables, c.context_lens,
        torch.tensor(start, dtype=torch.int32, device="cuda"), scale, c.max_context,
        max(1, max(drafts)) if max_draft is None else max_draft, mask, **c.kw(), **kw)


RAGGED = [(1, 1), (5, 5), (15, 1), (16, 3), (17, 2), (33, 0), (64, 64), (100, 64), (127, 7),
          (128, 12), (129, 21), (130, 22), (300, 33), (0, 0), (517, 43), (1033, 5), (70, 63)]


@pytest.mark.parametrize("kind", ["chain", "tree", "any"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,block", [(128, 16), (128, 32), (256, 16), (256, 32)])
def test_ragged_batch(d, block, fp8, kind, _lib):
    hk, g = 2, {128: 3, 256: 6}[d]
    lens, drafts = [a for a, _ in RAGGED], [b for _, b in RAGGED]
    c = Cache(lens, hk, d, block, fp8, seed=d + block + fp8)
    start = starts(drafts)
    q = queries(start[-1], hk * g, d, seed=5)
    masks = None if kind == "chain" else tree_masks(drafts, 9, kind)
    out = call(c, q, start, drafts, None if masks is None else to_mask(masks), d ** -0.5)
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0
    verify(c, q, start, drafts, masks, out, d ** -0.5, kind)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("g", [1, 2, 4, 5, 7, 8])
def test_query_groups(g, fp8, _lib):
    lens, drafts = [40, 200, 333, 700], [1, 16, 17, 64]
    c = Cache(lens, 3, 128, 16, fp8, seed=g)
    start = starts(drafts)
    q = queries(start[-1], 3 * g, 128, seed=g)
    masks = tree_masks(drafts, g, "tree")
    out = call(c, q, start, drafts, to_mask(masks), 0.1, max_draft=64)
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0
    verify(c, q, start, drafts, masks, out, 0.1, "g=%d" % g)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,lens,drafts", [(256, [70001], [5]), (128, [40000, 17], [64, 17]),
                                           (256, [9000, 1, 12345], [16, 1, 2])])
def test_long_contexts(d, lens, drafts, fp8, _lib):
    c = Cache(lens, 2, d, 32, fp8, seed=3)
    start = starts(drafts)
    q = queries(start[-1], 12, d, seed=4)
    out = call(c, q, start, drafts, None, d ** -0.5)
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0
    verify(c, q, start, drafts, None, out, d ** -0.5, "long")


def test_many_sequences(_lib):
    rng = random.Random(2)
    lens = [rng.randint(1, 90) for _ in range(700)]
    drafts = [rng.randint(0, min(4, n)) for n in lens]
    c = Cache(lens, 1, 128, 16, False, seed=8)
    start = starts(drafts)
    q = queries(start[-1], 8, 128, seed=8)
    out = call(c, q, start, drafts, None, 128 ** -0.5)
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0
    verify(c, q, start, drafts, None, out, 128 ** -0.5, "many")


def test_growing_logits(_lib):
    """Logits that grow by far more than the rescaling thresholds along the
    context, and a few that dwarf the others."""
    c = Cache([2000], 1, 256, 16, False, seed=6)
    ramp = torch.linspace(0.01, 6, 2000, device="cuda")[:, None, None]
    k = (c.K[0] * ramp).to(torch.bfloat16)
    slots = [int(c.tables[0, t // 16]) * 16 + t % 16 for t in range(2000)]
    pkv.kv_cache_write(k, c.V[0].to(torch.bfloat16), torch.tensor(slots, device="cuda"), c.k, c.v)
    c.K[0] = k.double()
    q = queries(9, 6, 256, seed=1, std=3)
    out = call(c, q, [0, 9], [9], None, 0.25)
    verify(c, q, [0, 9], [9], None, out, 0.25, "ramp")
    assert int(_lib.item()) == 0


def test_rows_outside_stay(_lib):
    """q_start may begin behind row 0; rows before it and behind the last
    sequence are left as they were, NaN queries there do no harm."""
    lens, drafts = [50, 60], [3, 4]
    c = Cache(lens, 2, 128, 16, False, seed=1)
    start = starts(drafts, first=2)
    q = queries(start[-1] + 5, 4, 128, seed=1)
    q[:2] = float("nan")
    q[start[-1]:] = float("nan")
    out = torch.full_like(q, 7.0)
    r = call(c, q, start, drafts, None, 0.1, out=out)
    assert r is out
    verify(c, q, start, drafts, None, out, 0.1, "offset")
    assert bool((out[:2] == 7).all()) and bool((out[start[-1]:] == 7).all())
    assert int(_lib.item()) == 0


def test_chain_is_its_mask(_lib):
    lens, drafts = [64, 333, 1500], [64, 20, 6]
    c = Cache(lens, 2, 256, 16, False, seed=2)
    start = starts(drafts)
    q = queries(start[-1], 12, 256, seed=2)
    masks = [(2 << i) - 1 for n in drafts for i in range(n)]
    masks = [m & ((1 << 64) - 1) for m in masks]
    a = call(c, q, start, drafts, None, 0.0625)
    b = call(c, q, start, drafts, to_mask(masks), 0.0625)
    assert torch.equal(a, b)


def test_one_draft_is_the_decode(_lib):
    """With one draft per sequence the call is the plain decode."""
    lens = [1, 31, 500, 3000]
    c = Cache(lens, 4, 256, 32, False, seed=12)
    q = queries(4, 24, 256, seed=12)
    a = call(c, q, [0, 1, 2, 3, 4], [1] * 4, None, 0.0625).double()
    b = pkv.paged_attention(q, c.k, c.v, c.tables, c.context_lens, 0.0625, 3000).double()
    for s in range(4):
        want, tol = attend(q[s:s + 1], c.K[s], c.V[s],
                           torch.ones(1, lens[s], dtype=torch.bool, device="cuda"), 0.0625)
        check(a[s:s + 1], want, tol, "tree")
        check(b[s:s + 1], want, tol, "decode")


def test_bad_drafts_are_reported(_lib):
    """A sequence with more drafts than the bound or than its context is
    reported and keeps its rows; the others are computed."""
    for lens, drafts, bound in (([100, 90, 80], [4, 9, 2], 8), ([100, 3, 80], [4, 5, 2], 8)):
        c = Cache(lens, 2, 128, 16, False, seed=5)
        start = starts(drafts)
        q = queries(start[-1], 4, 128, seed=5)
        out = torch.full_like(q, 3.0)
        call(c, q, start, drafts, None, 0.1, max_draft=bound, out=out)
        torch.cuda.synchronize()
        assert int(_lib.item()) == pkv.DEVERR_DRAFT
        _lib.zero_()
        assert bool((out[start[1]:start[2]] == 3).all())
        good = [drafts[0], 0, drafts[2]]
        verify(c, q, start, good, None, out, 0.1, "good ones")


def test_bad_block_is_reported(_lib):
    c = Cache([100, 90], 2, 128, 16, False, seed=5)
    c.tables[1, 2] = -1
    q = queries(6, 4, 128, seed=5)
    out = call(c, q, [0, 3, 6], [3, 3], None, 0.1)
    torch.cuda.synchronize()
    assert int(_lib.item()) == pkv.DEVERR_BLOCK_ID
    _lib.zero_()
    verify(c, q, [0, 3, 6], [3, 0], None, out, 0.1, "the other sequence")


def test_bad_context_is_reported(_lib):
    c = Cache([100, 90], 2, 128, 16, False, seed=5)
    q = queries(6, 4, 128, seed=5)
    for bad in (-1, c.tables.shape[1] * 16 + 1):
        lens = c.context_lens.clone()
        lens[1] = bad
        out = pkv.paged_attention_tree(
            q, c.k, c.v, c.tables, lens, torch.tensor([0, 3, 6], dtype=torch.int32,
                                                      device="cuda"), 0.1, 100, 3)
        torch.cuda.synchronize()
        assert int(_lib.item()) != 0
        _lib.zero_()
        verify(c, q, [0, 3, 6], [3, 0], None, out, 0.1, "the other sequence")


@pytest.mark.parametrize("fp8", [False, True])
def test_repeats_streams_and_graphs(fp8, _lib):
    """The same bits again, on another stream, from a captured graph, and
    from a graph replayed on new inputs in the same buffers."""
    lens, drafts = [2000, 64, 700, 9], [8, 64, 1, 9]
    c = Cache(lens, 2, 256, 16, fp8, seed=21)
    start = starts(drafts)
    st = torch.tensor(start, dtype=torch.int32, device="cuda")
    q = queries(start[-1], 8, 256, seed=21)
    n = pkv.tree_workspace_bytes(4, start[-1], 8, 2, 256, 2000, 64)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda").fill_(0xFF)
    out = torch.empty_like(q)

    def go(stream=None):
        pkv.paged_attention_tree(q, c.k, c.v, c.tables, c.context_lens, st, 0.0625, 2000, 64,
                                 out=out, workspace=ws, stream=stream, **c.kw())

    go()
    first = out.clone()
    for _ in range(3):
        out.zero_()
        go()
        assert torch.equal(out, first)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out.zero_()
    torch.cuda.synchronize()
    go(side)
    side.synchronize()
    assert torch.equal(out, first)
    # allocated by the call, on a stream that is not the current one
    mine = call(c, q, start, drafts, None, 0.0625, stream=side)
    side.synchronize()
    assert torch.equal(mine, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    out.zero_()
    graph.replay()
    assert torch.equal(out, first)
    q2 = queries(start[-1], 8, 256, seed=99)
    keep = q.clone()
    q.copy_(q2)
    graph.replay()
    verify(c, q, start, drafts, None, out, 0.0625, "replay")
    q.copy_(keep)
    graph.replay()
    assert torch.equal(out, first)
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_slow_first_loads(fp8, _lib):
    """Fresh caches whose pages come from memory and whose last pages hold NaN
    behind the context: what the kernel masks may not depend on when a page
    arrives (first and second run give the same finite bits)."""
    lens, drafts = [2000, 60, 700, 9, 1500], [8, 60, 1, 9, 3]
    start = starts(drafts)
    q = queries(start[-1], 8, 256, seed=21)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(60):
        c = Cache(lens, 2, 256, 16, fp8, seed=100 + i)
        flush.fill_(i)
        a = call(c, q, start, drafts, None, 0.0625)
        b = call(c, q, start, drafts, None, 0.0625)
        assert torch.isfinite(a.float()).all() and torch.equal(a, b), i
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_large_pool(fp8, _lib):
    """Blocks whose element offsets pass 2^32."""
    nb = (1 << 32) // (4 * 32 * 256) + 2000
    c = Cache([300, 77], 4, 256, 32, fp8, seed=4, pool_blocks=nb)
    assert int(c.tables[0, 0]) * 4 * 32 * 256 > 1 << 32
    q = queries(9, 24, 256, seed=4)
    out = call(c, q, [0, 4, 9], [4, 5], None, 0.0625)
    verify(c, q, [0, 4, 9], [4, 5], None, out, 0.0625, "large pool")
    assert int(_lib.item()) == 0
