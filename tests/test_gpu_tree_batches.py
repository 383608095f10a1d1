"""paged_attention_tree over batches whose sequences differ much, its bounds,
queries that are not finite, and calls that run beside each other."""
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


def starts(drafts):
    out = [0]
    for n in drafts:
        out.append(out[-1] + n)
    return out


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def call(c, q, start, drafts, scale, **kw):
    return pkv.paged_attention_tree(q, c.k, c.v, c.tables, c.context_lens, int32(start), scale,
                                    kw.pop("max_context", c.max_context), max(1, max(drafts)),
                                    **c.kw(), **kw)


def verify(c, q, start, drafts, out, scale, only=None):
    """Chains of drafts."""
    for s, n in enumerate(drafts):
        if n == 0 or (only is not None and s not in only):
            continue
        ctx = c.lens[s]
        see = torch.ones(n, ctx, dtype=torch.bool)
        see[:, ctx - n:] = torch.ones(n, n).tril() > 0
        want, tol = attend(q[start[s]:start[s] + n], c.K[s], c.V[s], see.cuda(), scale)
        check(out[start[s]:start[s] + n], want, tol, "sequence %d" % s)


# Where a CTA's share is long, a unit's start counts as several steps: short
# sequences among long ones, at the batch's start, end and everywhere; runs of
# several sequences per thread (more than 512 of them); every sequence with the
# same number of row tiles (teams) and none of them long.
BATCHES = {
    "short first": [(n % 90 + 1, 1 + n % 3) for n in range(300)] + [(9000, 2)] * 4,
    "short last": [(9000, 2)] * 4 + [(n % 90 + 1, n % 4) for n in range(300)],
    "among": [(17 + n, 2) if n % 9 else (5000 + 128 * n, 3) for n in range(60)],
    "empty ones": [(4000, 0) if n % 3 else (1 + 97 * n, 1) for n in range(90)],
    "many": [((7919 * n) % 500 + 8, n % 8) for n in range(1100)],
    "one step each": [(128, 1)] * 640,
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,hk,g", [(128, 2, 4), (256, 1, 6)])
@pytest.mark.parametrize("name", list(BATCHES))
def test_uneven_batches(name, d, hk, g, fp8, _lib):
    lens = [n for n, _ in BATCHES[name]]
    drafts = [min(n, k) for n, k in BATCHES[name]]
    c = Cache(lens, hk, d, 16 if d == 256 else 32, fp8, seed=31)
    start = starts(drafts)
    q = queries(start[-1], hk * g, d, seed=31)
    out = torch.full_like(q, float("nan"))
    call(c, q, start, drafts, d ** -0.5, out=out)
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0
    assert torch.isfinite(out.float()).all()
    rng = random.Random(1)
    long = [s for s, n in enumerate(lens) if n > 1000]
    verify(c, q, start, drafts, out, d ** -0.5,
           set(rng.sample(range(len(lens)), min(60, len(lens))) + long[:12]))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,g", [(64, 8), (40, 8), (64, 3)])
def test_teams_of_many_sequences(n, g, fp8, _lib):
    rng = random.Random(3)
    lens = [rng.randint(n, 700) for _ in range(150)]
    drafts = [n] * 150
    c = Cache(lens, 2, 128, 16, fp8, seed=32)
    start = starts(drafts)
    q = queries(start[-1], 2 * g, 128, seed=32)
    out = call(c, q, start, drafts, 128 ** -0.5)
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0
    verify(c, q, start, drafts, out, 128 ** -0.5, set(rng.sample(range(150), 30)))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,g", [(40, 8), (3, 2)])
def test_teams_among_idle_sequences(n, g, fp8, _lib):
    """More sequences than threads look for a share's place, most of them
    without a draft, the others all with the same number of row tiles."""
    rng = random.Random(4)
    lens = [rng.randint(n, 300) for _ in range(1300)]
    drafts = [n if s % 7 == 3 else 0 for s in range(1300)]
    c = Cache(lens, 2, 128, 16, fp8, seed=33)
    start = starts(drafts)
    q = queries(start[-1], 2 * g, 128, seed=33)
    out = torch.full_like(q, float("nan"))
    call(c, q, start, drafts, 128 ** -0.5, out=out)
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0
    assert torch.isfinite(out.float()).all()
    verify(c, q, start, drafts, out, 128 ** -0.5,
           set(rng.sample([s for s in range(1300) if drafts[s]], 40)))


def test_context_above_the_bound_is_reported(_lib):
    c = Cache([100, 300, 90], 2, 128, 16, False, seed=5)
    drafts, start = [3, 3, 3], [0, 3, 6, 9]
    q = queries(9, 4, 128, seed=5)
    out = torch.full_like(q, 3.0)
    call(c, q, start, drafts, 0.1, max_context=299, out=out)
    torch.cuda.synchronize()
    assert int(_lib.item()) == pkv.DEVERR_CONTEXT
    _lib.zero_()
    assert bool((out[3:6] == 3).all())
    verify(c, q, start, drafts, out, 0.1, {0, 2})


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_queries_that_are_not_finite(bad, d, fp8, _lib):
    """They make their own row NaN and no other one."""
    c = Cache([700, 40], 2, d, 16, fp8, seed=6)
    drafts, start = [5, 3], [0, 5, 8]
    q = queries(8, 8, d, seed=6)
    q[2, 5, 17] = bad
    out = call(c, q, start, drafts, d ** -0.5)
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0
    assert bool(torch.isnan(out[2, 5].float()).all())
    q[2, 5] = 0
    want = call(c, q, start, drafts, d ** -0.5)
    keep = torch.ones(8, 8, dtype=torch.bool, device="cuda")
    keep[2, 5] = False
    assert torch.equal(out[keep], want[keep])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("scale", [-0.07, 0.0, 1e-30])
def test_scales(scale, d, fp8, _lib):
    """Negative, zero and tiny scales, over committed tokens (no mask in their
    steps) and drafts."""
    c = Cache([900, 130, 64], 2, d, 16, fp8, seed=9)
    drafts, start = [4, 9, 64], [0, 4, 13, 77]
    q = queries(77, 8, d, seed=9)
    out = call(c, q, start, drafts, scale)
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0
    verify(c, q, start, drafts, out, scale)


@pytest.mark.parametrize("fp8", [False, True])
def test_unsigned_masks_and_padded_queries(fp8, _lib):
    """uint64 masks, more rows of q than drafts, a larger bound of drafts."""
    c = Cache([300, 77], 2, 128, 32, fp8, seed=10)
    drafts, start = [5, 7], [0, 5, 12]
    q = queries(40, 8, 128, seed=10)
    chain = torch.tensor([(2 << i) - 1 for n in drafts for i in range(n)] + [0] * 28,
                         dtype=torch.int64, device="cuda")
    out = torch.full_like(q, 3.0)
    pkv.paged_attention_tree(q, c.k, c.v, c.tables, c.context_lens, int32(start), 0.09, 300, 64,
                             chain.view(torch.uint64), out=out, **c.kw())
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0
    assert bool((out[12:] == 3).all())
    verify(c, q, start, drafts, out, 0.09)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,lens,drafts,hk,g", [(256, [70001], [5], 2, 4),
                                                (256, [33333, 70000, 5], [17, 30, 5], 2, 6),
                                                (128, [8192] * 32, [4] * 32, 8, 4)])
def test_long_repeats(d, lens, drafts, hk, g, fp8, _lib):
    """The same bits every time, from HBM and from L2: no slot of a ring is
    filled anew while it is still being read."""
    c = Cache(lens, hk, d, 32, fp8, seed=7)
    start = starts(drafts)
    q = queries(start[-1], hk * g, d, seed=7)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    first = call(c, q, start, drafts, d ** -0.5)
    verify(c, q, start, drafts, first, d ** -0.5, {0, len(lens) - 1})
    for i in range(60):
        if i % 3 == 0:
            flush.fill_(i)
        assert torch.equal(call(c, q, start, drafts, d ** -0.5), first), i
    assert int(_lib.item()) == 0


def test_calls_beside_each_other(_lib):
    """Calls on two streams at once, their workspaces allocated by the calls,
    between them memory that other work takes and gives back."""
    c = Cache([3000, 1200, 5000], 2, 256, 16, False, seed=7)
    drafts, start = [8, 20, 3], [0, 8, 28, 31]
    st = int32(start)
    q = [queries(31, 12, 256, seed=40 + i) for i in range(2)]

    def go(i):
        return pkv.paged_attention_tree(q[i], c.k, c.v, c.tables, c.context_lens, st, 0.0625,
                                        c.max_context, 20)

    want = [go(0), go(1)]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(30):
        for i in range(2):
            with torch.cuda.stream(side[i]):
                got[i].append(go(i))
                torch.empty(30 << 20, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])
    assert int(_lib.item()) == 0


def test_graphs_beside_each_other(_lib):
    """Two captured graphs, each with its own workspace, replayed at once."""
    c = Cache([3000, 1200, 5000], 2, 256, 16, False, seed=7)
    st = int32([0, 8, 28, 31])
    q = [queries(31, 12, 256, seed=40 + i) for i in range(2)]
    go = lambda i: pkv.paged_attention_tree(  # noqa: E731
        q[i], c.k, c.v, c.tables, c.context_lens, st, 0.0625, c.max_context, 20)
    want = [go(0), go(1)]
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            outs.append(go(i))
    side = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i in range(2):
            outs[i].zero_()
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(side[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    assert int(_lib.item()) == 0
