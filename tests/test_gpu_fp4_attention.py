"""paged_attention over 4-bit pools against 64-bit attention over a dense copy
of what the pools stand for; slots that hold no token have NaN scales."""
import random

import pytest
import torch

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build as pkv_build
from _dense_side import attend, check, queries
from _pool_side import AnyCache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.set_device_check(flag)
    yield flag
    pkv.set_device_check(None)


def verify(c, q, out, scale, what, skip=()):
    for s, ctx in enumerate(c.lens):
        if s in skip:
            continue
        see = torch.ones(1, ctx, dtype=torch.bool, device="cuda")
        want, tol = attend(q[s:s + 1], c.K[s], c.V[s], see, scale)
        check(out[s:s + 1], want, tol, "%s sequence %d" % (what, s))


def call(c, q, scale, **kw):
    return pkv.paged_attention(q, c.k, c.v, c.tables, c.context_lens, scale, c.max_context,
                               **c.kw(), **kw)


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 100, 127, 128, 129, 500, 1000, 2047]


@pytest.mark.parametrize("d,block", [(128, 16), (128, 32), (256, 16), (256, 32)])
def test_lengths(d, block, _lib):
    for hk, g, seed in ((2, 3, 1), (3, 6, 2), (8, 1, 3)):
        c = AnyCache(LENS, hk, d, block, "fp4", seed=seed)
        q = queries(len(LENS), hk * g, d, seed=seed)
        for bound in (2047, 2048, 2060, c.tables.shape[1] * block):
            c.max_context = bound
            out = call(c, q, d ** -0.5)
            torch.cuda.synchronize()
            assert int(_lib.item()) == 0
            verify(c, q, out, d ** -0.5, "d %d block %d" % (d, block))


@pytest.mark.parametrize("n", [1, 2, 5, 40, 127, 128, 129, 300, 1000])
def test_shares_cut_batches_anywhere(n, _lib):
    """Random lengths, empty contexts among them: a share has parts of many
    sequences, or a sequence parts in many shares."""
    r = random.Random(n)
    for most, d in ((40, 128), (700, 256), (5000, 128)):
        if n * most > 300000:
            continue
        lens = [r.choice([0, r.randint(1, most), r.randint(1, most)]) for _ in range(n)]
        c = AnyCache(lens, 2, d, 16, "fp4", seed=n)
        q = queries(n, 4, d, seed=n)
        out = call(c, q, 0.08)
        verify(c, q, out, 0.08, "n %d" % n, skip=[s for s in range(n) if n > 130 and s % 7])
        assert torch.isfinite(out).all()
    c = AnyCache([0] * n, 1, 128, 32, "fp4", seed=1)
    for bound in (0, 50):
        c.max_context = bound
        assert float(call(c, queries(n, 2, 128, seed=1), 0.1).abs().max()) == 0
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("g", [1, 2, 4, 5, 7, 8])
@pytest.mark.parametrize("d", [128, 256])
def test_query_groups(d, g, _lib):
    # in 40 sequences of 7 tokens nearly every pair is one warp's alone
    for lens in ([40, 200, 333, 700], [7] * 40):
        c = AnyCache(lens, 3, d, 16, "fp4", seed=g)
        q = queries(len(lens), 3 * g, d, seed=g)
        verify(c, q, call(c, q, 0.1), 0.1, "g=%d" % g)
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("lens", [[60000], [30000, 9, 20000], [5000] * 20, [300] * 700])
@pytest.mark.parametrize("d", [128, 256])
def test_long_and_many(lens, d, _lib):
    c = AnyCache(lens, 2, d, 32, "fp4", seed=3)
    q = queries(len(lens), 12, d, seed=4)
    out = call(c, q, d ** -0.5)
    if len(lens) > 100:
        for s in range(0, len(lens), 37):
            see = torch.ones(1, lens[s], dtype=torch.bool, device="cuda")
            want, tol = attend(q[s:s + 1], c.K[s], c.V[s], see, d ** -0.5)
            check(out[s:s + 1], want, tol, "sequence %d" % s)
    else:
        verify(c, q, out, d ** -0.5, "long")
    assert int(_lib.item()) == 0


def test_queries_far_from_one(_lib):
    """Rows of q of very different size, one behind f16's range and one below it."""
    c = AnyCache([300, 1000], 2, 128, 16, "fp4", seed=9)
    q = queries(2, 8, 128, seed=9)
    size = torch.tensor([1e6, 1.0, 1e-6, 3.0, 1e-30, 0.0, 1e10, 0.5], device="cuda")
    q = (q.float() * size[:, None]).to(torch.bfloat16)
    for j, scale in ((0, 1e-7), (2, 1e5), (1, 0.09)):
        out = call(c, q, scale)
        for s, ctx in enumerate(c.lens):
            see = torch.ones(1, ctx, dtype=torch.bool, device="cuda")
            want, tol = attend(q[s:s + 1], c.K[s], c.V[s], see, scale)
            rows = [j] if j != 1 else [1, 2, 3, 4, 5, 7]
            check(out[s:s + 1, rows], want[:, rows], tol[:, rows], "scale %g" % scale)
    assert int(_lib.item()) == 0


def test_many_small_weights(_lib):
    """One token of weight 1 with V = 0 and 40000 of weight 2^-26 each: their sum
    is the result."""
    n, d = 40001, 128
    c = AnyCache([n], 1, d, 32, "fp4", seed=1)
    c.ks.fill_(1.0)
    c.vs.fill_(1.0)
    # values that the format holds exactly: 6 = 6 * 1, 0.75 = 6 * 0.125
    k = torch.zeros(n, 1, d, dtype=torch.bfloat16, device="cuda")
    v = torch.full((n, 1, d), 0.75, dtype=torch.bfloat16, device="cuda")
    k[0, 0, 0], v[0] = 6.0, 0.0
    pages = c.tables[0, torch.arange(n, device="cuda") // 32].long()
    slots = pages * 32 + torch.arange(n, device="cuda") % 32
    pkv.kv_cache_write(k, v, slots, c.k, c.v, c.ks, c.vs)
    got_k, got_v = pkv.kv_cache_read(slots, c.k, c.v, c.ks, c.vs)
    assert torch.equal(got_k, k) and torch.equal(got_v, v)
    q = torch.zeros(1, 1, d, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0] = 1.0
    scale = 26 * 0.6931471805599453 / 6
    out = call(c, q, scale)
    w = torch.exp(q.double()[0, 0] @ k.double()[:, 0].T * scale)
    want = (w / w.sum() @ v.double()[:, 0]).view(1, 1, d)
    # the output's rounding; the weights' to 11 bits, a logit of 26 in fp32, ex2
    check(out, want, want.abs() * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16), "small weights")
    assert int(_lib.item()) == 0


def test_scales_of_the_logits(_lib):
    """Scales of zero and below, and a head whose scale is negative."""
    c = AnyCache([5, 100, 1000], 2, 256, 16, "fp4", seed=6)
    q = queries(3, 8, 256, seed=6)
    for scale in (0.0, -0.0625, 1e-30):
        verify(c, q, call(c, q, scale), scale, "scale %g" % scale)
    c.ks[1] = -c.ks[1]
    for s in range(3):
        c.K[s][:, 1] = -c.K[s][:, 1]
    verify(c, q, call(c, q, 0.0625), 0.0625, "negative scale")
    assert int(_lib.item()) == 0


def test_the_order_makes_no_difference_and_partitions_are_refused(_lib):
    c = AnyCache([40, 2000, 333, 700], 2, 256, 16, "fp4", seed=1)
    q = queries(4, 12, 256, seed=1)
    want = call(c, q, 0.0625)
    order = torch.tensor([3, 2, 1, 0], dtype=torch.int32, device="cuda")
    for partition in (0, None):
        assert torch.equal(call(c, q, 0.0625, partition_size=partition, seq_order=order), want)
    with pytest.raises(ValueError, match="partition_size"):
        call(c, q, 0.0625, partition_size=64)


def test_a_longer_context_than_the_bound_is_cut(_lib):
    c = AnyCache([500, 90], 2, 128, 16, "fp4", seed=5)
    q = queries(2, 4, 128, seed=5)
    c.max_context = 100
    out = call(c, q, 0.1)
    torch.cuda.synchronize()
    assert int(_lib.item()) == pkv.DEVERR_CONTEXT
    _lib.zero_()
    verify(c, q, out, 0.1, "the other", skip=(0,))
    see = torch.ones(1, 100, dtype=torch.bool, device="cuda")
    want, tol = attend(q[:1], c.K[0][:100], c.V[0][:100], see, 0.1)
    check(out[:1], want, tol, "cut")


@pytest.mark.parametrize("block", [16, 32])
def test_bad_block_and_context_are_reported(block, _lib):
    c = AnyCache([100, 90], 2, 128, block, "fp4", seed=5)
    q = queries(2, 4, 128, seed=5)
    keep = c.tables.clone()
    for bad in (-1, c.k.shape[0], 1 << 30):
        c.tables[1, 1] = bad
        out = call(c, q, 0.1)
        torch.cuda.synchronize()
        assert int(_lib.item()) == pkv.DEVERR_BLOCK_ID
        _lib.zero_()
        verify(c, q, out, 0.1, "the other", skip=(1,))
    c.tables.copy_(keep)
    for bad in (-3, 1 << 20):
        lens = c.context_lens.clone()
        c.context_lens[1] = bad
        out = call(c, q, 0.1)
        torch.cuda.synchronize()
        assert int(_lib.item()) in (pkv.DEVERR_CONTEXT, pkv.DEVERR_BLOCK_ID)
        _lib.zero_()
        c.context_lens.copy_(lens)
        verify(c, q, out, 0.1, "the other", skip=(1,))


@pytest.mark.parametrize("lens", [[2000, 64, 700, 9], [90] * 500, [30000]])
@pytest.mark.parametrize("d", [128, 256])
def test_repeats_streams_and_graphs(d, lens, _lib):
    n = len(lens)
    c = AnyCache(lens, 2, d, 16, "fp4", seed=21)
    q = queries(n, 8, d, seed=21)
    ws = torch.empty(pkv.fp4_workspace_bytes(c.k, n, c.max_context), dtype=torch.uint8,
                     device="cuda").fill_(0xFF)
    out = torch.empty_like(q)

    def go(stream=None):
        call(c, q, 0.0625, out=out, workspace=ws, stream=stream)

    go()
    first = out.clone()
    some = [s for s in range(n) if n > 100 and s % 17]
    verify(c, q, first, 0.0625, "first", skip=some)
    for _ in range(20):
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
    mine = call(c, q, 0.0625, stream=side)
    side.synchronize()
    assert torch.equal(mine, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    out.zero_()
    graph.replay()
    assert torch.equal(out, first)
    q.copy_(queries(n, 8, d, seed=22))
    graph.replay()
    verify(c, q, out, 0.0625, "replay", skip=some)
    # other lengths in the same graph
    c.context_lens.copy_((c.context_lens + 1) // 2)
    graph.replay()
    c.lens = c.context_lens.tolist()
    c.K, c.V = ([x[:m] for x, m in zip(y, c.lens)] for y in (c.K, c.V))
    verify(c, q, out, 0.0625, "shorter", skip=some)
    assert int(_lib.item()) == 0


def test_large_pool(_lib):
    nb = (1 << 32) // (4 * 32 * 144) + 2000
    c = AnyCache([300, 77], 4, 256, 32, "fp4", seed=4, pool_blocks=nb)
    q = queries(2, 24, 256, seed=4)
    verify(c, q, call(c, q, 0.0625), 0.0625, "large pool")
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_library_partition_of_other_pools(kind, _lib):
    """partition_size=None on bf16 and E4M3 pools."""
    for lens in ([40, 2000, 333, 700], [9000], [100] * 300):
        c = AnyCache(lens, 2, 128, 16, kind, seed=2)
        q = queries(len(lens), 8, 128, seed=2)
        verify(c, q, call(c, q, 0.09, partition_size=None), 0.09, kind)
    assert int(_lib.item()) == 0
