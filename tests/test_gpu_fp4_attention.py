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


def call(c, q, scale, partition, **kw):
    return pkv.paged_attention(q, c.k, c.v, c.tables, c.context_lens, scale, c.max_context,
                               partition, **c.kw(), **kw)


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 100, 127, 128, 129, 500, 1000, 2047]


@pytest.mark.parametrize("partition", [None, 0, 32, 96, 160, 1024])
@pytest.mark.parametrize("d,block", [(128, 16), (128, 32), (256, 16), (256, 32)])
def test_lengths(d, block, partition, _lib):
    for hk, g, seed in ((2, 3, 1), (3, 6, 2)):
        c = AnyCache(LENS, hk, d, block, "fp4", seed=seed)
        q = queries(len(LENS), hk * g, d, seed=seed)
        out = call(c, q, d ** -0.5, partition)
        torch.cuda.synchronize()
        assert int(_lib.item()) == 0
        verify(c, q, out, d ** -0.5, "d %d block %d" % (d, block))


def test_partitions_of_one_odd_block(_lib):
    """Partitions of an odd number of 16-token blocks: the work of a step ends
    inside a partition."""
    for p in (16, 48, 80, 112):
        c = AnyCache([700, 33, 16, 5], 2, 256, 16, "fp4", seed=p)
        q = queries(4, 8, 256, seed=p)
        verify(c, q, call(c, q, 0.0625, p), 0.0625, "partition %d" % p)
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("n", [1, 2, 5, 40, 129, 300, 1000])
def test_batches_of_random_lengths(n, _lib):
    """Empty contexts among them; one pass and the library's cut."""
    r = random.Random(n)
    for most, d in ((40, 128), (700, 256), (5000, 128)):
        if n * most > 300000:
            continue
        lens = [r.choice([0, r.randint(1, most), r.randint(1, most)]) for _ in range(n)]
        c = AnyCache(lens, 2, d, 16, "fp4", seed=n)
        q = queries(n, 4, d, seed=n)
        skip = [s for s in range(n) if n > 130 and s % 7]
        for partition in (None, 0, 256):
            out = call(c, q, 0.08, partition)
            verify(c, q, out, 0.08, "n %d" % n, skip)
            assert torch.isfinite(out).all()
    c = AnyCache([0] * n, 1, 128, 32, "fp4", seed=1)
    for bound, partition in ((0, None), (0, 32), (50, None), (50, 32)):
        c.max_context = bound
        assert float(call(c, queries(n, 2, 128, seed=1), 0.1, partition).abs().max()) == 0
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("partition", [0, 64])
def test_scales_of_the_logits(partition, _lib):
    """Scales of zero and below, and a head whose scale is negative."""
    c = AnyCache([5, 100, 1000], 2, 256, 16, "fp4", seed=6)
    q = queries(3, 8, 256, seed=6)
    for scale in (0.0, -0.0625, 1e-30):
        verify(c, q, call(c, q, scale, partition), scale, "scale %g" % scale)
    c.ks[1] = -c.ks[1]
    for s in range(3):
        c.K[s][:, 1] = -c.K[s][:, 1]
    verify(c, q, call(c, q, 0.0625, partition), 0.0625, "negative scale")
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("g", [1, 2, 4, 5, 7, 8])
@pytest.mark.parametrize("d", [128, 256])
def test_query_groups(d, g, _lib):
    for partition in (0, 64, None):
        c = AnyCache([40, 200, 333, 700], 3, d, 16, "fp4", seed=g)
        q = queries(4, 3 * g, d, seed=g)
        verify(c, q, call(c, q, 0.1, partition), 0.1, "g=%d" % g)
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("lens", [[60000], [30000, 9, 20000], [5000] * 20, [300] * 700])
@pytest.mark.parametrize("d", [128, 256])
def test_long_and_many(lens, d, _lib):
    c = AnyCache(lens, 2, d, 32, "fp4", seed=3)
    q = queries(len(lens), 12, d, seed=4)
    out = call(c, q, d ** -0.5, None)
    if len(lens) > 100:
        for s in range(0, len(lens), 37):
            see = torch.ones(1, lens[s], dtype=torch.bool, device="cuda")
            want, tol = attend(q[s:s + 1], c.K[s], c.V[s], see, d ** -0.5)
            check(out[s:s + 1], want, tol, "sequence %d" % s)
    else:
        verify(c, q, out, d ** -0.5, "long")
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("partition", [0, 512])
def test_queries_far_from_one(partition, _lib):
    """Rows of q of very different size, one behind f16's range and one below it."""
    c = AnyCache([300, 1000], 2, 128, 16, "fp4", seed=9)
    q = queries(2, 8, 128, seed=9)
    size = torch.tensor([1e6, 1.0, 1e-6, 3.0, 1e-30, 0.0, 1e10, 0.5], device="cuda")
    q = (q.float() * size[:, None]).to(torch.bfloat16)
    for j, scale in ((0, 1e-7), (2, 1e5), (1, 0.09)):
        out = call(c, q, scale, partition)
        for s, ctx in enumerate(c.lens):
            see = torch.ones(1, ctx, dtype=torch.bool, device="cuda")
            want, tol = attend(q[s:s + 1], c.K[s], c.V[s], see, scale)
            rows = [j] if j != 1 else [1, 2, 3, 4, 5, 7]
            check(out[s:s + 1, rows], want[:, rows], tol[:, rows], "scale %g" % scale)
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("partition", [0, 2048])
def test_many_small_weights(partition, _lib):
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
    out = call(c, q, scale, partition)
    w = torch.exp(q.double()[0, 0] @ k.double()[:, 0].T * scale)
    want = (w / w.sum() @ v.double()[:, 0]).view(1, 1, d)
    # the output's rounding; the weights' to 11 bits, a logit of 26 in fp32, ex2
    check(out, want, want.abs() * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16), "small weights")
    assert int(_lib.item()) == 0


def test_parts_of_the_call(_lib):
    """Decode and merge as two calls, the form without a workspace, every order
    of the sequences: the same bits."""
    c = AnyCache([40, 2000, 333, 700], 2, 256, 16, "fp4", seed=1)
    q = queries(4, 12, 256, seed=1)
    for partition in (64, 512):
        want = call(c, q, 0.0625, partition)
        verify(c, q, want, 0.0625, "one call")
        ws = pkv.alloc_workspace(4, 12, 256, 2000, partition)
        out = torch.empty_like(q)
        pkv.paged_attention_decode(out, q, c.k, c.v, c.tables, c.context_lens, 0.0625, 2000,
                                   partition, ws, **c.kw())
        pkv.paged_attention_reduce(out, ws, c.context_lens, 2000, partition)
        assert torch.equal(out, want)
        out.zero_()
        pkv.paged_attention_decode_noalloc(out, q, c.k, c.v, c.tables, c.context_lens, 0.0625,
                                           2000, partition, **c.kw())
        assert torch.equal(out, want)
    for partition in (0, 64):
        want = call(c, q, 0.0625, partition)
        for order in ([3, 2, 1, 0], [1, 3, 2, 0]):
            o = torch.tensor(order, dtype=torch.int32, device="cuda")
            assert torch.equal(call(c, q, 0.0625, partition, seq_order=o), want)
    assert int(_lib.item()) == 0
    bad = torch.tensor([1, 4, 2, 0], dtype=torch.int32, device="cuda")
    call(c, q, 0.0625, 0, seq_order=bad)
    torch.cuda.synchronize()
    assert int(_lib.item()) == pkv.DEVERR_ORDER
    _lib.zero_()


@pytest.mark.parametrize("partition", [0, 64])
@pytest.mark.parametrize("block", [16, 32])
def test_bad_block_and_context_are_reported(block, partition, _lib):
    c = AnyCache([100, 90], 2, 128, block, "fp4", seed=5)
    q = queries(2, 4, 128, seed=5)
    keep = c.tables.clone()
    for bad in (-1, c.k.shape[0], 1 << 30):
        c.tables[1, 1] = bad
        out = call(c, q, 0.1, partition)
        torch.cuda.synchronize()
        assert int(_lib.item()) == pkv.DEVERR_BLOCK_ID
        _lib.zero_()
        verify(c, q, out, 0.1, "the other", skip=(1,))
    c.tables.copy_(keep)
    for bad in (-3, 1 << 20):
        lens = c.context_lens.clone()
        c.context_lens[1] = bad
        out = call(c, q, 0.1, partition)
        torch.cuda.synchronize()
        assert int(_lib.item()) in (pkv.DEVERR_CONTEXT, pkv.DEVERR_BLOCK_ID)
        _lib.zero_()
        c.context_lens.copy_(lens)
        verify(c, q, out, 0.1, "the other", skip=(1,))


@pytest.mark.parametrize("partition", [0, 64, None])
@pytest.mark.parametrize("d", [128, 256])
def test_repeats_streams_and_graphs(d, partition, _lib):
    c = AnyCache([2000, 64, 700, 9], 2, d, 16, "fp4", seed=21)
    q = queries(4, 8, d, seed=21)
    if partition is None:
        partition = pkv.decode_partition_size(4, 2, d, 16, 2000, pkv.PKV_DTYPE_FP4_E2M1)
    n = pkv.decode_workspace_bytes(4, 8, d, 2000, partition)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda").fill_(0xFF)
    out = torch.empty_like(q)

    def go(stream=None):
        call(c, q, 0.0625, partition, out=out, workspace=ws, stream=stream)

    go()
    first = out.clone()
    verify(c, q, first, 0.0625, "first")
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
    mine = call(c, q, 0.0625, partition, stream=side)
    side.synchronize()
    assert torch.equal(mine, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    out.zero_()
    graph.replay()
    assert torch.equal(out, first)
    q.copy_(queries(4, 8, d, seed=22))
    graph.replay()
    verify(c, q, out, 0.0625, "replay")
    # other lengths in the same graph
    c.context_lens.copy_((c.context_lens + 1) // 2)
    graph.replay()
    c.lens = c.context_lens.tolist()
    c.K, c.V = ([x[:m] for x, m in zip(y, c.lens)] for y in (c.K, c.V))
    verify(c, q, out, 0.0625, "shorter")
    assert int(_lib.item()) == 0


def test_large_pool(_lib):
    nb = (1 << 32) // (4 * 32 * 144) + 2000
    c = AnyCache([300, 77], 4, 256, 32, "fp4", seed=4, pool_blocks=nb)
    q = queries(2, 24, 256, seed=4)
    for partition in (0, 64):
        verify(c, q, call(c, q, 0.0625, partition), 0.0625, "large pool")
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_library_partition_of_other_pools(kind, _lib):
    """partition_size=None on bf16 and E4M3 pools."""
    for lens in ([40, 2000, 333, 700], [9000], [100] * 300):
        c = AnyCache(lens, 2, 128, 16, kind, seed=2)
        q = queries(len(lens), 8, 128, seed=2)
        verify(c, q, call(c, q, 0.09, None), 0.09, kind)
    assert int(_lib.item()) == 0
