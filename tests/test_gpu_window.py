"""paged_attention_window against 64-bit attention over a dense copy of the
cache: windows and sinks of every alignment, blocks behind the window given
back, NaN in every masked slot."""
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


def visible(ctx, window, sinks):
    t = torch.arange(ctx, device="cuda")
    return (t < sinks) | (t >= ctx - window)


def hide_rest(c, window, sinks):
    """NaN into every slot that is not visible; blocks without a visible slot
    lose their table entry."""
    for s, ctx in enumerate(c.lens):
        lo = max(min(sinks, ctx), ctx - window)
        c.poison(s, min(sinks, ctx), lo) if lo > sinks else None
        first, last = -(-min(sinks, ctx) // c.block), max(0, ctx - window) // c.block
        if last > first:
            c.tables[s, first:last] = -9


def verify(c, q, out, window, sinks, scale, what):
    for s, ctx in enumerate(c.lens):
        see = visible(ctx, window, sinks)[None]
        K, V = c.K[s], c.V[s]
        want, tol = attend(q[s:s + 1], K, V, see, scale)
        check(out[s:s + 1], want, tol, "%s sequence %d" % (what, s))


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 100, 127, 128, 129, 500, 1000, 2047]


@pytest.mark.parametrize("partition", [None, 0, 32, 96, 512])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,block", [(128, 16), (128, 32), (256, 16), (256, 32)])
def test_alignments(d, block, fp8, partition, _lib):
    hk, g = 2, {128: 3, 256: 6}[d]
    q = queries(len(LENS), hk * g, d, seed=d)
    for window, sinks in ((1, 0), (1, 1), (7, 3), (16, 16), (17, 4), (33, 0), (100, 40),
                          (500, 17), (4096, 5), (128, 300)):
        c = Cache(LENS, hk, d, block, fp8, seed=window + sinks)
        hide_rest(c, window, sinks)
        out = pkv.paged_attention_window(q, c.k, c.v, c.tables, c.context_lens, d ** -0.5,
                                         c.max_context, window, sinks, partition, **c.kw())
        torch.cuda.synchronize()
        assert int(_lib.item()) == 0
        verify(c, q, out, window, sinks, d ** -0.5, "window %d sinks %d" % (window, sinks))


@pytest.mark.parametrize("g", [1, 2, 4, 5, 7, 8])
def test_query_groups(g, _lib):
    for fp8 in (False, True):
        c = Cache([40, 200, 333, 700], 3, 128, 16, fp8, seed=g)
        q = queries(4, 3 * g, 128, seed=g)
        hide_rest(c, 150, 5)
        out = pkv.paged_attention_window(q, c.k, c.v, c.tables, c.context_lens, 0.1, 700, 150, 5,
                                         **c.kw())
        verify(c, q, out, 150, 5, 0.1, "g=%d" % g)
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,window,sinks", [([60000], 50001, 77), ([30000, 9, 20000], 8192, 4),
                                               ([5000] * 20, 4000, 1),
                                               ([40000], 1 << 30, 1 << 30)])
def test_long_windows(lens, window, sinks, fp8, _lib):
    c = Cache(lens, 2, 256, 32, fp8, seed=3)
    q = queries(len(lens), 12, 256, seed=4)
    hide_rest(c, window, sinks)
    out = pkv.paged_attention_window(q, c.k, c.v, c.tables, c.context_lens, 0.0625,
                                     c.max_context, window, sinks, **c.kw())
    verify(c, q, out, window, sinks, 0.0625, "long")
    assert int(_lib.item()) == 0


def test_window_over_the_context_is_the_decode(_lib):
    c = Cache([1, 31, 500, 3000], 4, 256, 32, False, seed=12)
    q = queries(4, 24, 256, seed=12)
    want = pkv.paged_attention(q, c.k, c.v, c.tables, c.context_lens, 0.0625, 3000)
    got = pkv.paged_attention_window(q, c.k, c.v, c.tables, c.context_lens, 0.0625, 3000, 3000,
                                     7, 0)
    verify(c, q, got, 3000, 7, 0.0625, "window")
    verify(c, q, want, 3000, 7, 0.0625, "decode")


def test_orders_give_the_same_bits(_lib):
    c = Cache([40, 2000, 333, 700], 2, 256, 16, False, seed=1)
    q = queries(4, 12, 256, seed=1)
    for partition in (0, 64):
        ref = pkv.paged_attention_window(q, c.k, c.v, c.tables, c.context_lens, 0.0625, 2000,
                                         300, 4, partition)
        for order in ([3, 2, 1, 0], [1, 3, 2, 0]):
            o = torch.tensor(order, dtype=torch.int32, device="cuda")
            out = pkv.paged_attention_window(q, c.k, c.v, c.tables, c.context_lens, 0.0625, 2000,
                                             300, 4, partition, seq_order=o)
            assert torch.equal(out, ref)
    bad = torch.tensor([1, 4, 2, 0], dtype=torch.int32, device="cuda")
    pkv.paged_attention_window(q, c.k, c.v, c.tables, c.context_lens, 0.0625, 2000, 300, 4, 0,
                               seq_order=bad)
    torch.cuda.synchronize()
    assert int(_lib.item()) == pkv.DEVERR_ORDER
    _lib.zero_()


def test_bad_block_and_context_are_reported(_lib):
    c = Cache([100, 90], 2, 128, 16, False, seed=5)
    q = queries(2, 4, 128, seed=5)
    keep = c.tables.clone()
    c.tables[1, 5] = -1
    out = pkv.paged_attention_window(q, c.k, c.v, c.tables, c.context_lens, 0.1, 100, 20, 4)
    torch.cuda.synchronize()
    assert int(_lib.item()) == pkv.DEVERR_BLOCK_ID
    _lib.zero_()
    c.tables.copy_(keep)
    see = visible(100, 20, 4)[None]
    want, tol = attend(q[:1], c.K[0], c.V[0], see, 0.1)
    check(out[:1], want, tol, "the other sequence")
    lens = c.context_lens.clone()
    lens[1] = -3
    out = pkv.paged_attention_window(q, c.k, c.v, c.tables, lens, 0.1, 100, 20, 4)
    torch.cuda.synchronize()
    assert int(_lib.item()) == pkv.DEVERR_CONTEXT
    _lib.zero_()
    check(out[:1], want, tol, "the other sequence")


@pytest.mark.parametrize("partition", [0, 64, None])
@pytest.mark.parametrize("fp8", [False, True])
def test_repeats_streams_and_graphs(fp8, partition, _lib):
    c = Cache([2000, 64, 700, 9], 2, 256, 16, fp8, seed=21)
    q = queries(4, 8, 256, seed=21)
    if partition is None:
        partition = pkv.window_partition_size(4, 2, 256, 16, 2000, 600, 4)
    n = pkv.window_workspace_bytes(4, 8, 256, 16, 2000, 600, 4, partition)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda").fill_(0xFF)
    out = torch.empty_like(q)

    def go(stream=None):
        pkv.paged_attention_window(q, c.k, c.v, c.tables, c.context_lens, 0.0625, 2000, 600, 4,
                                   partition, out=out, workspace=ws, stream=stream, **c.kw())

    go()
    first = out.clone()
    verify(c, q, first, 600, 4, 0.0625, "first")
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
    mine = pkv.paged_attention_window(q, c.k, c.v, c.tables, c.context_lens, 0.0625, 2000, 600,
                                      4, partition, stream=side, **c.kw())
    side.synchronize()
    assert torch.equal(mine, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    out.zero_()
    graph.replay()
    assert torch.equal(out, first)
    q.copy_(queries(4, 8, 256, seed=22))
    graph.replay()
    verify(c, q, out, 600, 4, 0.0625, "replay")
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_large_pool(fp8, _lib):
    nb = (1 << 32) // (4 * 32 * 256) + 2000
    c = Cache([300, 77], 4, 256, 32, fp8, seed=4, pool_blocks=nb)
    q = queries(2, 24, 256, seed=4)
    hide_rest(c, 100, 3)
    out = pkv.paged_attention_window(q, c.k, c.v, c.tables, c.context_lens, 0.0625, 300, 100, 3,
                                     **c.kw())
    verify(c, q, out, 100, 3, 0.0625, "large pool")
    assert int(_lib.item()) == 0
