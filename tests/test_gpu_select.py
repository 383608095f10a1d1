"""select_blocks against the definition in whole numbers: lists and counts are
equal, ties included."""
import pytest
import torch

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build as pkv_build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.set_device_check(flag)
    yield flag
    pkv.set_device_check(None)


class Case:
    def __init__(self, lens, hk, g, d, block, seed, spread=127, nb=None):
        r = torch.Generator(device="cuda")
        r.manual_seed(seed)
        self.lens, self.hk, self.g, self.d, self.block = list(lens), hk, g, d, block
        pages = [-(-n // block) for n in self.lens]
        total = sum(pages) + 3
        nb = total if nb is None else nb
        ids = nb - total + torch.randperm(total, device="cuda", generator=r)
        self.tables = torch.full((len(self.lens), max([1] + pages) + 2), nb + 5,
                                 dtype=torch.int32, device="cuda")
        at = 0
        for s, n in enumerate(pages):
            self.tables[s, :n] = ids[at:at + n].int()
            at += n
        self.context_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.bounds = torch.empty(nb, hk, 2, d, dtype=torch.int8, device="cuda")
        b = torch.randint(-spread, spread + 1, (total, hk, 2, d), device="cuda", generator=r)
        self.bounds[ids] = b.sort(2).values.to(torch.int8)
        self.q = torch.randn(len(self.lens), hk * g, d, device="cuda",
                             generator=r).to(torch.bfloat16)
        self.max_context = max([0] + self.lens)

    def scores(self, s):
        n = -(-self.lens[s] // self.block)
        q = self.q[s].double().view(self.hk, self.g, self.d)
        top = q.abs().amax((1, 2), keepdim=True)
        code = torch.where(top > 0, torch.round(q * 127 / top), torch.zeros_like(q))
        b = self.bounds[self.tables[s, :n].long()].double()
        both = code[None, ..., None] * b.transpose(2, 3)[:, :, None]
        return both.amax(-1).sum((2, 3)).T.long().cpu()  # [Hk, n]

    def want(self, s, take, first, last, scores=None):
        n = -(-self.lens[s] // self.block)
        scores = self.scores(s) if scores is None else scores
        out = []
        for h in range(self.hk):
            if n <= take:
                got = list(range(n))
            else:
                row = scores[h].tolist()
                mid = sorted(range(first, n - last), key=lambda i: (-row[i], i))
                got = sorted(list(range(first)) + mid[:take - first - last]
                             + list(range(n - last, n)))
            out.append(got + [-1] * (take - len(got)))
        return out, [min(n, take)] * self.hk

    def call(self, take, first, last, **kw):
        return pkv.select_blocks(self.q, self.bounds, self.tables, self.context_lens, self.block,
                                 self.max_context, take, first, last, **kw)

    def verify(self, got, take, first, last, skip=()):
        blocks, counts = got[0].tolist(), got[1].tolist()
        for s in range(len(self.lens)):
            if s in skip:
                continue
            b, c = self.want(s, take, first, last)
            assert counts[s] == c, s
            assert blocks[s] == b, s


LENS = [0, 1, 16, 17, 33, 100, 257, 500, 1000, 2047, 4096, 5001]


@pytest.mark.parametrize("take,first,last", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (2, 1, 1),
                                             (8, 1, 2), (31, 0, 0), (64, 3, 5), (500, 1, 1)])
@pytest.mark.parametrize("d,block,hk,g", [(128, 16, 2, 4), (256, 32, 3, 6), (128, 32, 1, 1),
                                          (256, 16, 8, 8)])
def test_the_definition(d, block, hk, g, take, first, last, _lib):
    c = Case(LENS, hk, g, d, block, seed=take + d)
    c.verify(c.call(take, first, last), take, first, last)
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("spread", [0, 1])
def test_ties_go_to_the_lowest(spread, _lib):
    """Few values of the bounds: most scores are equal to others."""
    for n in (3000, 70000):
        c = Case([n, n // 3], 2, 1, 128, 16, seed=spread, spread=spread)
        # and a query of one channel: a handful of different scores
        c.q.zero_()
        c.q[:, 0, 5] = 1.0
        c.q[0, 1, 7] = -2.0
        for take, first, last in ((7, 0, 0), (64, 1, 2), (150, 0, 0)):
            c.verify(c.call(take, first, last), take, first, last)
    assert int(_lib.item()) == 0


def test_long_contexts(_lib):
    """More blocks than one CTA's shared memory holds, and the largest scores."""
    c = Case([900000, 50000], 1, 8, 128, 16, seed=3)
    for take in (2, 300, 40000):
        c.verify(c.call(take, 1, 1), take, 1, 1)
    c = Case([4000], 2, 8, 256, 16, seed=4)
    c.q[:] = 3.0
    c.q[:, :, ::2] = -3.0
    c.bounds[..., 0, :] = -127
    c.bounds[..., 1, :] = 127
    c.bounds[int(c.tables[0, 77]), 0, 1, 1] = 126
    c.verify(c.call(100, 0, 0), 100, 0, 0)
    c.bounds[..., 0, :], c.bounds[..., 1, :] = 127, -127
    c.verify(c.call(100, 0, 0), 100, 0, 0)
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("hk,g,d,lens,take", [
    (32, 8, 128, [3000, 40], 50), (32, 1, 256, [900] * 3, 10), (8, 4, 128, [4096] * 260, 40),
    (4, 6, 256, [70000] * 3, 900), (1, 2, 128, [100] * 400, 6), (2, 4, 128, [5000], 100000)])
def test_many_heads_blocks_and_sequences(hk, g, d, lens, take, _lib):
    c = Case(lens, hk, g, d, 16, seed=take)
    got = c.call(take, 1, 1)
    c.verify(got, take, 1, 1, skip=[s for s in range(len(lens)) if len(lens) > 100 and s % 41])
    # the lists of sequences that were skipped above: ascending, the ends among them
    n = (c.context_lens.long() + 15) // 16
    m = n.clamp(max=take)
    blocks = got[0].long()
    i = torch.arange(take, device="cuda")
    inside = i < m[:, None, None]
    assert torch.equal(blocks >= 0, inside.expand_as(blocks))
    step = blocks[..., 1:] - blocks[..., :-1]
    assert bool(((step > 0) | ~inside[..., 1:]).all())
    assert int(_lib.item()) == 0


def test_queries_of_any_size(_lib):
    """Zero, tiny and huge queries; elements that are exact halves of a step."""
    c = Case([2000] * 5, 2, 4, 128, 16, seed=6)
    c.q[0] = 0
    c.q[1] = (c.q[1].float() * 1e-38).to(torch.bfloat16)
    c.q[2] = (c.q[2].float() * 1e35).to(torch.bfloat16)
    c.q[3] = torch.randint(-254, 255, c.q[3].shape, device="cuda").to(torch.bfloat16)
    c.q[3, :, 0] = 254
    c.verify(c.call(20, 1, 1), 20, 1, 1)
    # not finite: some choice, and the others' as ever
    c.q[4, 0, 0] = float("nan")
    c.q[4, 5, 3] = float("inf")
    got = c.call(20, 1, 1)
    c.verify(got, 20, 1, 1, skip=(4,))
    for row in got[0][4].tolist():
        assert row == sorted(set(row)) and row[0] == 0 and row[-1] == 124 and len(row) == 20


def test_bad_blocks_and_contexts_are_reported(_lib):
    c = Case([1000, 1600], 2, 3, 128, 16, seed=8)
    for bad in (-1, c.bounds.shape[0]):
        keep = int(c.tables[1, 50])
        c.tables[1, 50] = bad
        got = c.call(99, 0, 0)
        torch.cuda.synchronize()
        assert int(_lib.item()) == pkv.DEVERR_BLOCK_ID
        _lib.zero_()
        # the one block of 100 that is not chosen
        assert got[0][1].tolist() == [[i for i in range(100) if i != 50]] * 2
        c.verify(got, 99, 0, 0, skip=(1,))
        c.tables[1, 50] = keep
    lens = c.context_lens.clone()
    for bad in (-5, 1601):
        c.context_lens[1] = bad
        got = c.call(20, 1, 1)
        torch.cuda.synchronize()
        assert int(_lib.item()) == pkv.DEVERR_CONTEXT
        _lib.zero_()
        c.verify(got, 20, 1, 1, skip=(1,))
        if bad < 0:
            assert got[1][1].tolist() == [0, 0] and int(got[0][1].max()) == -1
        c.context_lens.copy_(lens)
    c.verify(c.call(20, 1, 1), 20, 1, 1)


def test_bad_contexts_are_reported_where_all_blocks_are_chosen(_lib):
    c = Case([1600, 1500], 2, 4, 128, 16, seed=12)
    for bad in (-1, 1601):
        c.context_lens[1] = bad
        got = c.call(100, 1, 1)
        torch.cuda.synchronize()
        assert int(_lib.item()) == pkv.DEVERR_CONTEXT
        _lib.zero_()
        assert got[1].tolist() == [[100, 100], [0, 0] if bad < 0 else [100, 100]]


def test_streams_graphs_and_given_buffers(_lib):
    c = Case([4000, 70, 900], 2, 4, 256, 16, seed=9)
    blocks = torch.full((3, 2, 30), 7, dtype=torch.int32, device="cuda")
    counts = torch.full((3, 2), 7, dtype=torch.int32, device="cuda")
    n = pkv.select_workspace_bytes(3, 2, 16, 4000)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
    got = c.call(30, 1, 1, blocks=blocks, counts=counts, workspace=ws)
    assert got[0] is blocks and got[1] is counts
    c.verify(got, 30, 1, 1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    mine = c.call(30, 1, 1, stream=side)
    side.synchronize()
    assert torch.equal(mine[0], blocks) and torch.equal(mine[1], counts)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(30, 1, 1, blocks=blocks, counts=counts, workspace=ws)
    c.q.copy_(torch.randn(c.q.shape, device="cuda"))
    blocks.zero_()
    graph.replay()
    c.verify((blocks, counts), 30, 1, 1)
    assert int(_lib.item()) == 0


def test_large_pool(_lib):
    nb = (1 << 32) // (8 * 2 * 256) + 100
    c = Case([2000, 77], 8, 2, 256, 16, seed=10, nb=nb)
    c.verify(c.call(25, 1, 1), 25, 1, 1)
    assert int(_lib.item()) == 0
