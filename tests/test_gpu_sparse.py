"""paged_attention_sparse against 64-bit attention over the listed blocks of a
dense copy of the cache; every other block holds NaN or has no table entry."""
import random

import pytest
import torch

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build as pkv_build
from _dense_side import attend, check, queries
from _pool_side import KINDS, AnyCache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.set_device_check(flag)
    yield flag
    pkv.set_device_check(None)


def lists_of(c, take, seed, shuffle=False, counts=None):
    """Random blocks of every context, the last one always among them: (lists as
    Python, blocks, counts); entries behind a list are out of range."""
    r = random.Random(seed)
    out = []
    for s, n in enumerate(c.lens):
        nb = -(-n // c.block)
        rows = []
        for h in range(c.hk):
            m = min(nb, take) if counts is None else min(nb, counts[s][h])
            got = sorted(r.sample(range(nb - 1), m - 1) + [nb - 1]) if m else []
            if shuffle:
                r.shuffle(got)
            rows.append(got)
        out.append(rows)
    blocks = torch.tensor([[x + [1 << 29] * (take - len(x)) for x in rows] for rows in out],
                          dtype=torch.int32, device="cuda")
    cnt = torch.tensor([[len(x) for x in rows] for rows in out], dtype=torch.int32, device="cuda")
    return out, blocks, cnt


def call(c, q, blocks, counts, scale, **kw):
    return pkv.paged_attention_sparse(q, c.k, c.v, c.tables, c.context_lens, blocks, counts, scale,
                                      **c.kw(), **kw)


def expect(c, q, lists, s, scale):
    want, tol = [], []
    g = q.shape[1] // c.hk
    for h in range(c.hk):
        t = [b * c.block + i for b in lists[s][h] for i in range(c.block)
             if b * c.block + i < c.lens[s]]
        t = torch.tensor(t, dtype=torch.long, device="cuda")
        see = torch.ones(1, len(t), dtype=torch.bool, device="cuda")
        w, e = attend(q[s:s + 1, h * g:(h + 1) * g], c.K[s][t, h:h + 1], c.V[s][t, h:h + 1], see,
                      scale)
        want.append(w)
        tol.append(e)
    return torch.cat(want, 1), torch.cat(tol, 1)


def verify(c, q, out, lists, scale, what, skip=()):
    for s in range(len(c.lens)):
        if s not in skip:
            want, tol = expect(c, q, lists, s, scale)
            check(out[s:s + 1], want, tol, "%s sequence %d" % (what, s))


def hide_rest(c, lists):
    """No table entry for a block that no head lists."""
    for s, n in enumerate(c.lens):
        used = {b for rows in lists[s] for b in rows}
        for b in range(-(-n // c.block)):
            if b not in used:
                c.tables[s, b] = -9


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 64, 100, 128, 129, 500, 1000, 2047]


@pytest.mark.parametrize("take", [1, 2, 3, 8, 33, 130])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,block", [(128, 16), (128, 32), (256, 16), (256, 32)])
def test_lengths(d, block, kind, take, _lib):
    hk, g = 2, {128: 3, 256: 6}[d]
    c = AnyCache(LENS, hk, d, block, kind, seed=take)
    q = queries(len(LENS), hk * g, d, seed=d)
    for shuffle in (False, True):
        lists, blocks, counts = lists_of(c, take, take, shuffle)
        hide_rest(c, lists)
        out = call(c, q, blocks, counts, d ** -0.5)
        torch.cuda.synchronize()
        assert int(_lib.item()) == 0
        verify(c, q, out, lists, d ** -0.5, "take %d" % take)
        c = AnyCache(LENS, hk, d, block, kind, seed=take)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("g", [1, 2, 5, 7, 8])
def test_groups_and_counts(g, kind, _lib):
    """Every head its own number of blocks, none among them."""
    lens = [40, 200, 700, 3000]
    hk = 3
    c = AnyCache(lens, hk, 128, 16, kind, seed=g)
    q = queries(4, hk * g, 128, seed=g)
    for counts in ([[0, 1, 2], [3, 0, 9], [0, 0, 0], [70, 1, 33]], [[1, 1, 1]] * 4):
        lists, blocks, cnt = lists_of(c, 70, g, counts=counts)
        out = call(c, q, blocks, cnt, 0.1)
        verify(c, q, out, lists, 0.1, "g=%d" % g)
        for s in range(4):
            for h in range(hk):
                if not lists[s][h]:
                    assert float(out[s, h * g:(h + 1) * g].abs().max()) == 0
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,take,hk,d,block", [
    ([60000], 1500, 2, 256, 32), ([30000, 9, 20000], 512, 4, 256, 16), ([5000] * 20, 100, 2, 128, 32),
    ([2000] * 300, 40, 2, 128, 16), ([120000], 5000, 1, 128, 16), ([8000] * 64, 128, 4, 256, 16)])
def test_long_and_many(lens, take, hk, d, block, kind, _lib):
    c = AnyCache(lens, hk, d, block, kind, seed=3)
    q = queries(len(lens), 6 * hk, d, seed=4)
    lists, blocks, counts = lists_of(c, take, 5)
    out = call(c, q, blocks, counts, d ** -0.5)
    assert torch.isfinite(out).all()
    verify(c, q, out, lists, d ** -0.5, "long",
           skip=[s for s in range(len(lens)) if len(lens) > 10 and s % 29])
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("kind", KINDS)
def test_all_blocks_are_the_decode(kind, _lib):
    c = AnyCache([1, 31, 500, 3000], 4, 256, 32, kind, seed=12)
    q = queries(4, 24, 256, seed=12)
    lists, blocks, counts = lists_of(c, 94, 1)
    got = call(c, q, blocks, counts, 0.0625)
    verify(c, q, got, lists, 0.0625, "sparse")
    want = pkv.paged_attention(q, c.k, c.v, c.tables, c.context_lens, 0.0625, 3000, None, **c.kw())
    # both are within the tolerance of the same numbers
    for s in range(4):
        _, tol = expect(c, q, lists, s, 0.0625)
        check(got[s:s + 1], want[s:s + 1].double(), 2 * tol, "decode")


@pytest.mark.parametrize("kind", KINDS)
def test_a_block_listed_twice_counts_twice(kind, _lib):
    c = AnyCache([500], 1, 128, 16, kind, seed=2)
    q = queries(1, 4, 128, seed=2)
    lists = [[[3, 3, 31, 7, 31, 31, 0]]]
    blocks = torch.tensor(lists, dtype=torch.int32, device="cuda")
    counts = torch.tensor([[7]], dtype=torch.int32, device="cuda")
    verify(c, q, call(c, q, blocks, counts, 0.09), lists, 0.09, "twice")
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("block,take", [(16, 5), (32, 70)])
def test_bad_entries_are_reported(block, take, kind, _lib):
    c = AnyCache([100, 3000], 2, 128, block, kind, seed=5)
    q = queries(2, 4, 128, seed=5)
    lists, blocks, counts = lists_of(c, take, 5)
    # an entry that is no block of the context adds nothing
    for bad in (-1, -(1 << 31), -(-3000 // block), 1 << 30):
        b = blocks.clone()
        b[1, 0, 2] = bad
        out = call(c, q, b, counts, 0.1)
        torch.cuda.synchronize()
        assert int(_lib.item()) == pkv.DEVERR_SELECT
        _lib.zero_()
        less = [lists[0], [lists[1][0][:2] + lists[1][0][3:], lists[1][1]]]
        verify(c, q, out, less, 0.1, "entry %d" % bad)
    for bad in (-1, take + 1, 1 << 30):
        n = counts.clone()
        n[1, 1] = bad
        out = call(c, q, blocks, n, 0.1)
        torch.cuda.synchronize()
        assert int(_lib.item()) == pkv.DEVERR_SELECT
        _lib.zero_()
        cut = [lists[0], [lists[1][0], lists[1][1] if bad > 0 else []]]
        verify(c, q, out, cut, 0.1, "count %d" % bad)
    table = c.tables.clone()
    c.tables[1, lists[1][0][1]] = c.k.shape[0]
    out = call(c, q, blocks, counts, 0.1)
    torch.cuda.synchronize()
    assert int(_lib.item()) == pkv.DEVERR_BLOCK_ID
    _lib.zero_()
    verify(c, q, out, lists, 0.1, "the other", skip=(1,))
    c.tables.copy_(table)
    lens = c.context_lens.clone()
    for bad in (-3, 1 << 20):
        c.context_lens[1] = bad
        out = call(c, q, blocks, counts, 0.1)
        torch.cuda.synchronize()
        assert int(_lib.item()) == pkv.DEVERR_CONTEXT
        _lib.zero_()
        verify(c, q, out, lists, 0.1, "the other", skip=(1,))
    c.context_lens.copy_(lens)
    verify(c, q, call(c, q, blocks, counts, 0.1), lists, 0.1, "again")
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("take", [6, 200])
def test_repeats_streams_and_graphs(take, kind, _lib):
    c = AnyCache([4000, 64, 700, 9], 2, 256, 16, kind, seed=21)
    q = queries(4, 8, 256, seed=21)
    lists, blocks, counts = lists_of(c, take, 5)
    n = pkv.sparse_workspace_bytes(c.k, 4, 8, take)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda").fill_(0xFF)
    out = torch.empty_like(q)

    def go(stream=None):
        call(c, q, blocks, counts, 0.0625, out=out, workspace=ws, stream=stream)

    go()
    first = out.clone()
    verify(c, q, first, lists, 0.0625, "first")
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
    mine = call(c, q, blocks, counts, 0.0625, stream=side)
    side.synchronize()
    assert torch.equal(mine, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    out.zero_()
    graph.replay()
    assert torch.equal(out, first)
    lists, b2, c2 = lists_of(c, take, 6)
    blocks.copy_(b2)
    counts.copy_(c2)
    q.copy_(queries(4, 8, 256, seed=22))
    graph.replay()
    verify(c, q, out, lists, 0.0625, "replay")
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("kind", KINDS)
def test_large_pool(kind, _lib):
    nb = (1 << 32) // (4 * 32 * 144) + 2000
    c = AnyCache([3000, 77], 4, 256, 32, kind, seed=4, pool_blocks=nb)
    q = queries(2, 24, 256, seed=4)
    lists, blocks, counts = lists_of(c, 20, 5)
    verify(c, q, call(c, q, blocks, counts, 0.0625), lists, 0.0625, "large pool")
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("take", [5, 1300])
def test_many_small_weights(take, kind, _lib):
    """One token with V = 0 that takes nearly all of the weight, the rest counts:
    in E4M3 and 4-bit pools the weights are 16-bit numbers."""
    n, d, b = 40001, 128, 32
    c = AnyCache([n], 1, d, b, kind, seed=1)
    c.ks.fill_(1.0)
    c.vs.fill_(1.0)
    k = torch.zeros(n, 1, d, dtype=torch.bfloat16, device="cuda")
    v = torch.full((n, 1, d), 0.75, dtype=torch.bfloat16, device="cuda")
    k[0, 0, 0], v[0] = 6.0, 0.0
    pages = c.tables[0, torch.arange(n, device="cuda") // b].long()
    pkv.kv_cache_write(k, v, pages * b + torch.arange(n, device="cuda") % b, c.k, c.v, c.ks, c.vs)
    q = torch.zeros(1, 1, d, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0] = 1.0
    lists = list(range(min(take, 1251)))
    blocks = torch.tensor([[lists + [-1] * (take - len(lists))]], dtype=torch.int32, device="cuda")
    counts = torch.tensor([[len(lists)]], dtype=torch.int32, device="cuda")
    scale = 26 * 0.6931471805599453 / 6
    out = call(c, q, blocks, counts, scale)
    m = min(n, len(lists) * b)
    w = torch.exp(q.double()[0, 0] @ k.double()[:m, 0].T * scale)
    want = (w / w.sum() @ v.double()[:m, 0]).view(1, 1, d)
    check(out, want, want.abs() * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16), "small weights")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,block", [(128, 16), (256, 32)])
def test_a_decoding_run(d, block, kind, _lib):
    """A batch decodes: the allocator hands out slots, each step writes one
    token per sequence, takes the bounds of its block, selects and attends; two
    layers share the tables, forks copy their last block, and one step is also
    replayed from a graph."""
    hk, g, take = 2, 4, 6
    a = pkv.BlockAllocator(120, block, seed=3)
    r = torch.Generator(device="cuda")
    r.manual_seed(d)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=r)  # noqa: E731
    shape = (120, hk, block, d // 16 * 9 if kind == "fp4" else d)
    dt = torch.bfloat16 if kind == "bf16" else torch.uint8
    pools = [torch.zeros(shape, dtype=dt, device="cuda") for _ in range(4)]
    bounds = [torch.zeros(120, hk, 2, d, dtype=torch.int8, device="cuda") for _ in range(2)]
    scale8 = None if kind == "bf16" else torch.full((hk,), 1 / 64, device="cuda")
    step = torch.full((hk,), 1 / 30, device="cuda")
    seqs = [a.new_seq() for _ in range(3)]
    width = 40

    def write(slots, n):
        for layer in range(2):
            pkv.kv_cache_write(randn(n, hk, d).to(torch.bfloat16), randn(n, hk, d).to(
                torch.bfloat16), slots, pools[2 * layer], pools[2 * layer + 1], scale8, scale8)

    def state():
        t = torch.full((len(seqs), width), -1, dtype=torch.int32)
        for i, s in enumerate(seqs):
            table = torch.from_numpy(a.block_table(s).copy())
            t[i, :len(table)] = table
        lens = torch.tensor([a.seq_len(s) for s in seqs], dtype=torch.int32)
        return t.cuda(), lens.cuda()

    def rows(i, layer, tables, lens):
        """Dense K and V of a sequence, through kv_cache_read in fp32's place:
        exact values of the pools."""
        n = int(lens[i])
        t = torch.arange(n, device="cuda")
        slots = tables[i, t // block].long() * block + t % block
        out = []
        for p in (pools[2 * layer], pools[2 * layer + 1]):
            if kind == "bf16":
                out.append(p[slots // block, :, slots % block].double())
            elif kind == "fp8":
                out.append(p.view(torch.float8_e4m3fn)[slots // block, :, slots % block].double()
                           / 64)
            else:
                # powers of two as scales: the bf16 that the read gives is exact
                out.append(pkv.kv_cache_read(slots, p, p, scale8, scale8)[0].double())
        return out

    for i, n in enumerate((150, 33, 400)):
        slots, _ = a.append(seqs[i], n)
        write(torch.from_numpy(slots.copy()).cuda(), n)
    seqs.append(a.fork(seqs[0]))
    new = 400
    for it in range(2 * block + 3):
        tables, lens = state()
        for layer in range(2):
            pkv.block_bounds(bounds[layer], pools[2 * layer], tables, lens, step, new,
                             k_scale=scale8)
        new = 1
        q = (2 * randn(len(seqs), hk * g, d)).to(torch.bfloat16)
        for layer in range(2):
            def attend_step():
                sel = pkv.select_blocks(q, bounds[layer], tables, lens, block, width * block,  # noqa: B023
                                        take, 1, 2)
                return sel, pkv.paged_attention_sparse(
                    q, pools[2 * layer], pools[2 * layer + 1], tables, lens, *sel, d ** -0.5,  # noqa: B023
                    k_scale=scale8, v_scale=scale8)

            sel, out = attend_step()
            if it == 5 and layer == 1:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    again = attend_step()
                graph.replay()
                assert torch.equal(again[1], out) and torch.equal(again[0][0], sel[0])
            if it % 9 and it != 2 * block + 2:
                continue
            for i in range(len(seqs)):
                n = int(lens[i])
                nb = -(-n // block)
                K, V = rows(i, layer, tables, lens)
                # the blocks' scores from the dense rows
                code = q[i].double().view(hk, g, d)
                code = torch.round(code * 127 / code.abs().amax((1, 2), keepdim=True))
                x = (K.float() / step[:, None])
                score = torch.stack([torch.stack([
                    torch.maximum(code[h] * x[b * block:(b + 1) * block, h].floor().clamp(
                        -127, 127).amin(0).double(),
                        code[h] * x[b * block:(b + 1) * block, h].ceil().clamp(
                            -127, 127).amax(0).double()).sum() for b in range(nb)])
                    for h in range(hk)]).tolist()
                for h in range(hk):
                    mid = sorted(range(1, nb - 2), key=lambda j: (-score[h][j], j))[:take - 3]
                    want = sorted([0] + mid + [nb - 2, nb - 1]) if nb > take else list(range(nb))
                    assert sel[0][i, h, :len(want)].tolist() == want
                    assert int(sel[1][i, h]) == len(want)
                    t = torch.tensor([b * block + j for b in want for j in range(block)
                                      if b * block + j < n], device="cuda")
                    see = torch.ones(1, len(t), dtype=torch.bool, device="cuda")
                    w, tol = attend(q[i:i + 1, h * g:(h + 1) * g], K[t, h:h + 1], V[t, h:h + 1],
                                    see, d ** -0.5)
                    check(out[i:i + 1, h * g:(h + 1) * g], w, tol, "step %d" % it)
        slots = []
        for s in seqs:
            at, pairs = a.append(s, 1)
            if len(pairs):
                for layer in range(2):
                    pkv.copy_blocks(pools[2 * layer], pools[2 * layer + 1],
                                    torch.from_numpy(pairs.copy()).cuda())
            slots.append(int(at[0]))
        write(torch.tensor(slots, device="cuda"), len(seqs))
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0
