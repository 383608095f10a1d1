"""kv_cache_accept against the same moves on a host copy, byte for byte; the
drafting loop (append, write, tree attention, accept, truncate) against a
dense model of every sequence."""
import random

import pytest
import torch

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build as pkv_build
from _dense_side import attend, check, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.set_device_check(flag)
    yield flag
    pkv.set_device_check(None)


def pools(layers, nb, hk, b, d, fp8, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = torch.uint8 if fp8 else torch.int16
    x = [torch.randint(-128, 127, (nb, hk, b, d), device="cuda", generator=g).to(dt) * (
        1 if fp8 else 251) for _ in range(2 * layers)]
    x = [t if fp8 else t.view(torch.bfloat16) for t in x]
    return x[:layers], x[layers:]


def raw(t):
    return t if t.dtype == torch.uint8 else t.view(torch.int16)


def expected(pool, tables, lens, drafts, lists):
    """The moves on a host copy [slot][head][byte]; every row read first."""
    nb, hk, b, d = pool.shape
    flat = raw(pool).cpu().permute(0, 2, 1, 3).reshape(nb * b, hk, d).clone()
    old = flat.clone()
    for s, acc in enumerate(lists):
        base = lens[s] - drafts[s]
        for k, a in enumerate(acc):
            f, t = base + a, base + k
            flat[int(tables[s, t // b]) * b + t % b] = old[int(tables[s, f // b]) * b + f % b]
    return flat.view(nb, b, hk, d).permute(0, 2, 1, 3)


def plan(lens, b, seed, spare=2):
    rng = random.Random(seed)
    pages = [-(-n // b) for n in lens]
    ids = list(range(sum(pages) + spare))
    rng.shuffle(ids)
    t = torch.full((len(lens), max(pages) + 1), 1 << 20, dtype=torch.int32)
    at = 0
    for s, n in enumerate(pages):
        t[s, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        at += n
    return t, len(ids)


def dev32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts(drafts):
    out = [0]
    for n in drafts:
        out.append(out[-1] + n)
    return out


def run(k, v, tables, lens, drafts, lists, width=None, **kw):
    width = max([1] + [len(a) for a in lists]) if width is None else width
    acc = dev32([a + [-1] * (width - len(a)) for a in lists])
    return pkv.kv_cache_accept(k, v, tables.cuda(), dev32(lens), dev32(starts(drafts)), acc,
                               dev32([len(a) for a in lists]), **kw)


LISTS = [(40, 10, [0, 2, 5, 6]), (16, 16, []), (17, 16, [15]), (100, 64, list(range(64))),
         (64, 64, list(range(0, 64, 2))), (33, 1, [0]), (33, 1, []), (50, 0, []),
         (70, 33, [1, 2, 3, 4, 30, 32]), (130, 64, list(range(1, 64))), (90, 20, [0, 1, 2])]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hk,d,block", [(2, 128, 16), (5, 128, 32), (4, 256, 16), (1, 256, 32),
                                        (32, 128, 16)])
@pytest.mark.parametrize("layers", [1, 3])
def test_moves(hk, d, block, fp8, layers, _lib):
    lens, drafts = [a for a, _, _ in LISTS], [b for _, b, _ in LISTS]
    lists = [c for _, _, c in LISTS]
    tables, nb = plan(lens, block, 1)
    k, v = pools(layers, nb, hk, block, d, fp8, 2)
    want = [expected(t, tables, lens, drafts, lists) for t in k + v]
    new = run(k, v, tables, lens, drafts, lists)
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0
    assert new.tolist() == [n - d_ + len(a) for n, d_, a in LISTS]
    base = [n - d_ for n, d_ in zip(lens, drafts)]
    # every byte of the pool is compared, rows behind the new lengths too
    for got, w in zip(k + v, want):
        assert torch.equal(raw(got).cpu(), w)
    assert base[0] == 30


def test_long_lists_and_many_layers(_lib):
    """Lists of more than 64 moves, more than 64 layers."""
    lens, drafts = [400, 300], [390, 200]
    lists = [[i for i in range(390) if i % 5 != 1], list(range(100, 200))]
    tables, nb = plan(lens, 16, 3)
    k, v = pools(67, nb, 1, 16, 128, False, 4)
    want = [expected(t, tables, lens, drafts, lists) for t in k + v]
    run(k, v, tables, lens, drafts, lists)
    for got, w in zip(k + v, want):
        assert torch.equal(raw(got).cpu(), w)
    assert int(_lib.item()) == 0


BAD = [([0, 2, 2], "equal"), ([0, 3, 1], "falling"), ([0, 8], "behind the drafts"),
       ([-1, 2], "negative")]


@pytest.mark.parametrize("bad,why", BAD)
def test_bad_lists_move_nothing(bad, why, _lib):
    lens, drafts = [40, 50], [8, 8]
    tables, nb = plan(lens, 16, 5)
    k, v = pools(1, nb, 2, 16, 128, False, 6)
    lists = [bad, [1, 3]]
    want = expected(k[0], tables, lens, drafts, [[], [1, 3]])
    new = run(k, v, tables, lens, drafts, lists)
    torch.cuda.synchronize()
    assert int(_lib.item()) == pkv.DEVERR_DRAFT, why
    _lib.zero_()
    assert torch.equal(raw(k[0]).cpu(), want)
    assert new.tolist() == [32, 44]


def test_bad_numbers_move_nothing(_lib):
    lens, drafts = [40, 50], [8, 8]
    tables, nb = plan(lens, 16, 5)
    k, v = pools(1, nb, 2, 16, 128, False, 6)
    before = raw(k[0]).clone()
    acc = dev32([[0, 2, 4], [1, 3, 5]])
    for count, lens2, codes in (([4, 0], lens, pkv.DEVERR_DRAFT), ([-1, 0], lens, pkv.DEVERR_DRAFT),
                                ([2, 0], [5, 50], pkv.DEVERR_DRAFT),
                                ([2, 0], [10 ** 6, 50], pkv.DEVERR_CONTEXT),
                                ([2, 0], [-4, 50], pkv.DEVERR_CONTEXT)):
        new = pkv.kv_cache_accept(k, v, tables.cuda(), dev32(lens2), dev32([0, 8, 16]), acc,
                                  dev32(count))
        torch.cuda.synchronize()
        assert int(_lib.item()) == codes
        _lib.zero_()
        assert torch.equal(raw(k[0]), before)
        assert new.tolist()[1] == 42
        assert new.tolist()[0] == (32 if lens2 is lens else lens2[0])


def test_bad_block_is_skipped(_lib):
    lens, drafts = [40, 50], [8, 8]
    tables, nb = plan(lens, 16, 5)
    k, v = pools(1, nb, 2, 16, 128, False, 6)
    want = expected(k[0], tables, lens, drafts, [[], [1, 3]])
    broken = tables.clone()
    broken[0, 2] = nb
    run(k, v, broken, lens, drafts, [[2, 3], [1, 3]])
    torch.cuda.synchronize()
    assert int(_lib.item()) == pkv.DEVERR_BLOCK_ID
    _lib.zero_()
    assert torch.equal(raw(k[0]).cpu(), want)


def test_streams_and_graphs(_lib):
    lens, drafts, lists = [40, 50], [8, 8], [[0, 2, 5], [1, 3]]
    tables, nb = plan(lens, 16, 5)
    k, v = pools(2, nb, 2, 16, 128, False, 6)
    want = [expected(t, tables, lens, drafts, lists) for t in k + v]
    keep = [t.clone() for t in k + v]
    dt, dl, ds = tables.cuda(), dev32(lens), dev32(starts(drafts))
    acc, cnt, new = dev32([[0, 2, 5], [1, 3, 0]]), dev32([3, 2]), dev32([0, 0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    pkv.kv_cache_accept(k, v, dt, dl, ds, acc, cnt, new, stream=side)
    side.synchronize()
    for got, w in zip(k + v, want):
        assert torch.equal(raw(got).cpu(), w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.kv_cache_accept(k, v, dt, dl, ds, acc, cnt, new)
    for t, o in zip(k + v, keep):
        t.copy_(o)
    new.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for got, w in zip(k + v, want):
        assert torch.equal(raw(got).cpu(), w)
    assert new.tolist() == [35, 44]
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_drafting_loop(fp8, _lib):
    """Several steps of drafting over two layers: fork, append with
    copy-on-write, cache write, tree attention in each layer, accept in both
    at once, truncate, and a window decode of the result; every output is
    checked against a dense model of the sequences."""
    rng = random.Random(11)
    hk, g, d, b, layers = 2, 4, 128, 16, 2
    alloc = pkv.BlockAllocator(256, b, seed=3)
    dt = torch.uint8 if fp8 else torch.bfloat16
    k = [torch.zeros(256, hk, b, d, dtype=dt, device="cuda") for _ in range(layers)]
    v = [torch.zeros_like(k[0]) for _ in range(layers)]
    ks = vs = None
    if fp8:
        ks = torch.tensor([0.01, 0.02], device="cuda")
        vs = torch.tensor([0.015, 0.01], device="cuda")

    def stored(x, scale):
        if not fp8:
            return x.double()
        return (x.float() / scale[:, None]).to(torch.float8_e4m3fn).double() * scale.double()[:, None]

    def write(seq, n, seed):
        """Append n tokens and store their rows; the dense rows per layer."""
        slots, pairs = alloc.append(seq, n)
        if len(pairs):
            for i in range(layers):
                pkv.copy_blocks(k[i], v[i], torch.as_tensor(pairs, device="cuda"))
        rows = []
        for i in range(layers):
            a, c = queries(n, hk, d, seed + 10 * i, std=1), queries(n, hk, d, seed + 10 * i + 5, std=1)
            pkv.kv_cache_write(a, c, torch.as_tensor(slots, device="cuda"), k[i], v[i], ks, vs)
            rows.append((stored(a, ks), stored(c, vs)))
        return rows

    seqs, dense = [], []
    for i, n in enumerate((37, 5, 130)):
        seqs.append(alloc.new_seq())
        dense.append(write(seqs[i], n, 1000 + i))
    seqs.append(alloc.fork(seqs[0]))
    dense.append(list(dense[0]))
    for step in range(4):
        drafts = [rng.randint(1, 12) for _ in seqs]
        rows = [write(q, n, 100 * step + 7 * i) for i, (q, n) in enumerate(zip(seqs, drafts))]
        start = starts(drafts)
        masks, lists = [], []
        for n in drafts:
            mine = []
            for i in range(n):
                mine.append((mine[rng.randint(max(0, i - 3), i - 1)] if i else 0) | (1 << i))
            masks += mine
            leaf = rng.randint(0, n - 1)
            path = [i for i in range(n) if (mine[leaf] >> i) & 1]
            lists.append(path[:rng.randint(0, len(path))])
        lens = [alloc.seq_len(q) for q in seqs]
        tables = torch.as_tensor(alloc.block_tables(seqs, 32), device="cuda")
        clens, cstart = dev32(lens), dev32(start)
        mask = torch.tensor(masks, dtype=torch.int64, device="cuda")
        for layer in range(layers):
            q = queries(start[-1], hk * g, d, step * 3 + layer)
            out = pkv.paged_attention_tree(q, k[layer], v[layer], tables, clens, cstart, 0.1,
                                           max(lens), max(drafts), mask, k_scale=ks, v_scale=vs)
            for s, n in enumerate(drafts):
                K = torch.cat([dense[s][layer][0], rows[s][layer][0]])
                V = torch.cat([dense[s][layer][1], rows[s][layer][1]])
                see = torch.ones(n, lens[s], dtype=torch.bool)
                for i in range(n):
                    for c in range(n):
                        see[i, lens[s] - n + c] = bool((masks[start[s] + i] >> c) & 1)
                want, tol = attend(q[start[s]:start[s + 1]], K, V, see.cuda(), 0.1)
                check(out[start[s]:start[s + 1]], want, tol, "step %d layer %d" % (step, layer))
        width = max([1] + [len(a) for a in lists])
        new = pkv.kv_cache_accept(k, v, tables, clens, cstart,
                                  dev32([a + [0] * (width - len(a)) for a in lists]),
                                  dev32([len(a) for a in lists]))
        for s, acc in enumerate(lists):
            pick = torch.tensor(acc, dtype=torch.long, device="cuda")
            dense[s] = [(torch.cat([dk, rk[pick]]), torch.cat([dv, rv[pick]]))
                        for (dk, dv), (rk, rv) in zip(dense[s], rows[s])]
            alloc.truncate(seqs[s], dense[s][0][0].shape[0])
        assert new.tolist() == [alloc.seq_len(q) for q in seqs]
        q = queries(len(seqs), hk * g, d, step)
        tables = torch.as_tensor(alloc.block_tables(seqs, 32), device="cuda")
        out = pkv.paged_attention_window(q, k[1], v[1], tables, new, 0.1, max(new.tolist()), 30,
                                         3, k_scale=ks, v_scale=vs)
        for s in range(len(seqs)):
            K, V = dense[s][1]
            n = K.shape[0]
            t = torch.arange(n, device="cuda")
            want, tol = attend(q[s:s + 1], K, V, ((t < 3) | (t >= n - 30))[None], 0.1)
            check(out[s:s + 1], want, tol, "window, step %d" % step)
    assert int(_lib.item()) == 0
