"""Refusals of the window, tree and accept calls (nothing reaches a device),
and the allocator's truncate."""
import ctypes
import random

import pytest
import torch

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build

FAKE = ctypes.c_void_p(0x10000)      # never dereferenced: validation fails first
OTHER = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10008)
OK, INV, UNS = pkv.PKV_OK, pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pkv.lib()


def _desc(nb=8, bs=16, hk=2, d=128, dt=0):
    return pkv.CacheDesc(nb, bs, hk, d, dt)


def test_window_refusals(lib):
    f = lib.pkv_paged_attention_window

    def call(**k):
        return f(k.get("out", OTHER), k.get("q", FAKE), k.get("k", FAKE), FAKE,
                 k.get("desc", _desc()), k.get("ks"), k.get("vs"), k.get("bt", FAKE),
                 k.get("mb", 64), FAKE, k.get("S", 4), k.get("Hq", 8), k.get("maxc", 1024),
                 k.get("scale", 0.088), k.get("win", 100), k.get("sinks", 4), k.get("P", 64),
                 k.get("ws"), k.get("wsb", 0), None, None)

    assert call(S=0) == OK
    for bad in (dict(win=0), dict(win=-1), dict(sinks=-1), dict(P=-16), dict(P=24), dict(S=-1),
                dict(Hq=7), dict(Hq=0), dict(maxc=1025), dict(maxc=-1), dict(mb=0),
                dict(scale=float("inf")), dict(out=None), dict(q=None), dict(k=None),
                dict(bt=None), dict(out=FAKE), dict(q=ODD), dict(out=ODD), dict(k=ODD),
                dict(desc=_desc(dt=1)), dict(desc=_desc(dt=2)), dict(desc=_desc(nb=0)),
                dict(P=16, ws=None), dict(P=16, ws=FAKE, wsb=16),
                dict(P=16, ws=ODD, wsb=1 << 30)):
        assert call(**bad) == INV, bad
    for bad in (dict(Hq=18), dict(desc=_desc(bs=8)), dict(desc=_desc(d=64)), dict(S=65536),
                dict(desc=_desc(nb=1 << 27)), dict(mb=1 << 28)):
        assert call(**bad) == UNS, bad


def test_window_sizes(lib):
    f = lib.pkv_window_partition_size
    assert f(4, 2, 128, 16, 1024, 0, 0) == INV and f(4, 2, 128, 8, 1024, 10, 0) == INV
    assert f(4, 2, 128, 16, 1024, 10, -1) == INV and f(-1, 2, 128, 16, 1024, 10, 0) == INV
    assert f(4, 2, 64, 16, 1024, 10, 0) == UNS
    for S in (1, 7, 64, 300):
        for hk in (1, 4, 8):
            for b in (16, 32):
                for maxc in (0, 1, 700, 8192, 131072, 1 << 20):
                    for win, sinks in ((1, 0), (512, 4), (4096, 4), (1 << 30, 1 << 30)):
                        p = f(S, hk, 128, b, maxc, win, sinks)
                        assert p >= 0 and p % b == 0
                        n = lib.pkv_window_workspace_bytes(S, 4 * hk, 128, b, maxc, win, sinks, p)
                        assert (n == 0) if p == 0 else (n % (130 * 4) == 0)
                        # scratch stays small beside what the call reads
                        seen = min(maxc, win + sinks) + 2 * b
                        assert n <= max(S * hk * seen * 128 * 2 * 2, 1 << 20)


def test_tree_refusals(lib):
    f = lib.pkv_paged_attention_tree

    def call(**k):
        return f(k.get("out", OTHER), k.get("q", FAKE), k.get("k", FAKE), FAKE,
                 k.get("desc", _desc()), k.get("ks"), k.get("vs"), k.get("bt", FAKE),
                 k.get("mb", 64), FAKE, k.get("start", FAKE), k.get("S", 4), k.get("N", 12),
                 k.get("draft", 3), k.get("mask"), k.get("Hq", 8), k.get("maxc", 1024),
                 k.get("scale", 0.088), k.get("ws"), k.get("wsb", 0), None)

    assert call(S=0) == OK and call(N=0) == OK
    for bad in (dict(draft=0), dict(draft=65), dict(N=-1), dict(S=-1), dict(start=None),
                dict(Hq=7), dict(maxc=1025), dict(mb=0), dict(scale=float("nan")),
                dict(out=None), dict(q=None), dict(k=None), dict(bt=None), dict(out=FAKE),
                dict(q=ODD), dict(out=ODD), dict(k=ODD), dict(desc=_desc(dt=1)),
                dict(ws=FAKE, wsb=16), dict(ws=ODD, wsb=1 << 30), dict(ws=None)):
        assert call(**bad) == INV, bad
    for bad in (dict(Hq=18), dict(desc=_desc(bs=8)), dict(desc=_desc(d=64)), dict(S=65536),
                dict(desc=_desc(nb=1 << 27)), dict(mb=1 << 28)):
        assert call(**bad) == UNS, bad


def test_accept_refusals(lib):
    f = lib.pkv_kv_cache_accept
    arr = ctypes.c_void_p * 2

    def call(**k):
        return f(k.get("kp", arr(0x10000, 0x20000)), k.get("vp", arr(0x30000, 0x40000)),
                 k.get("L", 2), k.get("desc", _desc()), k.get("bt", FAKE), k.get("mb", 8),
                 k.get("lens", FAKE), k.get("start", FAKE), k.get("S", 4), k.get("acc", FAKE),
                 k.get("M", 4), k.get("cnt", FAKE), k.get("new"), None)

    assert call(S=0) == OK
    for bad in (dict(L=0), dict(S=-1), dict(mb=0), dict(M=-1), dict(kp=None), dict(vp=None),
                dict(bt=None), dict(lens=None), dict(start=None), dict(acc=None),
                dict(cnt=None), dict(new=FAKE), dict(kp=arr(0x10000, 0)),
                dict(vp=arr(0x10008, 0x20000)), dict(desc=_desc(nb=0))):
        assert call(**bad) == INV, bad
    assert call(desc=_desc(bs=8)) == UNS and call(desc=_desc(hk=33)) == UNS


def test_python_refusals():
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    k = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    bt, n = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    start = torch.arange(3, dtype=torch.int32)
    win = pkv.paged_attention_window
    with pytest.raises(ValueError, match="CUDA"):
        win(q, k, k, bt, n, 0.1, 16, 4, partition_size=0)
    with pytest.raises(ValueError, match="one row per sequence"):
        win(q[:1], k, k, bt, n, 0.1, 16, 4)
    with pytest.raises(ValueError, match="may not be q"):
        win(q, k, k, bt, n, 0.1, 16, 4, out=q)
    with pytest.raises(ValueError, match="contiguous"):
        win(q, k.transpose(2, 3).contiguous().transpose(2, 3), k, bt, n, 0.1, 16, 4)
    with pytest.raises(ValueError, match="v_cache has dtype"):
        win(q, k, k.float(), bt, n, 0.1, 16, 4)
    with pytest.raises(ValueError, match="v_cache has shape"):
        win(q, k, k[:2], bt, n, 0.1, 16, 4)
    with pytest.raises(ValueError, match="context_lens has shape"):
        win(q, k, k, bt, n[:1], 0.1, 16, 4)
    with pytest.raises(ValueError, match="context_lens must be a tensor"):
        pkv.kv_cache_accept(k, k.clone(), bt, [1, 1], start, torch.zeros(2, 3, dtype=torch.int32), n)
    with pytest.raises(ValueError, match="q must be"):
        win(q[:, :, :64], k, k, bt, n, 0.1, 16, 4)
    with pytest.raises(ValueError, match="q_start has shape"):
        pkv.paged_attention_tree(q, k, k, bt, n, start[:2], 0.1, 16, 4)
    with pytest.raises(ValueError, match="tree_mask has dtype"):
        pkv.paged_attention_tree(q, k, k, bt, n, start, 0.1, 16, 4, n)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_attention_tree(q, k, k, bt, n, start, 0.1, 16, 4)
    acc = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="equally many"):
        pkv.kv_cache_accept([k], [k, k], bt, n, start, acc, n)
    with pytest.raises(ValueError, match="equally many"):
        pkv.kv_cache_accept([], [], bt, n, start, acc, n)
    with pytest.raises(ValueError, match="v_caches has shape"):
        pkv.kv_cache_accept(k, k[:2], bt, n, start, acc, n)
    with pytest.raises(ValueError, match="new_context_lens may not be"):
        pkv.kv_cache_accept(k, k.clone(), bt, n, start, acc, n, n)
    with pytest.raises(ValueError, match="num_accepted has shape"):
        pkv.kv_cache_accept(k, k.clone(), bt, n, start, acc, n[:1])


def test_truncate_gives_blocks_back(lib):
    a = pkv.BlockAllocator(16, 16, seed=1)
    s = a.new_seq()
    a.append(s, 70)
    table = a.block_table(s).tolist()
    a.truncate(s, 70)
    assert a.block_table(s).tolist() == table and a.seq_len(s) == 70
    a.truncate(s, 33)
    assert a.block_table(s).tolist() == table[:3]
    assert a.stats() == {"free_blocks": 13, "used_blocks": 3, "used_slots": 33}
    slots, pairs = a.append(s, 20)
    assert slots[0] == table[2] * 16 + 1 and len(pairs) == 0
    # the earliest block given back is the first reused
    assert a.block_table(s).tolist() == table[:4]
    a.truncate(s, 0)
    assert a.stats() == {"free_blocks": 16, "used_blocks": 0, "used_slots": 0}
    a.append(s, 1)
    for bad in (-1, 2):
        with pytest.raises(pkv.PagedKVError) as e:
            a.truncate(s, bad)
        assert e.value.status == INV
    with pytest.raises(pkv.PagedKVError) as e:
        a.truncate(99, 0)
    assert e.value.status == pkv.PKV_ERR_NOT_FOUND
    assert a.seq_len(s) == 1
    assert lib.pkv_seq_truncate(None, 0, 0) == INV


def test_truncate_into_a_shared_block(lib):
    """Cut inside a block that a fork shares: the fork keeps its rows, the
    next append copies the block first."""
    a = pkv.BlockAllocator(16, 16, seed=2)
    s = a.new_seq()
    a.append(s, 32)
    f = a.fork(s)
    a.truncate(s, 20)
    assert a.stats()["used_slots"] == 32 and a.refcount(int(a.block_table(f)[1])) == 2
    slots, pairs = a.append(s, 1)
    assert pairs.tolist() == [[int(a.block_table(f)[1]), int(a.block_table(s)[1])]]
    assert slots[0] == int(a.block_table(s)[1]) * 16 + 4
    assert a.stats()["used_slots"] == 16 + 16 + 5
    # the other way round: the longer holder leaves, the cut one writes on in place
    b = a.fork(s)
    a.truncate(b, 18)
    a.free(s)
    assert a.stats()["used_slots"] == 16 + 16 + 2
    slots, pairs = a.append(b, 14)
    assert len(pairs) == 0 and a.stats()["used_slots"] == 48
    assert pkv.BlockAllocator.load(a.save()).stats() == a.stats()


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_truncate_against_a_model(seed, lib):
    """Random appends, forks, cuts, frees and checkpoints against a model that
    holds every sequence's tokens, block copies applied to its slots."""
    rng = random.Random(seed)
    nb, b = 48, 16
    a = pkv.BlockAllocator(nb, b, seed=seed)
    slot = {}
    seqs = {}
    token = 0
    for step in range(1500):
        op = rng.random()
        if op < 0.12 or not seqs:
            seqs[a.new_seq()] = []
        elif op < 0.6:
            s = rng.choice(list(seqs))
            n = rng.randint(1, 24)
            try:
                slots, pairs = a.append(s, n)
            except pkv.PagedKVError as e:
                assert e.status == pkv.PKV_ERR_OUT_OF_BLOCKS
                continue
            for src, dst in pairs.tolist():
                for i in range(b):
                    slot[dst * b + i] = slot.get(src * b + i)
            for x in slots.tolist():
                slot[x] = token
                seqs[s].append(token)
                token += 1
        elif op < 0.7:
            s = rng.choice(list(seqs))
            seqs[a.fork(s)] = list(seqs[s])
        elif op < 0.9:
            s = rng.choice(list(seqs))
            n = rng.randint(0, len(seqs[s]))
            a.truncate(s, n)
            del seqs[s][n:]
        elif op < 0.97:
            s = rng.choice(list(seqs))
            a.free(s)
            del seqs[s]
        else:
            a = pkv.BlockAllocator.load(a.save())
        used, held = {}, {}
        for s, tokens in seqs.items():
            assert a.seq_len(s) == len(tokens)
            t = a.block_table(s).tolist()
            assert len(t) == -(-len(tokens) // b)
            for x in t:
                held[x] = held.get(x, 0) + 1
            for i, x in enumerate(tokens):
                at = t[i // b] * b + i % b
                assert slot[at] == x
                used[at] = 1
        st = a.stats()
        assert st == {"free_blocks": nb - len(held), "used_blocks": len(held),
                      "used_slots": len(used)}
        for x, n in held.items():
            assert a.refcount(x) == n
