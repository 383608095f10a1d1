"""Refusals of the calls on 4-bit pools and of the sparse attention's calls
(nothing reaches a device)."""
import ctypes

import pytest
import torch

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build

OK, INV, UNS = pkv.PKV_OK, pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED


def at(x):
    """An address; never dereferenced: validation fails first."""
    return ctypes.c_void_p(x)


# far apart, so that nothing overlaps
A, B, C, D, E, F, G, H = (at((i + 1) << 40) for i in range(8))
ODD = at((9 << 40) + 8)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pkv.lib()


def _desc(nb=8, bs=16, hk=2, d=128, dt=0):
    return pkv.CacheDesc(nb, bs, hk, d, dt)


@pytest.mark.parametrize("name", ["pkv_kv_cache_write", "pkv_kv_cache_read"])
def test_rows(lib, name):
    f = getattr(lib, name)

    def call(**k):
        return f(k.get("k", A), k.get("v", B), k.get("slots", C), k.get("n", 4), k.get("kc", D),
                 k.get("vc", E), k.get("desc", _desc(dt=2)), k.get("ks", F), k.get("vs", G), None)

    assert call(n=0) == OK
    for bad in (dict(n=-1), dict(k=None), dict(v=None), dict(slots=None), dict(kc=None),
                dict(vc=None), dict(ks=None), dict(vs=None), dict(k=ODD), dict(v=ODD),
                dict(kc=ODD), dict(vc=ODD), dict(desc=_desc(dt=3)), dict(desc=_desc(nb=0)),
                dict(desc=_desc(dt=1), ks=None)):
        assert call(**bad) == INV, bad
    for bad in (dict(desc=_desc(bs=8, dt=2)), dict(desc=_desc(d=64, dt=2)),
                dict(desc=_desc(hk=33, dt=2))):
        assert call(**bad) == UNS, bad
    assert call(desc=_desc(hk=32, d=256, dt=2), n=0) == OK
    if name == "pkv_kv_cache_read":
        # rows 4 x 2 x 128 x 2 bytes, pools 8 x 2 x 16 x 72
        for bad in (dict(v=at(A.value + 2032)), dict(k=at(B.value - 2032)), dict(kc=A),
                    dict(vc=at(B.value - 18416)), dict(slots=at(A.value + 8))):
            assert call(**bad) == INV, bad


def test_decode_of_4_bit_pools(lib):
    def call(f=lib.pkv_paged_attention_decode, **k):
        return f(k.get("out", A), k.get("q", B), k.get("kc", C), k.get("vc", D),
                 k.get("desc", _desc(dt=2)), k.get("ks", E), k.get("vs", F), k.get("bt", G),
                 k.get("mb", 64), k.get("lens", H), k.get("S", 4), k.get("Hq", 8),
                 k.get("maxc", 1024), k.get("scale", 0.1), k.get("P", 0), k.get("ws"),
                 k.get("wsb", 0), None, None)

    for f in (lib.pkv_paged_attention_decode, lib.pkv_paged_attention):
        assert call(f, S=0) == OK
        for bad in (dict(ks=None), dict(vs=None), dict(out=None), dict(q=None), dict(kc=None),
                    dict(bt=None), dict(lens=None), dict(q=ODD), dict(out=ODD), dict(vc=ODD),
                    dict(Hq=7), dict(maxc=1025), dict(P=24), dict(P=-16), dict(P=64),
                    dict(P=64, ws=ODD, wsb=1 << 30), dict(P=64, ws=at(1 << 45), wsb=100),
                    dict(scale=float("nan")), dict(desc=_desc(dt=3))):
            assert call(f, **bad) == INV, bad
        for bad in (dict(Hq=18), dict(S=65536), dict(mb=(1 << 26) + 1),
                    dict(desc=_desc(d=64, dt=2))):
            assert call(f, **bad) == UNS, bad


def test_calls_that_take_no_4_bit_pool(lib):
    """Window, tree, shared prefix and acceptance."""
    d = _desc(dt=2)
    assert lib.pkv_paged_attention_window(A, B, C, D, d, E, F, G, 64, H, 4, 8, 1024, 0.1, 100, 4,
                                          0, None, 0, None, None) == INV
    assert lib.pkv_paged_attention_tree(A, B, C, D, d, E, F, G, 64, H, H, 4, 12, 3, None, 8, 1024,
                                        0.1, at(1 << 45), 1 << 40, None) == INV
    assert lib.pkv_paged_attention_decode_shared_prefix(
        A, B, C, D, d, E, F, G, 64, H, 4, 8, 1024, 0.1, H, 1, 4, H, 2, 64, at(1 << 45), 1 << 40,
        None, None) == INV
    arr = ctypes.c_void_p * 1
    assert lib.pkv_kv_cache_accept(arr(A.value), arr(B.value), 1, d, G, 8, H, H, 4, H, 4, H, None,
                                   None) == INV


def test_partition_size(lib):
    f = lib.pkv_decode_partition_size
    for bad in (_desc(nb=0), _desc(dt=3)):
        assert f(bad, 4, 1000) == INV
    assert f(_desc(), -1, 1000) == INV and f(_desc(), 4, -1) == INV
    assert f(_desc(d=64), 4, 1000) == UNS and f(_desc(bs=8), 4, 1000) == UNS
    for dt in (0, 1, 2):
        for d in (128, 256):
            for b in (16, 32):
                for hk in (1, 4, 8):
                    for S in (0, 1, 7, 64, 300, 2000):
                        for n in (0, 1, 16, 700, 8192, 131072, 1 << 20, 1 << 28):
                            p = f(_desc(bs=b, hk=hk, d=d, dt=dt), S, n)
                            assert p >= 0 and p % b == 0, (dt, d, b, hk, S, n, p)
                            # the merge's bound on partitions
                            assert p == 0 or -(-n // p) <= 32767
    assert pkv.decode_partition_size(4, 2, 128, 16, 1000, pkv.PKV_DTYPE_FP4_E2M1) >= 0
    with pytest.raises(pkv.PagedKVError):
        pkv.decode_partition_size(4, 2, 100, 16, 1000)


def test_bounds(lib):
    def call(**k):
        return lib.pkv_block_bounds(
            k.get("out", A), k.get("kc", B), k.get("desc", _desc()), k.get("ks", C),
            k.get("step", D), k.get("bt", E), k.get("mb", 64), k.get("lens", F), k.get("num"),
            k.get("new", 1), k.get("S", 4), None)

    assert call(S=0) == OK and call(new=0) == OK
    for bad in (dict(out=None), dict(kc=None), dict(step=None), dict(bt=None), dict(lens=None),
                dict(out=ODD), dict(kc=ODD), dict(new=-1), dict(S=-1), dict(mb=0),
                dict(desc=_desc(dt=1), ks=None), dict(desc=_desc(dt=2), ks=None),
                dict(desc=_desc(dt=3)), dict(out=at(B.value + 65536 - 16)), dict(out=D),
                dict(out=at(E.value - 16)), dict(out=F), dict(num=at(A.value + 16)),
                dict(desc=_desc(dt=1), out=C)):
        assert call(**bad) == INV, bad
    for bad in (dict(desc=_desc(bs=8)), dict(desc=_desc(d=64)), dict(mb=(1 << 26) + 1),
                dict(desc=_desc(hk=33)), dict(S=1 << 30, mb=1 << 20, new=1 << 28), dict(S=65536)):
        assert call(**bad) == UNS, bad


def test_select(lib):
    n = lib.pkv_select_workspace_bytes(4, 2, 16, 1024)
    assert n == 4 * 2 * 64 * 4
    assert lib.pkv_select_workspace_bytes(4, 2, 16, 0) == 0
    assert lib.pkv_select_workspace_bytes(65535, 32, 16, 1 << 30) == 65535 * 32 * (1 << 26) * 4

    def call(**k):
        return lib.pkv_select_blocks(
            k.get("blocks", A), k.get("counts", B), k.get("q", C), k.get("bounds", D),
            k.get("desc", _desc()), k.get("bt", E), k.get("mb", 64), k.get("lens", F),
            k.get("S", 4), k.get("Hq", 8), k.get("maxc", 1024), k.get("take", 8),
            k.get("first", 1), k.get("last", 1), k.get("ws", G), k.get("wsb", n), None)

    assert call(S=0) == OK
    for bad in (dict(blocks=None), dict(counts=None), dict(q=None), dict(bounds=None),
                dict(bt=None), dict(lens=None), dict(ws=None), dict(wsb=n - 1), dict(ws=ODD),
                dict(q=ODD), dict(bounds=ODD), dict(take=0), dict(first=-1), dict(last=-1),
                dict(first=5, last=4), dict(first=1 << 30, last=1 << 30, take=8), dict(Hq=7),
                dict(Hq=0), dict(S=-1), dict(mb=0), dict(maxc=1025), dict(maxc=-1),
                dict(counts=A), dict(blocks=C), dict(counts=F), dict(ws=D),
                dict(ws=at(C.value - 16)), dict(blocks=at(G.value + n - 4)),
                dict(desc=_desc(nb=0))):
        assert call(**bad) == INV, bad
    for bad in (dict(Hq=18), dict(S=65536, wsb=1 << 40), dict(mb=(1 << 26) + 1),
                dict(desc=_desc(bs=8)), dict(desc=_desc(d=64))):
        assert call(**bad) == UNS, bad


def test_sparse(lib):
    def call(**k):
        return lib.pkv_paged_attention_sparse(
            k.get("out", A), k.get("q", B), k.get("kc", C), k.get("vc", D),
            k.get("desc", _desc()), k.get("ks"), k.get("vs"), k.get("bt", E), k.get("mb", 64),
            k.get("lens", F), k.get("blocks", G), k.get("counts", H), k.get("take", 8),
            k.get("S", 4), k.get("Hq", 8), k.get("scale", 0.1), k.get("ws", at(1 << 45)),
            k.get("wsb", 1 << 40), None)

    assert call(S=0) == OK
    for bad in (dict(out=None), dict(q=None), dict(kc=None), dict(vc=None), dict(bt=None),
                dict(lens=None), dict(blocks=None), dict(counts=None), dict(take=0),
                dict(take=-1), dict(out=ODD), dict(q=ODD), dict(kc=ODD), dict(out=B),
                dict(out=at(B.value + 16)), dict(desc=_desc(dt=1)), dict(desc=_desc(dt=2)),
                dict(desc=_desc(dt=3)), dict(Hq=7), dict(S=-1), dict(mb=0),
                dict(scale=float("inf"))):
        assert call(**bad) == INV, bad
    for bad in (dict(Hq=18), dict(S=65536), dict(mb=(1 << 26) + 1), dict(take=(1 << 20) + 1),
                dict(desc=_desc(d=64)), dict(desc=_desc(bs=8))):
        assert call(**bad) == UNS, bad
    for dt in (0, 1, 2):
        for take in (1, 16, 128, 5000, 1 << 20):
            desc = _desc(dt=dt, hk=1, d=256)
            need = lib.pkv_sparse_workspace_bytes(desc, 1, 4, take)
            assert need % 4 == 0
            # scratch stays small beside what the call reads
            assert need <= max(take * 16 * 256, 1 << 20)
            if need:
                k = dict(desc=desc, S=1, Hq=4, take=take, ks=F, vs=F)
                assert call(wsb=need - 1, **k) == INV and call(ws=None, **k) == INV
                assert call(ws=ODD, **k) == INV


def test_python_refusals():
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    k4 = torch.zeros(4, 2, 16, 72, dtype=torch.uint8)
    k = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    bt, n = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    one = torch.ones(2)
    slots = torch.zeros(3, dtype=torch.int64)
    rows = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    bounds = torch.zeros(4, 2, 2, 128, dtype=torch.int8)
    lists, counts = torch.zeros(2, 2, 5, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32)
    d = pkv.cache_desc(k4)
    assert (d.num_blocks, d.block_size, d.num_kv_heads, d.head_dim, d.dtype) == (4, 16, 2, 128, 2)
    assert pkv.cache_desc(torch.zeros(4, 2, 32, 144, dtype=torch.uint8)).head_dim == 256
    assert pkv.fp4_cache(3, 2, 16, 256, device="cpu").shape == (3, 2, 16, 144)
    with pytest.raises(ValueError, match="head_dim"):
        pkv.fp4_cache(3, 2, 16, 64, device="cpu")

    def refuses(match, f, *a, **kw):
        with pytest.raises(ValueError, match=match):
            f(*a, **kw)

    att = pkv.paged_attention
    refuses("CUDA", att, q, k4, k4, bt, n, 0.1, 16, 0, one, one)
    refuses("CUDA", att, q, k4, k4, bt, n, 0.1, 16, None, one, one)
    refuses("q must be", att, q[:, :, :64], k4, k4, bt, n, 0.1, 16, 0, one, one)
    refuses("v_cache has dtype", att, q, k4, k, bt, n, 0.1, 16, 0, one, one)
    refuses("k_scale has shape", att, q, k4, k4, bt, n, 0.1, 16, 0, one[:1], one)
    refuses("may not be q", att, q, k4, k4, bt, n, 0.1, 16, 0, one, one, out=q)
    refuses("seq_order has shape", att, q, k4, k4, bt, n, 0.1, 16, 0, one, one, seq_order=n[:1])
    for f in (lambda *a, **kw: pkv.kv_cache_write(rows, rows, *a, **kw), pkv.kv_cache_read):
        refuses("CUDA", f, slots, k4, k4, one, one)
        refuses("v_cache has shape", f, slots, k4, k4[:2], one, one)
        refuses("slot_mapping has dtype", f, slots.int(), k4, k4, one, one)
        refuses("slot_mapping must be", f, slots[None], k4, k4, one, one)
        refuses("k_scale has dtype", f, slots, k4, k4, one.double(), one)
    refuses("k has shape", pkv.kv_cache_write, rows[:2], rows, slots, k4, k4, one, one)
    refuses("v has dtype", pkv.kv_cache_read, slots, k4, k4, one, one, v=rows.float())
    bb = pkv.block_bounds
    refuses("CUDA", bb, bounds, k, bt, n, one)
    refuses("bounds has shape", bb, bounds[:3], k, bt, n, one)
    refuses("bounds has dtype", bb, bounds.int(), k, bt, n, one)
    refuses("step has shape", bb, bounds, k, bt, n, one[:1])
    refuses("num_new has dtype", bb, bounds, k, bt, n, one, 1, slots[:2])
    refuses("contiguous", bb, bounds, k.transpose(1, 2).contiguous().transpose(1, 2), bt, n, one)
    sel = pkv.select_blocks
    refuses("CUDA", sel, q, bounds, bt, n, 16, 32, 5)
    refuses("bounds must be", sel, q, bounds[:, :, :1], bt, n, 16, 32, 5)
    refuses("q must be", sel, q[:, :, :64], bounds, bt, n, 16, 32, 5)
    refuses("block_tables must be", sel, q[:1], bounds, bt, n, 16, 32, 5)
    refuses("blocks has shape", sel, q, bounds, bt, n, 16, 32, 5, blocks=lists[:, :, :4])
    refuses("counts has dtype", sel, q, bounds, bt, n, 16, 32, 5, counts=counts.long())
    sp = pkv.paged_attention_sparse
    refuses("CUDA", sp, q, k, k, bt, n, lists, counts, 0.1)
    refuses("one row per sequence", sp, q[:1], k, k, bt, n, lists, counts, 0.1)
    refuses("blocks has shape", sp, q, k, k, bt, n, lists[:, :1], counts, 0.1)
    refuses("blocks must be", sp, q, k, k, bt, n, lists[0], counts, 0.1)
    refuses("counts has shape", sp, q, k, k, bt, n, lists, counts[:1], 0.1)
    refuses("blocks has dtype", sp, q, k, k, bt, n, lists.long(), counts, 0.1)
