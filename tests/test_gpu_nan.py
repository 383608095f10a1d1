"""A NaN in a query, or in a cached row that is seen, makes NaN of the outputs it
enters however the call is cut (clusters, single CTAs, partitions), and of no
other one. Rows without a token are zeros whatever their query holds."""
import functools

import pytest
import torch

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build as pkv_build
from _dense_side import attend, check, queries
from _pool_side import AnyCache
from test_gpu_sparse import call as sparse
from test_gpu_sparse import expect as sparse_expect
from test_gpu_sparse import lists_of

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.set_device_check(flag)
    yield flag
    pkv.set_device_check(None)
    cache_of.cache_clear()
    cache_with_bad_rows.cache_clear()


@functools.lru_cache(None)
def cache_of(lens, kind, d):
    return AnyCache(lens, 2, d, 16, kind, seed=len(lens))


@functools.lru_cache(None)
def cache_with_bad_rows(lens, kind):
    """A NaN row in the middle of the first context, and one of NaN rows alone."""
    c = AnyCache(lens, 2, 128, 16, kind, seed=len(lens))
    c.poison(0, lens[0] // 2, lens[0] // 2 + 1)
    if len(lens) > 1:
        c.poison(1, 0, lens[1])
    return c


def whole(c, q, scale, partition):
    return pkv.paged_attention(q, c.k, c.v, c.tables, c.context_lens, scale, c.max_context,
                               partition, **c.kw())


def window(c, q, scale, partition):
    """A window behind which nothing lies."""
    return pkv.paged_attention_window(q, c.k, c.v, c.tables, c.context_lens, scale,
                                      c.max_context, c.max_context + 1, 3, partition, **c.kw())


def is_nan(out):
    return bool(out.float().isnan().all())


def verify(c, q, out, scale, bad, rows):
    """Rows (s, head) of `bad` are NaN, the others of sequences `rows` attention."""
    for s in rows:
        see = torch.ones(1, c.lens[s], dtype=torch.bool, device="cuda")
        want, tol = attend(q[s:s + 1].nan_to_num(0.0), c.K[s], c.V[s], see, scale)
        keep = torch.tensor([(s, j) not in bad for j in range(q.shape[1])], device="cuda")
        check(out[s:s + 1, keep], want[:, keep], tol[:, keep], "sequence %d" % s)
        assert is_nan(out[s, ~keep]), s


# (lengths, how a pass or the partitions are cut): one sequence takes a cluster to
# a pair, hundreds one CTA each
BATCHES = [[1000], [1000] + [130] * 3, [200] * 130, [40] * 600, [1] * 3]


@pytest.mark.parametrize("partition", [0, 32, 512, None])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("call,kind", [(whole, "fp4"), (whole, "bf16"), (whole, "fp8"),
                                       (window, "bf16"), (window, "fp8")])
def test_queries(call, kind, d, partition, _lib):
    scale, hk, g = d ** -0.5, 2, 3
    for lens in BATCHES:
        n = len(lens)
        c = cache_of(tuple(lens + [0]), kind, d)
        q = queries(n + 1, hk * g, d, seed=n)
        q[0, 1, 5] = NAN          # one element of a row
        q[0, 4] = NAN             # a whole row
        q[n // 2, 2, d - 1] = NAN
        q[n] = NAN                # no token
        out = call(c, q, scale, partition)
        bad = {(0, 1), (0, 4), (n // 2, 2)}
        verify(c, q, out, scale, bad, sorted({0, n // 2, n - 1}))
        assert float(out[n].float().abs().max()) == 0
        keep = torch.ones(n + 1, hk * g, dtype=torch.bool, device="cuda")
        for s, j in bad:
            keep[s, j] = False
        assert torch.isfinite(out[keep]).all()
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("partition", [0, 32, 512, None])
@pytest.mark.parametrize("call,kind", [(whole, "fp4"), (whole, "bf16"), (whole, "fp8"),
                                       (window, "bf16"), (window, "fp8")])
def test_cached_rows(call, kind, partition, _lib):
    for lens in BATCHES:
        n = len(lens)
        c = cache_with_bad_rows(tuple(lens), kind)
        q = queries(n, 6, 128, seed=n)
        out = call(c, q, 0.09, partition)
        bad = {(s, j) for s in range(min(n, 2)) for j in range(6)}
        verify(c, q, out, 0.09, bad, sorted({0, min(1, n - 1), n - 1}))
        assert torch.isfinite(out[2:]).all()
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0


# (lengths, blocks of a list): a cluster, one CTA, partitions (for each kind of pool)
LISTS = [([1000], 40), ([700] * 130, 30), ([40] * 600, 2), ([20000, 9], 1200),
         ([30000] + [3000] * 11, 180)]


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("d", [128, 256])
def test_listed_blocks(d, kind, _lib):
    hk, g, cut = 2, 3, set()
    for lens, take in LISTS:
        n = len(lens)
        c = AnyCache(lens, hk, d, 16, kind, seed=n)
        cut.add(pkv.sparse_workspace_bytes(c.k, n, hk * g, take) > 0)
        counts = None if n == 1 else [[take, take]] * (n - 1) + [[0, 1]]
        lists, blocks, cnt = lists_of(c, take, n, counts=counts)
        q = queries(n, hk * g, d, seed=n)
        q[0, 1, 5] = NAN
        q[0, 4] = NAN
        mid = (n - 1) // 2
        q[mid, 2, 0] = NAN
        # a NaN row in the last block, which every list has
        s = min(1, n - 1)
        if n > 2:
            c.poison(s, lens[s] - 1, lens[s])
        bad = {(0, 1), (0, 4), (mid, 2)} | {(s, j) for j in range(6) if n > 2}
        if n > 1:
            q[n - 1] = NAN
            bad |= {(n - 1, j) for j in range(g, 2 * g)}
        out = sparse(c, q, blocks, cnt, d ** -0.5)
        if n > 1:
            assert float(out[n - 1, :g].float().abs().max()) == 0
        keep = torch.ones(n, hk * g, dtype=torch.bool, device="cuda")
        for i, j in bad:
            keep[i, j] = False
            assert is_nan(out[i, j]), (i, j)
        assert torch.isfinite(out[keep]).all()
        for i in sorted({0, mid}):
            want, tol = sparse_expect(c, q.nan_to_num(0.0), lists, i, d ** -0.5)
            if i != s or n <= 2:
                check(out[i:i + 1, keep[i]], want[:, keep[i]], tol[:, keep[i]], "sequence %d" % i)
    assert cut == {False, True}  # one pass and partitions
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0
