"""Decode attention (whole, windowed, over listed blocks) with rows of q of very
different size, behind f16's range and below it, over every kind of pool."""
import pytest
import torch

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build as pkv_build
from _dense_side import attend, check, queries
from _pool_side import KINDS, AnyCache
from test_gpu_sparse import call, expect, lists_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.set_device_check(flag)
    yield flag
    pkv.set_device_check(None)


SIZE = [1e6, 1.0, 1e-6, 3.0, 1e-30, 0.0, 1e10, 0.5]


# one pass in a cluster, one CTA to a pair, partitions
@pytest.mark.parametrize("lens,take", [([300, 1000], 40), ([300] * 300, 10), ([20000, 9], 1200)])
@pytest.mark.parametrize("d,block", [(128, 16), (128, 32), (256, 16), (256, 32)])
@pytest.mark.parametrize("kind", KINDS)
def test_listed_blocks(kind, d, block, lens, take, _lib):
    n = len(lens)
    c = AnyCache(lens, 2, d, block, kind, seed=9)
    lists, blocks, counts = lists_of(c, take, 3)
    q = queries(n, 8, d, seed=9)
    q = (q.float() * torch.tensor(SIZE, device="cuda")[:, None]).to(torch.bfloat16)
    # the scale that makes a row's logits of ordinary size, and the rows it does that for
    for scale, rows in ((1e-7, [0]), (1e5, [2]), (1e-11, [6]), (0.09, [1, 2, 3, 4, 5, 7])):
        out = call(c, q, blocks, counts, scale)
        for s in (0, 1):
            want, tol = expect(c, q, lists, s, scale)
            check(out[s:s + 1, rows], want[:, rows], tol[:, rows], "scale %g" % scale)
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0


def whole(c, q, scale, partition):
    return pkv.paged_attention(q, c.k, c.v, c.tables, c.context_lens, scale, c.max_context,
                               partition, **c.kw())


def window(c, q, scale, partition):
    """A window behind which nothing lies."""
    return pkv.paged_attention_window(q, c.k, c.v, c.tables, c.context_lens, scale,
                                      c.max_context, c.max_context + 1, 3, partition, **c.kw())


@pytest.mark.parametrize("partition", [0, 64, None])
@pytest.mark.parametrize("d,block", [(128, 16), (128, 32), (256, 16), (256, 32)])
@pytest.mark.parametrize("op,kind", [(whole, "bf16"), (whole, "fp8"), (whole, "fp4"),
                                     (window, "bf16"), (window, "fp8")])
def test_whole_contexts(op, kind, d, block, partition, _lib):
    c = AnyCache([300, 1000], 2, d, block, kind, seed=9)
    q = queries(2, 8, d, seed=9)
    q = (q.float() * torch.tensor(SIZE, device="cuda")[:, None]).to(torch.bfloat16)
    for scale, rows in ((1e-7, [0]), (1e5, [2]), (1e-11, [6]), (0.09, [1, 2, 3, 4, 5, 7])):
        out = op(c, q, scale, partition)
        for s, ctx in enumerate(c.lens):
            see = torch.ones(1, ctx, dtype=torch.bool, device="cuda")
            want, tol = attend(q[s:s + 1], c.K[s], c.V[s], see, scale)
            check(out[s:s + 1, rows], want[:, rows], tol[:, rows], "scale %g" % scale)
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0
