"""Long contexts where every run of 16 tokens shows in the output: equal
weights, and V with a one in a column of the run's own. A run that is left out
or counted twice changes its column by 5 % or more."""
import pytest
import torch

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build as pkv_build
from _dense_side import Cache, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.set_device_check(flag)
    yield flag
    pkv.set_device_check(None)


def columns(c):
    """K = 0, V[t] = 1 in column (t / 16) % d, in the pools of c."""
    for s, n in enumerate(c.lens):
        t = torch.arange(n, device="cuda")
        v = torch.zeros(n, c.hk, c.d, device="cuda")
        v[t, :, (t // 16) % c.d] = 1
        k = torch.zeros_like(v)
        blk = c.tables[s, t // c.block].long()
        for pool, x in ((c.k, k), (c.v, v)):
            x = x.to(torch.float8_e4m3fn).view(torch.uint8) if c.fp8 else x.to(torch.bfloat16)
            pool[blk, :, t % c.block] = x
    if c.fp8:
        c.ks.fill_(1)
        c.vs.fill_(1)


def verify(out, d, see, what):
    """out [..., d] of a query that sees the tokens `see` [T]: column j is the
    share of them in its runs. Logits are 0 and weights 1, sums of ones are
    exact in fp32; the division, the partials' weights and their sum (up to 160
    parts) are 2^-16 together, the rounding to bf16 2^-8."""
    t = torch.nonzero(see)[:, 0]
    want = torch.zeros(d, dtype=torch.float64, device="cuda")
    want.index_add_(0, (t // 16) % d, torch.ones(len(t), dtype=torch.float64, device="cuda"))
    want /= len(t)
    over = (out.double() - want).abs() - want * (2.0 ** -8 + 2.0 ** -16)
    assert bool((over <= 0).all()), "%s: %d columns off" % (what, int((over > 0).sum()))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,lens,n,g", [(256, [70001], 5, 6), (128, [40000], 5, 4),
                                        (256, [33333, 50000, 4101], 3, 6),
                                        (128, [20000] * 5 + [333], 17, 8),
                                        (256, [12000] * 3, 64, 8)])
def test_tree(d, lens, n, g, fp8, _lib):
    c = Cache(lens, 2, d, 32, fp8, seed=3)
    columns(c)
    S = len(lens)
    q = queries(S * n, 2 * g, d, seed=4)
    st = torch.arange(S + 1, dtype=torch.int32, device="cuda") * n
    out = pkv.paged_attention_tree(q, c.k, c.v, c.tables, c.context_lens, st, d ** -0.5,
                                   c.max_context, n, **c.kw())
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0
    for s, ctx in enumerate(lens):
        t = torch.arange(ctx, device="cuda")
        for i in range(n):
            verify(out[s * n + i], d, t <= ctx - n + i, "sequence %d draft %d" % (s, i))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,block", [(128, 16), (256, 16), (256, 32)])
@pytest.mark.parametrize("partition", [None, 0, 512, 4096])
def test_window(d, block, fp8, partition, _lib):
    lens = [60000, 30000, 51234]
    c = Cache(lens, 2, d, block, fp8, seed=3)
    columns(c)
    q = queries(3, 12, d, seed=4)
    for window, sinks in ((50001, 77), (1 << 30, 0), (8195, 4000)):
        out = pkv.paged_attention_window(q, c.k, c.v, c.tables, c.context_lens, d ** -0.5,
                                         c.max_context, window, sinks, partition, **c.kw())
        torch.cuda.synchronize()
        assert int(_lib.item()) == 0
        for s, ctx in enumerate(lens):
            t = torch.arange(ctx, device="cuda")
            verify(out[s], d, (t < sinks) | (t >= ctx - window),
                   "window %d sequence %d" % (window, s))
