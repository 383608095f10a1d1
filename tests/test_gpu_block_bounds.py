"""block_bounds against the definition over a dense copy of K."""
import pytest
import torch

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build as pkv_build
from _pool_side import KINDS, AnyCache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.set_device_check(flag)
    yield flag
    pkv.set_device_check(None)


def bounds_of(c, step, s, b):
    """[Hk, 2, D] of block b of sequence s."""
    x = c.K[s][b * c.block:(b + 1) * c.block].float() / step[:, None]
    x = torch.where(x.isnan(), 0.0, x)
    return torch.stack([x.floor().clamp(-127, 127).amin(0), x.ceil().clamp(-127, 127).amax(0)],
                       1).to(torch.int8)


def fresh(c):
    return torch.full((c.k.shape[0], c.hk, 2, c.d), 99, dtype=torch.int8, device="cuda")


LENS = [0, 1, 5, 15, 16, 17, 31, 32, 33, 64, 100, 129, 1000]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,block,hk", [(128, 16, 3), (128, 32, 2), (256, 16, 1), (256, 32, 8)])
def test_the_definition(d, block, hk, kind, _lib):
    c = AnyCache(LENS, hk, d, block, kind, seed=d + hk)
    # some values pass 127 steps, most do not
    step = (torch.rand(hk, device="cuda") + 0.5) / 30
    for new in (0, 1, 2, 16, 17, 40, 5000):
        out = fresh(c)
        pkv.block_bounds(out, c.k, c.tables, c.context_lens, step, new, k_scale=c.ks)
        want = fresh(c)
        for s, n in enumerate(c.lens):
            if n and new:
                for b in range(max(0, n - new) // block, -(-n // block)):
                    want[int(c.tables[s, b])] = bounds_of(c, step, s, b)
        assert torch.equal(out, want), new
    num = torch.tensor([i * 7 % 40 for i in range(len(LENS))], dtype=torch.int32, device="cuda")
    out, want = fresh(c), fresh(c)
    pkv.block_bounds(out, c.k, c.tables, c.context_lens, step, 40, num, k_scale=c.ks)
    for s, n in enumerate(c.lens):
        new = min(int(num[s]), n)
        if new:
            for b in range((n - new) // block, -(-n // block)):
                want[int(c.tables[s, b])] = bounds_of(c, step, s, b)
    assert torch.equal(out, want)
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_scales_below_zero_and_nan_codes(kind, _lib):
    c = AnyCache([70, 33], 2, 256, 32, kind, seed=9)
    c.ks[1] = -c.ks[1]
    for s in range(2):
        c.K[s][:, 1] = -c.K[s][:, 1]
    # one token of NaN (a scale of 16 channels, or all channels) and a whole block
    c.poison(0, 5, 6)
    c.K[0][5] = float("nan")
    c.poison(1, 0, 32)
    c.K[1][:32] = float("nan")
    step = torch.full((2,), 1 / 40, device="cuda")
    out = fresh(c)
    pkv.block_bounds(out, c.k, c.tables, c.context_lens, step, 100, k_scale=c.ks)
    for s, n in enumerate(c.lens):
        for b in range(-(-n // 32)):
            assert torch.equal(out[int(c.tables[s, b])], bounds_of(c, step, s, b)), (s, b)
    assert float(out[int(c.tables[1, 0])].abs().max()) == 0
    assert int(_lib.item()) == 0


def test_nan_counts_as_zero(_lib):
    c = AnyCache([40], 2, 128, 16, "bf16", seed=1)
    c.k[int(c.tables[0, 1]), 1, 3, 7] = float("nan")
    c.k[int(c.tables[0, 1]), 0, 2, 9] = float("inf")
    c.K[0][19, 1, 7] = float("nan")
    c.K[0][18, 0, 9] = float("inf")
    step = torch.ones(2, device="cuda") / 40
    out = fresh(c)
    pkv.block_bounds(out, c.k, c.tables, c.context_lens, step, 40)
    for b in range(3):
        assert torch.equal(out[int(c.tables[0, b])], bounds_of(c, step, 0, b))
    assert int(out[int(c.tables[0, 1]), 0, 1, 9]) == 127


def test_bad_arguments_on_the_device_are_reported(_lib):
    c = AnyCache([40, 50], 2, 128, 16, "bf16", seed=2)
    step = torch.ones(2, device="cuda") / 40
    want = fresh(c)
    for b in range(3):
        want[int(c.tables[0, b])] = bounds_of(c, step, 0, b)
    keep = c.context_lens.clone()
    for n in (-1, c.tables.shape[1] * 16 + 1):
        c.context_lens[1] = n
        out = fresh(c)
        pkv.block_bounds(out, c.k, c.tables, c.context_lens, step, 100)
        torch.cuda.synchronize()
        assert int(_lib.item()) == pkv.DEVERR_CONTEXT and torch.equal(out, want)
        _lib.zero_()
    c.context_lens.copy_(keep)
    for n in (-1, 101):
        num = torch.tensor([100, n], dtype=torch.int32, device="cuda")
        out = fresh(c)
        pkv.block_bounds(out, c.k, c.tables, c.context_lens, step, 100, num)
        torch.cuda.synchronize()
        assert int(_lib.item()) == pkv.DEVERR_CONTEXT and torch.equal(out, want)
        _lib.zero_()
    for b in (0, 2, 3):
        want[int(c.tables[1, b])] = bounds_of(c, step, 1, b)
    for bad in (-1, c.k.shape[0]):
        table = c.tables.clone()
        table[1, 1] = bad
        out = fresh(c)
        pkv.block_bounds(out, c.k, table, c.context_lens, step, 100)
        torch.cuda.synchronize()
        assert int(_lib.item()) == pkv.DEVERR_BLOCK_ID and torch.equal(out, want)
        _lib.zero_()


def test_large_pool_stream_and_graph(_lib):
    nb = (1 << 32) // (4 * 32 * 256 * 2) + 2000
    c = AnyCache([300, 77], 4, 256, 32, "bf16", seed=4, pool_blocks=nb)
    step = torch.ones(4, device="cuda") / 50
    out = torch.zeros(nb, 4, 2, 256, dtype=torch.int8, device="cuda")

    def verify():
        for s, n in enumerate(c.lens):
            for b in range(max(0, n - 100) // 32, -(-n // 32)):
                assert torch.equal(out[int(c.tables[s, b])], bounds_of(c, step, s, b))

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    pkv.block_bounds(out, c.k, c.tables, c.context_lens, step, 100, stream=side)
    side.synchronize()
    verify()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.block_bounds(out, c.k, c.tables, c.context_lens, step, 100)
    out.zero_()
    graph.replay()
    verify()
    assert int(_lib.item()) == 0
