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


@pytest.mark.parametrize("d,block", [(128, 16), (256, 32)])
def test_values_and_steps_of_any_size(d, block, _lib):
    c = AnyCache([5 * block, 3 * block - 1], 8, d, block, "bf16", seed=6)
    r = torch.Generator(device="cuda")
    r.manual_seed(8)
    for s, n in enumerate(c.lens):
        for b in range(-(-n // block)):
            # every exponent, zeros, infinities, or few exponents
            bits = torch.randint(0, 1 << 16, (8, block, d), device="cuda", generator=r)
            if b == 1:
                bits = bits & 0x81FF | 0x3F00
            if b == 2:
                bits = bits & 0x807F  # below the normal numbers
            x = bits.to(torch.int32).to(torch.int16).view(torch.bfloat16)
            x = torch.where(x.isnan(), 0.0, x.float()).to(torch.bfloat16)
            c.k[int(c.tables[s, b])] = x
            lo, hi = b * block, min(n, (b + 1) * block)
            c.K[s][lo:hi] = x.transpose(0, 1)[:hi - lo].to(c.K[s].dtype)
    for steps in ([1e-30, 2.0 ** -41, 2.0 ** -40, 1e-7, 0.0123, 0.5, 1.0, 3.0],
                  [700.0, 2.0 ** 16, 2.0 ** 17, 1e9, 1e30, 1.9999999, 1e-38, 3e38]):
        step = torch.tensor(steps, device="cuda")
        out = fresh(c)
        pkv.block_bounds(out, c.k, c.tables, c.context_lens, step, 5 * block)
        for s, n in enumerate(c.lens):
            for b in range(-(-n // block)):
                assert torch.equal(out[int(c.tables[s, b])], bounds_of(c, step, s, b)), (s, b)


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("d", [128, 256])
def test_scales_of_any_size(d, kind, _lib):
    c = AnyCache([50, 64], 4, d, 16, kind, seed=7)
    keep = c.ks.clone()
    for by, step in ((1e-9, 1e-10), (1e9, 1e8), (1e-35, 1e-36), (1e-3, 1e-38), (1.0, 2.0 ** -5),
                     (1e20, 1e18)):
        c.ks.copy_(keep * by)
        steps = torch.full((4,), step, device="cuda")
        out = fresh(c)
        pkv.block_bounds(out, c.k, c.tables, c.context_lens, steps, 64, k_scale=c.ks)
        kv = pkv.kv_cache_read  # the codes' values without the scale are bf16 numbers
        one = torch.ones_like(c.ks)
        for s, n in enumerate(c.lens):
            slots = (c.tables[s].long().repeat_interleave(16)[:n] * 16
                     + torch.arange(n, device="cuda") % 16)
            x = kv(slots, c.k, c.k, one, one)[0].float() * c.ks[:, None]
            x = x / steps[:, None]
            for b in range(-(-n // 16)):
                y = x[16 * b:16 * b + 16]
                want = torch.stack([y.floor().clamp(-127, 127).amin(0),
                                    y.ceil().clamp(-127, 127).amax(0)], 1).to(torch.int8)
                assert torch.equal(out[int(c.tables[s, b])], want), (by, s, b)
