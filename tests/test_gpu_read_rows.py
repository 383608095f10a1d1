"""kv_cache_read of bf16 and E4M3 pools with more rows than one to a thread:
bit for bit what the slots hold."""
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


def pool_of(kind, nb, hk, block, d, g):
    """Any bits but a NaN's, and their values without the head's scale."""
    if kind == "bf16":
        x = torch.randint(-(1 << 15), 1 << 15, (nb, hk, block, d), device="cuda", generator=g)
        x = torch.where((x & 0x7F80) == 0x7F80, x & ~0x4000, x)
        pool = x.to(torch.int16).view(torch.bfloat16)
        return pool, pool
    x = torch.randint(0, 256, (nb, hk, block, d), dtype=torch.uint8, device="cuda", generator=g)
    pool = torch.where((x & 0x7F) == 0x7F, x - 1, x)
    return pool, pool.view(torch.float8_e4m3fn).float()


def expect(values, scale, slots, block):
    got = values[slots // block, :, slots % block]
    if scale is not None:
        got = (got * scale[:, None]).to(torch.bfloat16)
    return got


def bits(x):
    return x.contiguous().view(torch.int16)


# rows of 256 threads and less (with and without threads to spare), and of more
@pytest.mark.parametrize("hk", [1, 3, 5, 8, 17])
@pytest.mark.parametrize("d,block", [(128, 16), (128, 32), (256, 16), (256, 32)])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_many_rows(kind, d, block, hk, _lib):
    per = hk * d // 8
    least = -(-2 * 2048 * 152 // per)  # two rows to a thread from here on
    g = torch.Generator(device="cuda")
    g.manual_seed(per + block)
    ks = vs = None
    if kind == "fp8":
        ks = (torch.rand(hk, device="cuda", generator=g) + 0.5) / 64
        vs = -(torch.rand(hk, device="cuda", generator=g) + 0.5) / 64
    nb = 2 * least // block + 3
    kc, k_values = pool_of(kind, nb, hk, block, d, g)
    vc, v_values = pool_of(kind, nb, hk, block, d, g)
    for n in (least - 1, least, 2 * (least // 2) + 1, least + 4097):
        slots = torch.randint(0, nb * block, (n,), device="cuda", generator=g)
        skip = torch.rand(n, device="cuda", generator=g) < 0.1
        slots[skip] = -1 - torch.randint(0, 9, (int(skip.sum()),), device="cuda", generator=g)
        slots[-1] = nb * block - 1
        slots[-2] = -1
        # what lies behind the last row stays as it is
        k_out, v_out = (torch.full((n + 1, hk, d), 7.0, dtype=torch.bfloat16, device="cuda")
                        for _ in "kv")
        pkv.kv_cache_read(slots, kc, vc, ks, vs, k=k_out[:n], v=v_out[:n])
        for out, values, scale in ((k_out, k_values, ks), (v_out, v_values, vs)):
            want = expect(values, scale, slots.clamp(min=0), block)
            want[slots < 0] = 0
            assert torch.equal(bits(out[:n]), bits(want)), n
            assert bool((out[n] == 7).all()), n
        torch.cuda.synchronize()
        assert int(_lib.item()) == 0


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("hk,d", [(3, 128), (8, 256)])
def test_slots_behind_the_pool(hk, d, kind, _lib):
    """Reported, their rows zeros, in the first and in the second row of a thread."""
    n, block = 2 * 2048 * 152 // (hk * d // 8) + 5, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(hk)
    ks = vs = torch.full((hk,), 0.125, device="cuda") if kind == "fp8" else None
    kc, k_values = pool_of(kind, 40, hk, block, d, g)
    vc, v_values = pool_of(kind, 40, hk, block, d, g)
    slots = torch.randint(0, 40 * block, (n,), device="cuda", generator=g)
    for first in range(9):
        bad = torch.arange(n, device="cuda") % 1009 == first
        s = torch.where(bad, 40 * block + first * (1 << 40), slots)
        k, v = pkv.kv_cache_read(s, kc, vc, ks, vs)
        torch.cuda.synchronize()
        assert int(_lib.item()) == pkv.DEVERR_SLOT
        _lib.zero_()
        for out, values, scale in ((k, k_values, ks), (v, v_values, vs)):
            want = expect(values, scale, slots, block)
            want[bad] = 0
            assert torch.equal(bits(out), bits(want))
