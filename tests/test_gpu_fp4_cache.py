"""4-bit pools: what kv_cache_write stores, byte for byte against the format's
definition; kv_cache_read of every pool type; block copies and swaps."""
import pytest
import torch

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build as pkv_build
from _pool_side import AnyCache, from_lines, quantize, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.set_device_check(flag)
    yield flag
    pkv.set_device_check(None)


def rows(n, hk, d, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    size = torch.exp(2 * torch.randn(n, hk, d // 16, 1, device="cuda", generator=g))
    x = torch.randn(n, hk, d // 16, 16, device="cuda", generator=g) * size
    return x.flatten(-2).to(torch.bfloat16)


def at_slots(pool, slots, d):
    """Codes and scale codes [T, Hk, *] that the slots hold."""
    nb, hk, b, _ = pool.shape
    codes, scales = from_lines(pool.view(nb * hk, b, -1), d)
    pick = lambda t: t.view(nb, hk, b, -1)[slots // b, :, slots % b]  # noqa: E731
    return pick(codes), pick(scales)


@pytest.mark.parametrize("hk", [1, 2, 3, 8])
@pytest.mark.parametrize("d,block", [(128, 16), (128, 32), (256, 16), (256, 32)])
@pytest.mark.parametrize("n", [1, 17, 300])
def test_write_is_the_definition(d, block, hk, n, _lib):
    nb = 40
    k, v = rows(n, hk, d, 1), rows(n, hk, d, 2)
    ks = torch.rand(hk, device="cuda") + 0.01
    vs = torch.rand(hk, device="cuda") + 0.01
    slots = torch.randperm(nb * block, device="cuda")[:n]
    slots[n // 2] = -1
    kc, vc = (torch.randint(0, 256, (nb, hk, block, d // 16 * 9), dtype=torch.uint8,
                            device="cuda") for _ in "kv")
    before = kc.clone(), vc.clone()
    pkv.kv_cache_write(k, v, slots, kc, vc, ks, vs)
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0
    live = slots >= 0
    for pool, old, x, scale in ((kc, before[0], k, ks), (vc, before[1], v, vs)):
        codes, scales = at_slots(pool, slots[live], d)
        want_c, want_s = quantize(x[live], scale)
        assert torch.equal(scales, want_s)
        assert torch.equal(codes, want_c)
        # every other row is as it was
        every = torch.arange(nb * block, device="cuda")
        rest = every[~torch.isin(every, slots[live])]
        for a, b in zip(at_slots(pool, rest, d), at_slots(old, rest, d)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("scale", [1.0, 1 / 64, 0.0123, 3e-13, 9e11, 2e-38, 3e37, -0.37])
def test_every_size_of_row(scale, _lib):
    """Rows of every exponent, in groups whose largest is any bf16 and the others
    anything below it, zeros of both signs among them; scales on both sides of
    what the quick division takes."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    n, d = 4096, 128
    bits = torch.randint(0, 1 << 15, (n, 8, d // 16, 16), device="cuda", generator=g)
    bits = torch.where(bits >= 0x7F80, bits - 0x7F80, bits)  # finite
    top = bits[..., :1]
    near = top - torch.randint(0, 900, bits.shape, device="cuda", generator=g)
    bits = torch.where(torch.rand(bits.shape, device="cuda", generator=g) < 0.8, near, bits % (
        top + 1)).clamp(min=0)
    bits = torch.where(torch.rand(bits.shape, device="cuda", generator=g) < 0.05, 0, bits)
    bits = bits | torch.randint(0, 2, bits.shape, device="cuda", generator=g) << 15
    x = bits.to(torch.int32).to(torch.int16).view(torch.bfloat16).view(n, 8, d)
    ks = scale * (1 + torch.rand(8, device="cuda", generator=g))
    ks[0], ks[1] = scale, scale * 0.5
    kc = pkv.fp4_cache(n // 32, 8, 32, d)
    vc = torch.zeros_like(kc)
    slots = torch.randperm(n, device="cuda", generator=g)
    pkv.kv_cache_write(x, -x, slots, kc, vc, ks, ks)
    for pool, y in ((kc, x), (vc, -x)):
        codes, scales = at_slots(pool, slots, d)
        want_c, want_s = quantize(y, ks)
        assert torch.equal(scales, want_s)
        assert torch.equal(codes, want_c)
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("hk,d,n", [(32, 256, 3), (32, 128, 700), (5, 128, 9001), (7, 256, 1)])
def test_many_heads_and_many_rows(hk, d, n, _lib):
    """Rows and heads on both sides of what a CTA takes, the read back included."""
    b = 32
    nb = -(-n // b) + 1
    k, v = rows(n, hk, d, 5), rows(n, hk, d, 6)
    ks, vs = torch.rand(hk, device="cuda") + 0.1, torch.rand(hk, device="cuda") + 0.1
    kc, vc = pkv.fp4_cache(nb, hk, b, d), pkv.fp4_cache(nb, hk, b, d)
    slots = torch.randperm(nb * b, device="cuda")[:n]
    pkv.kv_cache_write(k, v, slots, kc, vc, ks, vs)
    got = pkv.kv_cache_read(slots, kc, vc, ks, vs)
    for x, y, scale in ((k, got[0], ks), (v, got[1], vs)):
        want = (values(*quantize(x, scale)) * scale.double()[:, None]).float().to(torch.bfloat16)
        assert torch.equal(y, want)
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("d", [128, 256])
def test_write_of_special_values(d, _lib):
    """Zeros, groups too small for a scale, infinities, NaN, largest values and
    every midpoint between two codes."""
    x = torch.zeros(8, 1, d, dtype=torch.bfloat16, device="cuda")
    x[1] = 1e-30
    x[2, 0, 3] = float("inf")
    x[2, 0, 20] = -float("inf")
    x[3, 0, 5] = float("nan")
    x[4] = 3e38
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], device="cuda")
    x[5, 0, :16] = torch.cat([mid, -mid])
    x[6] = 2.0 ** -9 * 6
    x[7] = 2.0 ** -10 * 6  # its scale is a tie between 0 and the smallest
    one = torch.ones(1, device="cuda")
    kc, vc = pkv.fp4_cache(2, 1, 16, d), pkv.fp4_cache(2, 1, 16, d)
    slots = torch.arange(8, device="cuda") + 3
    pkv.kv_cache_write(x, -x, slots, kc, vc, one, one)
    for pool, y in ((kc, x), (vc, -x)):
        codes, scales = at_slots(pool, slots, d)
        want_c, want_s = quantize(y, one)
        assert torch.equal(scales & 0x7F, want_s & 0x7F) and torch.equal(codes, want_c)
    got, _ = pkv.kv_cache_read(slots, kc, vc, one, one)
    assert float(got[0].abs().max()) == 0 and float(got[1].abs().max()) == 0
    assert float(got[2, 0, 3]) == 2688 and float(got[2, 0, 20]) == -2688
    assert got[3, 0, :16].isnan().all() and float(got[3, 0, 16:].abs().max()) == 0
    assert float(got[4].min()) == 2688
    assert got[5, 0, :8].tolist() == [0, 1, 1, 2, 2, 4, 4, 6]
    assert float(got[6].min()) == 2.0 ** -9 * 6 and float(got[7].max()) == 0
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("d,block,hk", [(128, 16, 3), (128, 32, 8), (256, 16, 1), (256, 32, 4)])
def test_read(d, block, hk, kind, _lib):
    c = AnyCache([50, 7, 133], hk, d, block, kind, seed=d + hk)
    slots, want = [], ([], [])
    for s, n in enumerate(c.lens):
        for t in (0, 1, n // 2, n - 1):
            slots.append(int(c.tables[s, t // block]) * block + t % block)
            for w, dense in zip(want, (c.K, c.V)):
                w.append(dense[s][t])
    slots = torch.tensor(slots + [-1, -7], device="cuda")
    k, v = pkv.kv_cache_read(slots, c.k, c.v, **c.kw())
    for got, w in zip((k, v), want):
        w = torch.stack(w)
        # an fp32 product of an exact value and the head's scale, then bf16
        tol = w.abs() * (2.0 ** -8 + 2.0 ** -23)
        assert bool(((got[:-2].double() - w).abs() <= tol).all())
        assert float(got[-2:].abs().max()) == 0
        if kind != "bf16":
            # the scales of this cache times exact codes: one rounding each, so
            # that of fp32 then bf16 is the plain computation's
            assert torch.equal(got[:-2], w.float().to(torch.bfloat16))
    # into given tensors, on another stream, and captured
    k2, v2 = torch.full_like(k, 9), torch.full_like(v, 9)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert pkv.kv_cache_read(slots, c.k, c.v, k=k2, v=v2, stream=side, **c.kw())[0] is k2
    side.synchronize()
    assert torch.equal(k, k2) and torch.equal(v, v2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.kv_cache_read(slots, c.k, c.v, k=k2, v=v2, **c.kw())
    k2.zero_()
    graph.replay()
    assert torch.equal(k, k2) and int(_lib.item()) == 0


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_bad_slots_are_reported(kind, _lib):
    c = AnyCache([32], 2, 128, 16, kind, seed=5)
    end = c.k.shape[0] * 16
    slots = torch.tensor([int(c.tables[0, 0]) * 16, end], device="cuda")
    k, _ = pkv.kv_cache_read(slots, c.k, c.v, **c.kw())
    torch.cuda.synchronize()
    assert int(_lib.item()) == pkv.DEVERR_SLOT and float(k[1].abs().max()) == 0
    assert bool(((k[0].double() - c.K[0][0]).abs() <= c.K[0][0].abs() * 2.0 ** -7).all())
    _lib.zero_()
    if kind == "fp4":
        before = c.k.clone()
        pkv.kv_cache_write(k, k, torch.tensor([-1, end], device="cuda"), c.k, c.v, **c.kw())
        torch.cuda.synchronize()
        assert int(_lib.item()) == pkv.DEVERR_SLOT and torch.equal(c.k, before)
        _lib.zero_()


def test_slots_behind_32_bits(_lib):
    """A pool of more than 2^32 bytes: rows at its end."""
    hk, d, block = 8, 256, 32
    nb = (1 << 32) // (hk * block * 144) + 100
    kc = torch.empty(nb, hk, block, 144, dtype=torch.uint8, device="cuda")
    vc = torch.empty_like(kc)
    k, v = rows(5, hk, d, 3), rows(5, hk, d, 4)
    scale = torch.rand(hk, device="cuda") + 0.1
    slots = nb * block - 1 - torch.tensor([0, 1, 33, 500, 70], device="cuda")
    pkv.kv_cache_write(k, v, slots, kc, vc, scale, scale)
    got, gov = pkv.kv_cache_read(slots, kc, vc, scale, scale)
    for x, y in ((k, got), (v, gov)):
        want = values(*quantize(x, scale)) * scale.double()[:, None]
        assert bool(((y.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -23)).all())
    assert int(_lib.item()) == 0


@pytest.mark.parametrize("d,block", [(128, 16), (256, 32)])
def test_copies_and_swaps(d, block, _lib):
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    kc, vc = (torch.randint(0, 256, (12, 3, block, d // 16 * 9), dtype=torch.uint8, device="cuda",
                            generator=g) for _ in "kv")
    k0, v0 = kc.clone(), vc.clone()
    pairs = torch.tensor([[1, 7], [3, 0]], dtype=torch.int32, device="cuda")
    pkv.copy_blocks(kc, vc, pairs)
    k0[[7, 0]], v0[[7, 0]] = k0[[1, 3]], v0[[1, 3]]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)
    ids = torch.tensor([4, 11, 2], dtype=torch.int32, device="cuda")
    kb, vb = torch.empty_like(kc[:3]), torch.empty_like(vc[:3])
    pkv.swap_out(kc, vc, ids, kb, vb)
    assert torch.equal(kb, k0[[4, 11, 2]]) and torch.equal(vb, v0[[4, 11, 2]])
    back = torch.tensor([5, 6, 8], dtype=torch.int32, device="cuda")
    pkv.swap_in(kc, vc, back, kb, vb)
    k0[[5, 6, 8]], v0[[5, 6, 8]] = kb, vb
    assert torch.equal(kc, k0) and torch.equal(vc, v0) and int(_lib.item()) == 0


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("hk", [1, 3, 9, 15, 16, 17, 31])
def test_rows_that_do_not_fill_a_cta(hk, d, _lib):
    """Numbers of rows around multiples of what a CTA takes, up to two rows to a thread."""
    per = hk * d // 8
    many = 2 * 2048 * 152 // per + 1
    nb = -(-many // 16) + 1
    ks, vs = torch.rand(hk, device="cuda") + 0.1, torch.rand(hk, device="cuda") + 0.1
    for n in (1, 256 // per + 1, 5, many):
        k, v = rows(n, hk, d, n), rows(n, hk, d, n + 1)
        kc, vc = pkv.fp4_cache(nb, hk, 16, d), pkv.fp4_cache(nb, hk, 16, d)
        slots = torch.randperm(nb * 16, device="cuda")[:n]
        pkv.kv_cache_write(k, v, slots, kc, vc, ks, vs)
        got = pkv.kv_cache_read(slots, kc, vc, ks, vs)
        for x, y, pool, scale in ((k, got[0], kc, ks), (v, got[1], vc, vs)):
            codes, scales = quantize(x, scale)
            want = (values(codes, scales) * scale.double()[:, None]).float().to(torch.bfloat16)
            assert torch.equal(y, want), n
            # nothing else was written
            have = at_slots(pool, slots, d)
            assert torch.equal(have[0], codes) and torch.equal(have[1], scales), n
            for b in range(0, nb, max(1, nb // 3)):
                used = slots[slots // 16 == b] % 16
                free = torch.ones(16, dtype=torch.bool, device="cuda")
                free[used] = False
                lines = pool[b].view(hk, -1, 144)
                per_line = 256 // d
                for t in free.nonzero().flatten().tolist():
                    r, i = t // per_line, t % per_line
                    assert int(lines[:, r, i * d // 2:(i + 1) * d // 2].max()) == 0
    assert int(_lib.item()) == 0
