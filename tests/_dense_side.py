"""Random paged caches with a dense copy of their rows, the attention of a few
query rows over them in 64 bits, and how far a kernel's bf16 result may be
from it.

Every slot that no sequence owns holds NaN (bf16 and E4M3 alike) and every
table entry behind a sequence's blocks is out of range, so a kernel that reads
either shows it."""
import math

import torch

HALF_BF16 = 2.0 ** -8  # a rounding to bf16 is off by at most this, relative


class Cache:
    def __init__(self, lens, hk, d, block, fp8, seed, width=None, spare=3, pool_blocks=None,
                 std=1.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.lens, self.hk, self.d, self.block, self.fp8 = list(lens), hk, d, block, fp8
        pages = [-(-c // block) for c in self.lens]
        total = sum(pages)
        nb = total + spare if pool_blocks is None else pool_blocks
        # the blocks in use: scattered; in a large pool, its last ones
        ids = (nb - (total + spare) + torch.randperm(total + spare, device="cuda", generator=g))
        width = max([1] + pages) + 2 if width is None else width
        self.tables = torch.full((len(self.lens), width), nb + 5, dtype=torch.int32,
                                 device="cuda")
        at = 0
        for s, n in enumerate(pages):
            self.tables[s, :n] = ids[at:at + n].int()
            at += n
        self.context_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.ks = self.vs = None
        if fp8:
            self.ks = (torch.rand(hk, device="cuda", generator=g) + 0.5) / 64
            self.vs = (torch.rand(hk, device="cuda", generator=g) + 0.5) / 64
        self.k, self.K = self._pool(nb, ids, pages, self.ks, g, std)
        self.v, self.V = self._pool(nb, ids, pages, self.vs, g, 1.0)
        self.max_context = max([0] + self.lens)

    def _pool(self, nb, ids, pages, scale, g, std):
        dt = torch.float8_e4m3fn if self.fp8 else torch.bfloat16
        pool = torch.empty(nb, self.hk, self.block, self.d, dtype=dt, device="cuda")
        raw = pool.view(torch.uint8 if self.fp8 else torch.int16)
        raw[ids] = 0x7F if self.fp8 else 0x7FC0  # NaN
        dense = []
        at = 0
        for c, n in zip(self.lens, pages):
            x = torch.randn(n * self.block, self.hk, self.d, device="cuda", generator=g) * std
            x = (x * 64 if self.fp8 else x).to(dt)
            y = x.view(raw.dtype)
            y[c:] = 0x7F if self.fp8 else 0x7FC0
            raw[ids[at:at + n]] = y.view(n, self.block, self.hk, self.d).permute(0, 2, 1, 3)
            x = x[:c].double()
            dense.append(x * scale.double()[:, None] if self.fp8 else x)
            at += n
        return (raw if self.fp8 else pool), dense

    def poison(self, s, t0, t1):
        """NaN into the slots of tokens [t0, t1) of sequence s, in the pools only."""
        for p in (self.k, self.v):
            raw = p if self.fp8 else p.view(torch.int16)
            for t in range(t0, t1):
                raw[int(self.tables[s, t // self.block]), :, t % self.block] = (
                    0x7F if self.fp8 else 0x7FC0)

    def kw(self):
        return dict(k_scale=self.ks, v_scale=self.vs)


def queries(n, hq, d, seed, std=2.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 77)
    return (std * torch.randn(n, hq, d, device="cuda", generator=g)).to(torch.bfloat16)


def attend(q, K, V, see, scale):
    """q [n, Hq, D] over K, V [T, Hk, D] (64 bits) where see [n, T]: the output
    [n, Hq, D] and the distance a kernel may have from it.

    Where the distance comes from, w_t the softmax weights, A = sum w_t |V_t|:
    - the output's rounding to bf16: 2^-8 |out|;
    - the weights' rounding to bf16 (or f16) before the product: 2^-8 A;
    - a logit's error dz, as an error 2 dz of every weight (numerator and
      sum): an fp32 sum of D products is off by at most (D + 4) 2^-23 of the
      sum of their magnitudes;
    - the fp32 sums over up to 2^18 tokens in blocks, ex2: 2^-12 A;
    - f16 weights of E4M3 pools below 2^-24 of the largest: 2^-25 |V| each."""
    n, hq, d = q.shape
    hk = K.shape[1]
    g = hq // hk
    x = q.double().view(n, hk, g, d)
    if K.shape[0] == 0:
        z = torch.zeros(n, hq, d, dtype=torch.float64, device=q.device)
        return z, z.clone()
    logit = torch.einsum("nhgd,thd->nhgt", x, K) * scale
    size = torch.einsum("nhgd,thd->nhgt", x.abs(), K.abs()) * abs(scale)
    hide = ~see[:, None, None, :]
    logit = logit.masked_fill(hide, -math.inf)
    w = torch.softmax(logit, -1)
    w = torch.where(see.any(-1)[:, None, None, None], w, torch.zeros_like(w))
    o = torch.einsum("nhgt,thd->nhgd", w, V)
    A = torch.einsum("nhgt,thd->nhgd", w, V.abs())
    dz = size.masked_fill(hide, 0).amax(-1, keepdim=True) * (d + 4) * 2.0 ** -23
    small = see.double().sum(-1)[:, None, None, None] * 2.0 ** -25 * V.abs().amax()
    some = see.any(-1)[:, None, None, None]
    tol = HALF_BF16 * o.abs() + A * (HALF_BF16 + 2 * dz + 2.0 ** -12) + small * some
    return o.reshape(n, hq, d), tol.reshape(n, hq, d)


def check(got, want, tol, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), "%s: not finite" % what
    over = (got - want).abs() - tol
    assert bool((over <= 0).all()), "%s: over by %.3e (|err| %.3e)" % (
        what, float(over.max()), float((got - want).abs().max()))
