"""Random paged caches of every pool type with a dense copy of their rows, and
the 4-bit format in plain arithmetic."""
import torch

from _dense_side import Cache

KINDS = ["bf16", "fp8", "fp4"]
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def quantize(x, scale):
    """x [..., heads, d] fp32, scale [heads] -> (codes 0..15 as uint8 [..., heads, d],
    scale codes uint8 [..., heads, d/16]): the definition, division by division.
    (A quotient in 64 bits rounded to 32 is the quotient rounded to 32: 53 bits are
    more than 2 * 24 + 1. A tensor divided by a Python number on the GPU is a product
    with 1/6 and not that.)"""
    y = (x.double() / scale.double()[:, None]).float().unflatten(-1, (-1, 16))
    a = y.abs().amax(-1)  # a NaN stays one
    s8 = torch.where(a.isnan(), a, (a.double() / 6).float().clamp(max=448)).to(torch.float8_e4m3fn)
    s = s8.float()[..., None]
    z = torch.where(s > 0, (y.double() / s.double()).float(), torch.zeros_like(y))
    m = z.abs()
    code = ((m > 0.25).int() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5)
            + (m > 5)) + 8 * torch.signbit(z)
    return code.flatten(-2).to(torch.uint8), s8.view(torch.uint8)


def values(codes, scales):
    """What codes [..., d] and scale codes [..., d/16] stand for, without the
    head's scale (64 bits)."""
    grid = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=codes.device)
    by = scales.contiguous().view(torch.float8_e4m3fn).double()
    return (grid[codes.long()].unflatten(-1, (-1, 16)) * by[..., None]).flatten(-2)


def to_lines(codes, scales):
    """Codes [n, block, d] and scale codes [n, block, d/16] -> pages [n, block, 9d/16]."""
    n, b, d = codes.shape
    out = torch.empty(n, b * d // 16 * 9, dtype=torch.uint8, device=codes.device)
    lines = out.view(n, -1, 144)
    per = 256 // d
    for t in range(b):
        line, half = t // per, t % per
        lines[:, line, half * d // 2:(half + 1) * d // 2] = (
            codes[:, t, 0::2] | codes[:, t, 1::2] << 4)
        lines[:, line, 128 + half * d // 16:128 + (half + 1) * d // 16] = scales[:, t]
    return out.view(n, b, -1)


def from_lines(pages, d):
    """Pages [n, block, 9d/16] -> codes [n, block, d], scale codes [n, block, d/16]."""
    n, b, _ = pages.shape
    lines = pages.reshape(n, -1, 144)
    per = 256 // d
    codes = torch.empty(n, b, d, dtype=torch.uint8, device=pages.device)
    scales = torch.empty(n, b, d // 16, dtype=torch.uint8, device=pages.device)
    for t in range(b):
        line, half = t // per, t % per
        c = lines[:, line, half * d // 2:(half + 1) * d // 2]
        codes[:, t, 0::2], codes[:, t, 1::2] = c & 15, c >> 4
        scales[:, t] = lines[:, line, 128 + half * d // 16:128 + (half + 1) * d // 16]
    return codes, scales


class AnyCache(Cache):
    """Cache of a kind; 4-bit pools hold quantised normal rows, and NaN scales
    (with codes of 6) in every slot that holds no token."""

    def __init__(self, lens, hk, d, block, kind, seed, **kw):
        self.kind = kind
        super().__init__(lens, hk, d, block, kind != "bf16", seed, **kw)

    def _pool(self, nb, ids, pages, scale, g, std):
        if self.kind != "fp4":
            return super()._pool(nb, ids, pages, scale, g, std)
        d = self.d
        raw = torch.empty(nb, self.hk, self.block, d // 16 * 9, dtype=torch.uint8, device="cuda")
        raw[ids] = 0x7F
        dense, at = [], 0
        for c, n in zip(self.lens, pages):
            x = torch.randn(n * self.block, self.hk, d, device="cuda", generator=g) * std
            # channels of different size, as K's are
            x = x * torch.exp(torch.randn(d, device="cuda", generator=g) / 2)
            codes, scales = quantize(x, scale)
            codes[c:], scales[c:] = 0x07, 0x7F
            dense.append(values(codes[:c], scales[:c]) * scale.double()[:, None])
            view = lambda t: t.view(n, self.block, self.hk, -1).transpose(1, 2).flatten(0, 1)  # noqa: E731,B023
            raw[ids[at:at + n]] = to_lines(view(codes), view(scales)).view(
                n, self.hk, self.block, -1) if n else raw[:0]
            at += n
        return raw, dense

    def poison(self, s, t0, t1):
        if self.kind != "fp4":
            return super().poison(s, t0, t1)
        per = 256 // self.d
        for p in (self.k, self.v):
            lines = p.view(p.shape[0], self.hk, -1, 144)
            for t in range(t0, t1):
                r = t % self.block
                at = 128 + r % per * (self.d // 16)
                lines[int(self.tables[s, t // self.block]), :, r // per,
                      at:at + self.d // 16] = 0x7F
