"""The 4-bit cache and the sparse attention of the paged cache: inputs, plain
forms and exact forms of the calls that are measured.

A case is one pass on one shape. ``own`` False computes it from elementary
torch operations; ``own`` True makes the framework's calls.

  write4  K and V rows go into a 4-bit cache (E2M1 codes, an E4M3 scale for
          every 16 channels, an fp32 scale per head) and the values that were
          stored come back, for the attention of the step that wrote them.
  decode4 attention of one token per sequence over a 4-bit cache.
  bounds  the lowest and the highest K of every channel of the blocks that the
          sequences' newest tokens are in, as whole numbers of a head's step.
  select  the blocks of a context with the highest bounds of their logits, for
          each sequence and KV head: `take` of them, the first and the last
          always among them, in order.
  sparse  attention of one token per sequence over given blocks of its context,
          for each KV head its own, in bf16, E4M3 and 4-bit caches.

The 4-bit pool is bytes [blocks, heads, block, 9 d / 16], in lines of 144: the
128 code bytes of 256 / d tokens (two codes a byte, the even channel low), then
their 16 scales.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a decoding step of 64 sequences: one new token each
        dict(name="write4_step", op="write4", tokens=64, hk=4, d=256, block=16),
        # prompts of 32768 tokens together
        dict(name="write4_prompt", op="write4", tokens=32768, hk=8, d=128, block=32),
        # one user, a short context: the smallest attention of a step
        dict(name="decode4_one", op="decode4", seqs=1, lo=1033, hi=1033, hq=8, hk=2, d=128,
             block=16),
        # a batch of long contexts
        dict(name="decode4_batch", op="decode4", seqs=64, lo=8192, hi=8192, hq=24, hk=4, d=256,
             block=16),
        # continuous batching: every sequence its own length
        dict(name="decode4_mixed", op="decode4", seqs=96, lo=16, hi=16384, hq=32, hk=8, d=128,
             block=32),
        # the block that each sequence of a batch writes to, after one step
        dict(name="bounds_step", op="bounds", seqs=64, lo=8192, hi=8192, new=1, pool="bf16", hk=4,
             d=256, block=16),
        # the blocks of whole prompts, over an E4M3 cache
        dict(name="bounds_prompt", op="bounds", seqs=16, lo=1000, hi=16384, new=16384, pool="fp8",
             hk=8, d=128, block=32),
        # a batch of long contexts: a quarter of their blocks
        dict(name="select_batch", op="select", seqs=64, lo=8192, hi=8192, take=128, first=1,
             last=2, hq=24, hk=4, d=256, block=16),
        # few very long contexts: a sixteenth of their blocks
        dict(name="select_long", op="select", seqs=8, lo=131072, hi=131072, take=256, first=1,
             last=1, hq=24, hk=4, d=256, block=32),
        # one user: 64 blocks of a long context
        dict(name="sparse_one", op="sparse", seqs=1, lo=32768, hi=32768, take=64, pool="bf16",
             hq=8, hk=2, d=128, block=16),
        # a batch: 2048 tokens of each context
        dict(name="sparse_batch", op="sparse", seqs=64, lo=8192, hi=8192, take=128, pool="bf16",
             hq=24, hk=4, d=256, block=16),
        # few very long contexts over a 4-bit cache: 16384 tokens of each
        dict(name="sparse_long4", op="sparse", seqs=8, lo=131072, hi=131072, take=512, pool="fp4",
             hq=24, hk=4, d=256, block=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["write4", "decode4", "decode4", "bounds", "select", "sparse", "sparse"])
    hk = rng.choice([1, 2, 4, 8])
    c = dict(op=op, hk=hk, d=rng.choice([128, 256]), block=rng.choice([16, 32]))
    row = hk * c["d"]  # K elements of one token
    if op == "write4":
        c["tokens"] = _log(rng, 1, (1 << 25) // row)
        return c
    if op != "bounds":
        c["hq"] = hk * rng.randint(1, 8)
    if op in ("bounds", "sparse"):
        c["pool"] = rng.choice(["bf16", "fp8", "fp4"])
    c["seqs"] = _log(rng, 1, 128)
    # tokens of the whole batch: K of at most 2^29 elements
    most = max(64, (1 << 29) // (row * c["seqs"]))
    c["hi"] = _log(rng, 64, min(most, 131072))
    c["lo"] = c["hi"] if rng.random() < 0.4 else _log(rng, 16, c["hi"])
    if op == "bounds":
        c["new"] = rng.choice([1, 1, rng.randint(2, 64), c["hi"]])
    if op in ("select", "sparse"):
        c["take"] = _log(rng, 4, max(4, c["hi"] // c["block"]))
    if op == "select":
        c["first"], c["last"] = rng.randint(0, 2), rng.randint(0, 2)
    return c


def _lens(case):
    """Context lengths from lo to hi, evenly spread over the logarithm."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    return [int(round(lo * (hi / lo) ** ((i + 0.5) / n))) for i in range(n)]


# ------------------------------------------------------------------ inputs

def _halves():
    """[256, 2]: the two values of a byte of E2M1 codes."""
    v = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    v = torch.tensor(v + [-x for x in v], device="cuda")
    b = torch.arange(256, device="cuda")
    return torch.stack([v[b % 16], v[b // 16]], -1)


def _pack4(x, scale):
    """x [..., heads, d] fp32, scale [heads] -> code bytes [..., d / 2] and scale
    bytes [..., d / 16]."""
    y = (x / scale[:, None]).unflatten(-1, (-1, 16))
    s = (y.abs().amax(-1, keepdim=True) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    # where the scale rounds to zero so do the codes
    z = torch.where(s.float() > 0, y / s.float(), torch.zeros_like(y))
    a = z.abs()
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5)
            + (a > 5))
    code = (code + 8 * (z < 0)).flatten(-2)
    return (code[..., ::2] + 16 * code[..., 1::2]).to(torch.uint8), s[..., 0].view(torch.uint8)


def _lines(codes, scales):
    """Codes and scales of whole blocks [..., block, *] -> their lines [..., block, 9 d / 16]."""
    per = 128 // codes.shape[-1]
    b = codes.shape[-2]
    lines = torch.cat([codes.unflatten(-2, (b // per, per)).flatten(-2),
                       scales.unflatten(-2, (b // per, per)).flatten(-2)], -1)
    return lines.flatten(-2).unflatten(-1, (b, -1))


def _split(pages, d):
    """Lines [..., block, 9 d / 16] -> code and scale bytes of their tokens."""
    b = pages.shape[-2]
    lines = pages.flatten(-2).unflatten(-1, (-1, 144))
    return (lines[..., :128].flatten(-2).unflatten(-1, (b, d // 2)),
            lines[..., 128:].flatten(-2).unflatten(-1, (b, d // 16)))


def _pool(kind, total, case, g):
    """Random rows everywhere, as a pool that has been in use, and its scale."""
    hk, b, d = case["hk"], case["block"], case["d"]
    scale = None if kind == "bf16" else (torch.rand(hk, device="cuda", generator=g) + 0.5) / 64
    last = d * 9 // 16 if kind == "fp4" else d
    pool = torch.empty((total, hk, b, last), device="cuda",
                       dtype=torch.bfloat16 if kind == "bf16" else torch.uint8)
    step = max(1, (1 << 27) // (hk * b * d))
    for a in range(0, total, step):
        x = torch.randn(min(step, total - a), hk, b, d, device="cuda", generator=g)
        if kind == "bf16":
            pool[a:a + step] = x.to(torch.bfloat16)
        elif kind == "fp8":
            pool[a:a + step] = (x * 64).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            codes, scales = _pack4(x.transpose(1, 2), scale)
            pool[a:a + step] = _lines(codes.transpose(1, 2), scales.transpose(1, 2))
    return pool, scale


def prepare(case, seed):
    rng = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, hk, d, b = case["op"], case["hk"], case["d"], case["block"]
    st = dict(op=op, hk=hk, d=d, block=b)
    if op == "write4":
        n = case["tokens"]
        total = -(-n // b) + 8
        st["k"], st["ks"] = _pool("fp4", total, case, g)
        st["v"], st["vs"] = _pool("fp4", total, case, g)
        st["slots"] = torch.randperm(total * b, device="cuda", generator=g)[:n]
        # rows whose channels differ in size, as K's do
        size = torch.exp(torch.randn(hk, d, device="cuda", generator=g) / 2)
        rows = torch.randn(2, n, hk, d, device="cuda", generator=g) * size
        st["new_k"], st["new_v"] = rows.to(torch.bfloat16).unbind(0)
        st["halves"] = _halves()
        return st
    lens = _lens(case)
    rng.shuffle(lens)
    pages = [-(-c // b) for c in lens]
    total, width = sum(pages), max(pages)
    perm = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    tables = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(pages):
        tables[s, :n] = perm[at:at + n]
        at += n
    st.update(tables=tables, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
              max_context=max(lens),
              scale=float(torch.tensor(1 / math.sqrt(d), dtype=torch.float32)))
    if op in ("decode4", "sparse", "bounds"):
        st["pool"] = "fp4" if op == "decode4" else case["pool"]
        st["k"], st["ks"] = _pool(st["pool"], total, case, g)
    if op in ("decode4", "sparse"):
        st["v"], st["vs"] = _pool(st["pool"], total, case, g)
    if op != "bounds":
        # queries a little longer than unit rows, so that some tokens stand out
        st["q"] = (2 * torch.randn(len(lens), case["hq"], d, device="cuda",
                                   generator=g)).to(torch.bfloat16)
    if op == "bounds":
        st["new"] = min(case["new"], max(lens))
        st["bounds"] = torch.randint(-127, 128, (total, hk, 2, d), dtype=torch.int8,
                                     device="cuda", generator=g)
        # a step that lets the largest values pass its 127 multiples now and then
        st["step"] = (torch.rand(hk, device="cuda", generator=g) + 1) / 48
    if op == "select":
        # what 16 to 32 normal rows leave, as multiples of 1 / 32
        mid = torch.randn(total, hk, d, device="cuda", generator=g) / 2
        half = 1.5 + torch.randn(total, hk, d, device="cuda", generator=g).abs() / 3
        st["bounds"] = (torch.stack([mid - half, mid + half], 2) * 32).clamp(-127, 127).round() \
            .to(torch.int8)
        st["take"], st["first"], st["last"] = case["take"], case["first"], case["last"]
    if op == "sparse":
        # every head its own blocks, the last one always among them
        n = torch.tensor(pages, device="cuda")
        i = torch.arange(width, device="cuda")
        key = torch.rand(len(lens), hk, width, device="cuda", generator=g)
        key = torch.where(i == n[:, None, None] - 1, 2.0, key)
        key = torch.where(i < n[:, None, None], key, -1.0)
        take = min(case["take"], width)
        best = key.argsort(-1, descending=True)[..., :take]
        best = torch.where(torch.arange(take, device="cuda") < n[:, None, None], best, width)
        st["count"] = n[:, None].clamp(max=take).expand(-1, hk).to(torch.int32).contiguous()
        best = best.sort(-1).values
        st["list"] = torch.where(best < width, best, -1).to(torch.int32)
    if st.get("pool") == "fp4":
        st["halves"] = _halves()
    return st


# ------------------------------------------------------------- plain forms

def _rows(st, pages, scale):
    """Pages of K or V [S, P, heads, block, *] as fp32 rows [S, heads, P block, d]."""
    if st["pool"] == "bf16":
        x = pages.float()
    elif st["pool"] == "fp8":
        x = pages.view(torch.float8_e4m3fn).float()
    else:
        codes, scales = _split(pages, st["d"])
        x = st["halves"][codes.long()].flatten(-2).unflatten(-1, (-1, 16))
        x = (x * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)
    if scale is not None:
        x = x * scale[:, None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _attend(st, k, v, see):
    """q over k, v [S, heads, T, d] where see [S, heads, T]."""
    s, hq, d = st["q"].shape
    hk = st["hk"]
    z = st["q"].float().view(s, hk, hq // hk, d) @ k.transpose(2, 3) * st["scale"]
    z = z.masked_fill(~see[:, :, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    o = torch.where(total > 0, (e @ v) / total.clamp(min=1e-38), torch.zeros_like(total))
    return o.reshape(s, hq, d).to(torch.bfloat16)


def _plain_decode4(st):
    page = st["tables"].long().clamp(min=0)
    k, v = _rows(st, st["k"][page], st["ks"]), _rows(st, st["v"][page], st["vs"])
    t = torch.arange(k.shape[2], device=k.device)
    return _attend(st, k, v, (t < st["lens"][:, None])[:, None].expand(-1, st["hk"], -1))


def _plain_sparse(st):
    lst = st["list"].long()
    live = torch.arange(lst.shape[2], device=lst.device) < st["count"][..., None]
    lst = torch.where(live, lst, torch.zeros_like(lst))
    page = torch.gather(st["tables"].long()[:, None].expand(-1, st["hk"], -1), 2, lst)
    head = torch.arange(st["hk"], device=lst.device)[None, :, None]
    # [S, heads, P, block, *] -> heads behind the pages
    k = _rows(st, st["k"][page, head].transpose(1, 2), st["ks"])
    v = _rows(st, st["v"][page, head].transpose(1, 2), st["vs"])
    b = st["block"]
    pos = lst[..., None] * b + torch.arange(b, device=lst.device)
    see = (pos < st["lens"][:, None, None, None]) & live[..., None]
    return _attend(st, k, v, see.flatten(2))


def _plain_write4(st):
    slot, b, d = st["slots"], st["block"], st["d"]
    per = 256 // d
    line, half = slot % b // per, slot % b % per
    out = []
    for pool, scale, rows in ((st["k"], st["ks"], st["new_k"]), (st["v"], st["vs"], st["new_v"])):
        codes, scales = _pack4(rows.float(), scale)
        lines = pool.view(pool.shape[0], st["hk"], b // per, 144)
        cv = lines[..., :128].unflatten(-1, (per, -1))
        sv = lines[..., 128:].unflatten(-1, (per, -1))
        cv[slot // b, :, line, half] = codes
        sv[slot // b, :, line, half] = scales
        got = st["halves"][cv[slot // b, :, line, half].long()].flatten(-2)
        by = sv[slot // b, :, line, half].view(torch.float8_e4m3fn).float()
        got = (got.unflatten(-1, (-1, 16)) * by[..., None]).flatten(-2)
        out.append((got * scale[:, None]).to(torch.bfloat16))
    return out


def _plain_bounds(st):
    b, lens = st["block"], st["lens"].long()
    first = (lens - st["new"]).clamp(min=0) // b
    most = (st["new"] + b - 2) // b + 1
    blk = first[:, None] + torch.arange(most, device=lens.device)
    live = (blk * b < lens[:, None]) & (blk < st["tables"].shape[1])
    # blocks behind a sequence's last one stand for that one once more
    blk = torch.where(live, blk, (lens[:, None] - 1) // b)
    page = torch.gather(st["tables"].long(), 1, blk)
    x = _rows(st, st["k"][page], st["ks"]).unflatten(2, (-1, b)) / st["step"][:, None, None, None]
    pos = blk[..., None] * b + torch.arange(b, device=blk.device)
    hide = (pos >= lens[:, None, None])[:, None, :, :, None]
    lo = torch.floor(x).masked_fill(hide, math.inf).amin(3).clamp(-127, 127)
    hi = torch.ceil(x).masked_fill(hide, -math.inf).amax(3).clamp(-127, 127)
    new = torch.stack([lo, hi], 3).transpose(1, 2).to(torch.int8)
    st["bounds"][page.flatten()] = new.flatten(0, 1)
    return st["bounds"]


def _plain_select(st):
    s, hq, d = st["q"].shape
    hk, b = st["hk"], st["block"]
    q = st["q"].float().view(s, hk, hq // hk, d)
    code = torch.round(q * 127 / q.abs().amax((2, 3), keepdim=True).clamp(min=1e-38)).int()
    up = code.clamp(min=0).sum(2, dtype=torch.int32)
    down = (-code).clamp(min=0).sum(2, dtype=torch.int32)
    lo, hi = st["bounds"][st["tables"].long().clamp(min=0)].int().unbind(3)
    score = (up[:, None] * hi - down[:, None] * lo).sum(-1).transpose(1, 2)
    n = ((st["lens"] + b - 1) // b).long()[:, None, None]
    i = torch.arange(score.shape[2], device=score.device)
    score = torch.where((i < st["first"]) | (i >= n - st["last"]), 1 << 40, score)
    score = torch.where(i < n, score, -1 << 40)
    width = score.shape[2]
    best = score.sort(dim=-1, descending=True, stable=True).indices[..., :st["take"]]
    best = torch.where(best < n, best, width).sort(-1).values
    count = n[..., 0].clamp(max=st["take"]).expand(-1, hk)
    best = torch.where(best < width, best, -1)
    best = torch.nn.functional.pad(best, (0, st["take"] - best.shape[-1]), value=-1)
    return best.to(torch.int32), count.to(torch.int32)


def run(st):
    op = st["op"]
    if own:
        import paged_kv_cache_220_gb300 as pkv
        if op == "write4":
            pkv.kv_cache_write(st["new_k"], st["new_v"], st["slots"], st["k"], st["v"], st["ks"],
                               st["vs"])
            return pkv.kv_cache_read(st["slots"], st["k"], st["v"], st["ks"], st["vs"])
        if op == "decode4":
            return pkv.paged_attention(st["q"], st["k"], st["v"], st["tables"], st["lens"],
                                       st["scale"], st["max_context"], None, st["ks"], st["vs"])
        if op == "bounds":
            pkv.block_bounds(st["bounds"], st["k"], st["tables"], st["lens"], st["step"],
                             st["new"], k_scale=st["ks"])
            return st["bounds"]
        if op == "select":
            return pkv.select_blocks(st["q"], st["bounds"], st["tables"], st["lens"], st["block"],
                                     st["max_context"], st["take"], st["first"], st["last"])
        return pkv.paged_attention_sparse(st["q"], st["k"], st["v"], st["tables"], st["lens"],
                                          st["list"], st["count"], st["scale"],
                                          k_scale=st["ks"], v_scale=st["vs"])
    plain = {"write4": _plain_write4, "decode4": _plain_decode4, "bounds": _plain_bounds,
             "select": _plain_select, "sparse": _plain_sparse}
    return plain[op](st)


# ------------------------------------------------------------ work, exact

_BITS = {"bf16": 16, "fp8": 8, "fp4": 4.5}


def work(case):
    op, hk, d, b = case["op"], case["hk"], case["d"], case["block"]
    if op == "write4":
        n = case["tokens"] * hk * d * 2  # elements of K and V
        return {"bytes": int(n * (2 + 9 / 16 + 9 / 16 + 2)) + 16 * case["tokens"], "flops": 0}
    lens = _lens(case)
    if op == "bounds":
        total, tables = 0, 0
        for c in lens:
            first = max(0, c - min(case["new"], max(lens))) // b
            total += hk * d * ((c - first * b) * _BITS[case["pool"]] / 8
                               + 2 * (-(-c // b) - first))
            tables += 4 * (-(-c // b) - first)
        return {"bytes": int(total + tables), "flops": 0}
    blocks = [-(-c // b) for c in lens]
    q = 2 * case["hq"] * d
    if op == "select":
        return {"bytes": sum(n * (2 * hk * d + 4) + q + 4 * hk * (case["take"] + 1)
                             for n in blocks),
                "flops": sum(4 * n * hk * d for n in blocks)}
    if op == "sparse":
        # the last block may be a part of one
        seen = [min(c, min(n, case["take"]) * b - (n * b - c)) for c, n in zip(lens, blocks)]
        tables = [8 * hk * min(n, case["take"]) for n in blocks]
        bits = _BITS[case["pool"]]
    else:
        seen, bits = lens, 4.5
        tables = [4 * n for n in blocks]
    return {"bytes": sum(int(2 * t * hk * d * bits / 8) + i + 2 * q for t, i in zip(seen, tables)),
            "flops": sum(4 * t * case["hq"] * d for t in seen)}


def _exact_dense(st, pool, scale, pages):
    """Rows [heads, tokens, d] in 64 bits of the given blocks, each channel read
    from its place in the block's bytes."""
    hk, d, b = st["hk"], st["d"], st["block"]
    x = pool[pages]
    if st["pool"] == "bf16":
        return x.double().transpose(0, 1).reshape(hk, -1, d)
    if st["pool"] == "fp8":
        x = x.view(torch.float8_e4m3fn).double()
    else:
        x = _exact_4bit(x.reshape(len(pages), hk, -1), d, b)
    return (x * scale.double()[None, :, None, None]).transpose(0, 1).reshape(hk, -1, d)


def _exact_4bit(raw, d, b):
    """[..., bytes of a block] -> the values of its codes times their scales."""
    per = 256 // d
    t = torch.arange(b, device="cuda")[:, None]
    c = torch.arange(d, device="cuda")[None]
    line = t // per * 144
    byte = raw[..., line + t % per * (d // 2) + c // 2].int()
    nib = torch.where(c % 2 == 1, byte >> 4, byte & 15)
    exp, man = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(exp == 0, man / 2, (1 + man / 2) * torch.pow(2.0, (exp - 1).double()))
    val = torch.where(nib >= 8, -mag, mag)
    by = raw[..., line + 128 + t % per * (d // 16) + c // 16]
    return val * by.contiguous().view(torch.float8_e4m3fn).double()


def _exact_write4(st):
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    out = []
    for scale, rows in ((st["ks"], st["new_k"]), (st["vs"], st["new_v"])):
        y = rows.double() / scale.double()[:, None]
        y = y.view(*y.shape[:-1], -1, 16)
        top = y.abs().max(-1, keepdim=True).values / 6
        # E4M3: steps of 2^-3 of the binade, of 2^-9 below 2^-6
        e = torch.floor(torch.log2(top.clamp(min=2.0 ** -6)))
        e = torch.where(torch.pow(2.0, e) > top.clamp(min=2.0 ** -6), e - 1, e)
        e = torch.where(torch.pow(2.0, e + 1) <= top.clamp(min=2.0 ** -6), e + 1, e)
        ulp = torch.pow(2.0, e - 3)
        s = (torch.round(top / ulp) * ulp).clamp(max=448)
        z = torch.where(s > 0, y / s, torch.zeros_like(y))
        # nearest of the grid, ties to the even code
        gap = (z.abs().clamp(max=6)[..., None] - grid).abs()
        near = gap.amin(-1, keepdim=True)
        tied = gap == near
        even = tied & (torch.arange(8, device="cuda") % 2 == 0)
        pick = torch.where(even.any(-1, keepdim=True), even, tied).int().argmax(-1)
        val = torch.sign(z) * grid[pick] * s
        out.append(val.flatten(-2) * scale.double()[:, None])
    return out


def exact(case, seed):
    op, hk, d, b = case["op"], case["hk"], case["d"], case["block"]
    st = prepare(case, seed)
    if op == "write4":
        return _exact_write4(st) if case["tokens"] * hk * d <= 1 << 26 else None
    lens, tables = st["lens"].tolist(), st["tables"].tolist()
    if op == "bounds":
        out = st["bounds"].clone()
        for s, c in enumerate(lens):
            first = max(0, c - st["new"]) // b
            ids = torch.tensor(tables[s][first:-(-c // b)], device="cuda")
            x = _exact_dense(st, st["k"], st["ks"], ids)
            # what a cached value is, and its quotient, are fp32 numbers
            x = (x.float().double() / st["step"].double()[:, None, None]).float().double()
            x = x.view(hk, -1, b, d)
            t = first * b + torch.arange(len(ids) * b, device="cuda").view(1, -1, b, 1)
            lo = torch.where(t < c, x.floor(), math.inf).min(2).values
            hi = torch.where(t < c, x.ceil(), -math.inf).max(2).values
            both = torch.stack([lo, hi], 2).clamp(-127, 127).to(torch.int8)
            out[ids] = both.transpose(0, 1)
        return out
    hq = case["hq"]
    g = hq // hk
    q = st["q"].double().view(-1, hk, g, d)
    if op == "select":
        lists, counts = [], []
        for s, c in enumerate(lens):
            n = -(-c // b)
            code = torch.round(q[s] * 127 / q[s].abs().amax((1, 2), keepdim=True))
            bound = st["bounds"][torch.tensor(tables[s][:n], device="cuda")].double()
            score = sum(torch.maximum(code[:, j] * bound[:, :, 0], code[:, j] * bound[:, :, 1])
                        .sum(-1) for j in range(g))
            score[:st["first"]] = math.inf
            score[max(0, n - st["last"]):] = math.inf
            score = score.cpu()
            got = []
            for h in range(hk):
                row = score[:, h].tolist()
                best = sorted(sorted(range(n), key=lambda i: (-row[i], i))[:st["take"]])
                got.append(best + [-1] * (st["take"] - len(best)))
            lists.append(got)
            counts.append([min(n, st["take"])] * hk)
        return (torch.tensor(lists, dtype=torch.int32), torch.tensor(counts, dtype=torch.int32))
    out = torch.zeros(len(lens), hk, g, d, dtype=torch.float64, device="cuda")
    for s, c in enumerate(lens):
        for h in range(hk):
            if op == "decode4":
                ids = range(-(-c // b))
            else:
                ids = st["list"][s, h, :int(st["count"][s, h])].tolist()
            page = torch.tensor([tables[s][i] for i in ids], device="cuda")
            one = dict(st, hk=1)
            sl = lambda x: None if x is None else x[h:h + 1]  # noqa: E731
            k = _exact_dense(one, st["k"][:, h:h + 1], sl(st["ks"]), page)[0]
            v = _exact_dense(one, st["v"][:, h:h + 1], sl(st["vs"]), page)[0]
            t = torch.tensor([i * b for i in ids], device="cuda")[:, None]
            t = (t + torch.arange(b, device="cuda")).flatten()
            z = (q[s, h] @ k.T * st["scale"]).masked_fill(t >= c, -math.inf)
            out[s, h] = torch.softmax(z, -1) @ v
    return out.view(-1, hq, d)
