"""The paged cache's draft-tree attention, sliding-window attention and draft
acceptance: inputs, plain forms and exact forms of the calls that are measured.

A case is one call on one shape. ``own`` False computes it from elementary
torch operations; ``own`` True makes the framework's call.

  tree    attention of n drafted tokens per sequence over a paged cache. The
          drafts are the last n of the sequence's tokens; a draft sees every
          earlier (committed) token and the drafts its 64-bit mask names.
  window  decode of one token per sequence that sees the last `window` tokens
          and the first `sinks` ones.
  accept  the rows of the accepted drafts move up behind the committed tokens,
          in every layer's pools.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one user, a short window: the smallest call of a decoding step
        dict(name="window_one", op="window", seqs=1, lo=700, hi=700, window=512, sinks=4,
             hq=8, hk=2, d=128, block=16, fp8=False),
        # a batch of long contexts through a 4096-token window with four sinks
        dict(name="window_batch", op="window", seqs=64, lo=8192, hi=8192, window=4096, sinks=4,
             hq=24, hk=4, d=256, block=16, fp8=False),
        # continuous batching: lengths from below the window to far above it
        dict(name="window_mixed", op="window", seqs=256, lo=16, hi=16384, window=1024, sinks=16,
             hq=24, hk=4, d=256, block=32, fp8=False),
        # few very long contexts over an E4M3 cache, a wide window of odd size
        dict(name="window_long_fp8", op="window", seqs=8, lo=131072, hi=131072, window=32001,
             sinks=64, hq=24, hk=4, d=256, block=32, fp8=True),
        # one user, a chain of five drafts
        dict(name="tree_one", op="tree", seqs=1, lo=1033, hi=1033, nlo=5, nhi=5, chain=True,
             hq=8, hk=2, d=128, block=16, fp8=False),
        # a batch verifying trees of 16 drafts against long contexts
        dict(name="tree_batch", op="tree", seqs=32, lo=8192, hi=8192, nlo=16, nhi=16,
             chain=False, hq=24, hk=4, d=256, block=16, fp8=False),
        # wide trees: 64 drafts a sequence, many query rows to a cached row
        dict(name="tree_wide", op="tree", seqs=16, lo=4096, hi=4096, nlo=64, nhi=64,
             chain=False, hq=24, hk=4, d=256, block=16, fp8=False),
        # ragged batch: every sequence its own length and number of drafts
        dict(name="tree_mixed", op="tree", seqs=96, lo=16, hi=16384, nlo=1, nhi=24,
             chain=False, hq=32, hk=8, d=128, block=32, fp8=False),
        # few long contexts over an E4M3 cache, short chains
        dict(name="tree_long_fp8", op="tree", seqs=8, lo=65536, hi=65536, nlo=8, nhi=8,
             chain=True, hq=24, hk=4, d=256, block=32, fp8=True),
        # one user's accepted drafts, one layer
        dict(name="accept_one", op="accept", seqs=1, lo=1033, hi=1033, nlo=5, nhi=5, layers=1,
             hq=8, hk=2, d=128, block=16, fp8=False),
        # a batch's accepted drafts in all layers' pools
        dict(name="accept_layers", op="accept", seqs=64, lo=256, hi=512, nlo=16, nhi=16,
             layers=16, hq=24, hk=4, d=256, block=16, fp8=False),
        # a large ragged batch with wide trees over an E4M3 cache
        dict(name="accept_fp8", op="accept", seqs=512, lo=64, hi=256, nlo=1, nhi=64, layers=4,
             hq=32, hk=8, d=128, block=32, fp8=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "window", "window", "accept"])
    hk = rng.choice([1, 2, 4, 8])
    c = dict(op=op, hk=hk, hq=hk * rng.randint(1, 8), d=rng.choice([128, 256]),
             block=rng.choice([16, 32]), fp8=rng.random() < 0.4)
    c["seqs"] = _log(rng, 1, 128)
    row = 2 * hk * c["d"]  # K and V elements of one token
    if op == "accept":
        c["lo"] = _log(rng, 64, 512)
        c["hi"] = c["lo"] + rng.randint(0, 255)
        c["layers"] = _log(rng, 1, max(1, min(16, (1 << 30) // (row * c["seqs"] * c["hi"]))))
        c["nlo"] = rng.randint(1, 32)
        c["nhi"] = min(64, c["nlo"] + rng.randint(0, 32))
        return c
    # tokens of the whole batch: at most 1 GiB of K and V in bf16
    most = max(64, (1 << 29) // (row * c["seqs"]))
    c["hi"] = _log(rng, 64, min(most, 65536))
    c["lo"] = c["hi"] if rng.random() < 0.4 else _log(rng, 64, c["hi"])
    if op == "tree":
        # at most 10^11 operations
        c["nhi"] = _log(rng, 1, max(1, min(64, 25 * 10**9 // (c["hq"] * c["d"] * c["seqs"]
                                                             * c["hi"]))))
        c["nlo"] = rng.randint(1, c["nhi"])
        c["chain"] = rng.random() < 0.3
    else:
        c["window"] = _log(rng, 1, 2 * c["hi"])
        c["sinks"] = rng.choice([0, 1, 4, rng.randint(2, 100)])
    return c


def _spread(n, lo, hi):
    """n lengths from lo to hi, evenly spread over the logarithm."""
    return [int(round(lo * (hi / lo) ** ((i + 0.5) / n))) for i in range(n)]


def _shape(case):
    """Per sequence (context length, drafts), the drafts included in the length."""
    n = case["seqs"]
    ctx = _spread(n, case["lo"], case["hi"])
    if case["op"] == "window":
        return [(c, 1) for c in ctx]
    drafts = [case["nlo"] + (i * 7919 + 3) % (case["nhi"] - case["nlo"] + 1) for i in range(n)]
    return [(max(c, d), d) for c, d in zip(ctx, drafts)]


def _paths(case):
    """Per sequence the accepted drafts: an increasing list, not all kept."""
    rng = random.Random(17)
    out = []
    for _, n in _shape(case):
        m = rng.randint(0, max(1, n // 2)) if n > 1 else rng.randint(0, 1)
        out.append(sorted(rng.sample(range(n), m)))
    return out


# ------------------------------------------------------------------ inputs

def _pool(shape, fp8, g):
    """Random rows everywhere, as a pool that has been in use: bf16, or E4M3
    codes (their bytes)."""
    x = torch.empty(shape, dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16, device="cuda")
    flat = x.view(-1)
    step = 1 << 27
    for a in range(0, flat.numel(), step):
        part = torch.randn(min(step, flat.numel() - a), device="cuda", generator=g)
        flat[a:a + step] = (part * 64).to(x.dtype) if fp8 else part.to(x.dtype)
    return x.view(torch.uint8) if fp8 else x


def prepare(case, seed):
    rng = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    order = list(range(case["seqs"]))
    rng.shuffle(order)
    shape = [_shape(case)[i] for i in order]
    b, hk, hq, d = case["block"], case["hk"], case["hq"], case["d"]
    pages = [-(-c // b) for c, _ in shape]
    total = sum(pages)
    width = max(pages)
    perm = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    tables = torch.full((len(shape), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(pages):
        tables[s, :n] = perm[at:at + n]
        at += n
    st = dict(op=case["op"], fp8=case["fp8"], block=b, tables=tables,
              scale=float(torch.tensor(1 / math.sqrt(d), dtype=torch.float32)),
              lens=torch.tensor([c for c, _ in shape], dtype=torch.int32, device="cuda"),
              max_context=max(c for c, _ in shape), ks=None, vs=None)
    layers = case.get("layers", 1)
    st["k"] = [_pool((total, hk, b, d), case["fp8"], g) for _ in range(layers)]
    st["v"] = [_pool((total, hk, b, d), case["fp8"], g) for _ in range(layers)]
    if case["fp8"]:
        st["ks"] = (torch.rand(hk, device="cuda", generator=g) + 0.5) / 64
        st["vs"] = (torch.rand(hk, device="cuda", generator=g) + 0.5) / 64
    starts = [0]
    for _, n in shape:
        starts.append(starts[-1] + n)
    st["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    st["max_draft"] = max(n for _, n in shape)
    if case["op"] == "accept":
        paths = [_paths(case)[i] for i in order]
        st["count"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
        most = max(1, max(len(p) for p in paths))
        st["accepted"] = torch.tensor([p + [0] * (most - len(p)) for p in paths],
                                      dtype=torch.int32, device="cuda")
        return st
    # queries a little longer than unit rows, so that some tokens stand out
    q = 2 * torch.randn(starts[-1], hq, d, device="cuda", generator=g)
    st["q"] = q.to(torch.bfloat16)
    if case["op"] == "window":
        st["window"], st["sinks"] = case["window"], case["sinks"]
        return st
    st["mask"] = None
    if not case["chain"]:
        # a tree grown in order: each draft hangs below one of the four before it
        masks = []
        for _, n in shape:
            mine = [1]
            for i in range(1, n):
                mine.append(mine[rng.randint(max(0, i - 4), i - 1)] | (1 << i))
            masks += [m - (1 << 64) if m >> 63 else m for m in mine]
        st["mask"] = torch.tensor(masks, dtype=torch.int64, device="cuda")
    return st


# ------------------------------------------------------------- plain forms

def _gather(st, pool, scale, pos):
    """fp32 rows [S, T, Hk, D] of the tokens at positions pos [S, T]."""
    page = torch.gather(st["tables"], 1, (pos // st["block"]).long()).long().clamp(min=0)
    rows = (pool.view(torch.float8_e4m3fn) if st["fp8"] else pool)[page, :, (pos % st["block"])]
    rows = rows.float()
    return rows * scale[:, None] if st["fp8"] else rows


def _attend(st, q, pos, see):
    """q [S, T, Hq, D] over the tokens at pos [S, L] where see [S, T, L]."""
    k = _gather(st, st["k"][0], st["ks"], pos)
    v = _gather(st, st["v"][0], st["vs"], pos)
    s, t, hq, d = q.shape
    hk = k.shape[2]
    rows = q.float().view(s, t, hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(s, hk, -1, d)
    z = rows @ k.permute(0, 2, 3, 1) * st["scale"]
    hide = ~see[:, None, :, None, :]
    z = z.view(s, hk, t, hq // hk, -1).masked_fill(hide, -math.inf)
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1)
    o = (e.view(s, hk, -1, e.shape[-1]) @ v.permute(0, 2, 1, 3)).view(s, hk, t, hq // hk, d)
    o = torch.where(total[..., None] > 0, o / total[..., None].clamp(min=1e-38),
                    torch.zeros_like(o))
    return o.permute(0, 2, 1, 3, 4).reshape(s, t, hq, d).to(torch.bfloat16)


def _plain_window(st):
    ctx = st["lens"].long()[:, None]
    dev = ctx.device
    first = torch.arange(st["sinks"], device=dev)[None]
    last = ctx - st["window"] + torch.arange(st["window"], device=dev)[None]
    pos = torch.cat([first.expand(ctx.shape[0], -1), last], 1)
    see = torch.cat([first < ctx - st["window"], last >= 0], 1)
    pos = torch.where(see, pos, torch.zeros_like(pos))
    return _attend(st, st["q"][:, None], pos, see[:, None])[:, 0]


def _plain_tree(st):
    start = st["q_start"].long()
    ctx = st["lens"].long()
    n = start[1:] - start[:-1]
    dev = ctx.device
    i = torch.arange(st["max_draft"], device=dev)
    row = (start[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    pos = torch.arange(st["max_context"], device=dev)
    bit = pos[None] - (ctx - n)[:, None]  # the draft a position holds; negative: committed
    mask = (2 << i).expand_as(row) - 1 if st["mask"] is None else st["mask"][row]
    drawn = (mask[:, :, None] >> bit.clamp(0, 63)[:, None]) & 1
    inside = (pos[None] < ctx[:, None])[:, None]
    see = ((bit < 0)[:, None] | (drawn > 0)) & inside
    pos = torch.where(inside[:, 0], pos[None].expand(ctx.shape[0], -1), torch.zeros_like(bit))
    o = _attend(st, st["q"][row], pos, see)
    at = torch.arange(st["q"].shape[0], device=dev)
    seq = torch.searchsorted(start, at, right=True) - 1
    return o[seq, at - start[seq]]


def _plain_accept(st):
    start = st["q_start"].long()
    base = st["lens"].long() - (start[1:] - start[:-1])
    k = torch.arange(st["accepted"].shape[1], device=base.device)[None]
    live = k < st["count"][:, None]
    # a list's padding writes rows behind the accepted ones onto themselves
    dst = torch.minimum(base[:, None] + k, st["lens"][:, None] - 1).long()
    src = torch.where(live, base[:, None] + st["accepted"], dst)
    b = st["block"]
    sp, dp = (torch.gather(st["tables"], 1, x // b).long() for x in (src, dst))
    pools = st["k"] + st["v"]
    rows = [p[sp, :, src % b] for p in pools]
    for p, r in zip(pools, rows):
        p.transpose(1, 2).index_put_((dp, dst % b), r)
    return (base + st["count"]).to(torch.int32)


def run(st):
    if own:
        import paged_kv_cache_220_gb300 as pkv
        if st["op"] == "window":
            return pkv.paged_attention_window(
                st["q"], st["k"][0], st["v"][0], st["tables"], st["lens"], st["scale"],
                st["max_context"], st["window"], st["sinks"], k_scale=st["ks"], v_scale=st["vs"])
        if st["op"] == "tree":
            return pkv.paged_attention_tree(
                st["q"], st["k"][0], st["v"][0], st["tables"], st["lens"], st["q_start"],
                st["scale"], st["max_context"], st["max_draft"], st["mask"],
                k_scale=st["ks"], v_scale=st["vs"])
        lens = pkv.kv_cache_accept(st["k"], st["v"], st["tables"], st["lens"], st["q_start"],
                                   st["accepted"], st["count"])
    elif st["op"] == "window":
        return _plain_window(st)
    elif st["op"] == "tree":
        return _plain_tree(st)
    else:
        lens = _plain_accept(st)
    see = (lambda p: p.view(torch.float8_e4m3fn)) if st["fp8"] else (lambda p: p)
    return [lens, [see(p) for p in st["k"][:2]], [see(p) for p in st["v"][:2]],
            see(st["k"][-1]), see(st["v"][-1])]


# ------------------------------------------------------------ work, exact

def work(case):
    hk, hq, d = case["hk"], case["hq"], case["d"]
    row = 2 * hk * d * (1 if case["fp8"] else 2)  # one token's K and V
    shape = _shape(case)
    if case["op"] == "accept":
        moved = sum(sum(1 for k, a in enumerate(p) if a != k) for p in _paths(case))
        return {"bytes": 2 * moved * row * case["layers"] + 12 * len(shape), "flops": 0}
    if case["op"] == "window":
        seen = [min(c, case["window"]) + min(case["sinks"], max(0, c - case["window"]))
                for c, _ in shape]
    else:
        seen = [c for c, _ in shape]
    return {"bytes": sum(t * row + 4 * -(-t // case["block"]) + 4 * n * hq * d
                         for t, (_, n) in zip(seen, shape)),
            "flops": sum(4 * t * n * hq * d for t, (_, n) in zip(seen, shape))}


def exact(case, seed):
    st = prepare(case, seed)
    lens, starts = st["lens"].tolist(), st["q_start"].tolist()
    tables, b = st["tables"].tolist(), case["block"]
    if case["op"] == "accept":
        lists, count = st["accepted"].tolist(), st["count"].tolist()
        pools = [p.view(torch.float8_e4m3fn) if case["fp8"] else p for p in st["k"] + st["v"]]
        src, dst, new = [], [], []
        for s, c in enumerate(lens):
            base = c - (starts[s + 1] - starts[s])
            new.append(base + count[s])
            for k in range(count[s]):
                f, t = base + lists[s][k], base + k
                src.append(tables[s][f // b] * b + f % b)
                dst.append(tables[s][t // b] * b + t % b)
        src, dst = (torch.tensor(x, dtype=torch.long, device="cuda") for x in (src, dst))
        n = len(st["k"])
        want = sorted({0, min(1, n - 1), n - 1})
        done = {}
        for i in [*want, *(n + w for w in want)]:
            flat = pools[i].double().permute(0, 2, 1, 3).reshape(-1, case["hk"], case["d"])
            old = flat.clone()
            flat[dst] = old[src]
            flat = flat.view(-1, b, case["hk"], case["d"]).permute(0, 2, 1, 3).contiguous()
            done[i] = flat
        return [torch.tensor(new, dtype=torch.int32), [done[i] for i in range(min(2, n))],
                [done[n + i] for i in range(min(2, n))], done[n - 1], done[2 * n - 1]]
    hk, hq, d = case["hk"], case["hq"], case["d"]
    g = hq // hk
    q = st["q"].double()
    out = torch.zeros_like(q)
    masks = None if st.get("mask") is None else st["mask"].tolist()
    for s, c in enumerate(lens):
        page = torch.tensor(tables[s][: -(-c // b)], dtype=torch.long, device="cuda")
        kv = []
        for pool, scale in ((st["k"][0], st["ks"]), (st["v"][0], st["vs"])):
            x = (pool.view(torch.float8_e4m3fn) if case["fp8"] else pool)[page].double()
            x = x.permute(1, 0, 2, 3).reshape(hk, -1, d)[:, :c]
            kv.append(x * scale.double()[:, None, None] if case["fp8"] else x)
        n = starts[s + 1] - starts[s]
        hide = torch.zeros(n, c, dtype=torch.bool, device="cuda")
        if case["op"] == "window":
            hide[:, case["sinks"]:max(case["sinks"], c - case["window"])] = True
        else:
            see = [[(masks[starts[s] + i] >> j) & 1 if masks else int(j <= i) for j in range(n)]
                   for i in range(n)]
            hide[:, c - n:] = torch.tensor(see, device="cuda") == 0
        mine = q[starts[s]:starts[s + 1]].view(n, hk, g, d)
        z = torch.einsum("nhgd,htd->hngt", mine, kv[0]) * st["scale"]
        z.masked_fill_(hide[None, :, None, :], -math.inf)
        o = torch.einsum("hngt,htd->nhgd", torch.softmax(z, -1), kv[1])
        out[starts[s]:starts[s + 1]] = o.reshape(n, hq, d)
    return out
