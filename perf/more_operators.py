"""Cases for the operators of a batch that shares prefixes and lives within a
budget: attention of the newest tokens over a paged cache whose sequences share
their first pages, the attention weight that each cached token has received,
and the eviction of the tokens that received least.

Every case is one call of a serving program, over one attention layer:
`prepare` makes what the program has in hand before it, `run` is the pass, in
elementary torch operations or, with `own`, through the library; `exact` is the
operators' definition in 64 bits, written apart from both.

The cache is the library's bf16 one: pools [blocks][KV heads][page][128] and a
block table.  Weights (float) and positions (int32) of the cached tokens lie in
pools [blocks][KV heads][page] beside it.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128                      # head dimension of the cache


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _prefix(name, batch, groups, hq, hkv, page, prefix, suffix, rows=1, empty=False):
    return dict(name=name, op="prefix", batch=batch, groups=groups, hq=hq, hkv=hkv, page=page,
                prefix=prefix, suffix=suffix, rows=rows, empty=empty)


def _weigh(name, batch, hq, hkv, page, ctx, rows=1, fixed=0, decay=1.0, fresh=False):
    return dict(name=name, op="weigh", batch=batch, hq=hq, hkv=hkv, page=page, ctx=ctx, rows=rows,
                fixed=fixed, decay=decay, fresh=fresh)


def _evict(name, batch, hq, hkv, page, ctx, budget, recent, fixed=0, settled=False):
    return dict(name=name, op="evict", batch=batch, hq=hq, hkv=hkv, page=page, ctx=ctx,
                budget=budget, recent=recent, fixed=fixed, settled=settled)


def listed():
    return [
        # four short answers to one short instruction, small pages: latency
        _prefix("prefix_short", 4, 1, 32, 8, 16, 512, 64),
        # a batch of conversations behind one system prompt
        _prefix("prefix_system_8k", 32, 1, 32, 8, 64, 8192, 2048),
        # questions about one long document
        _prefix("prefix_document_32k", 64, 1, 32, 8, 64, 32768, 512),
        # a mixed batch: five prefixes (one of them empty), a padded sequence, five heads to a KV head
        _prefix("prefix_mixed", 24, 5, 40, 8, 32, 4001, 999, empty=True),
        # six drafted tokens a sequence to be verified at once
        _prefix("prefix_draft", 16, 1, 32, 8, 64, 4096, 1024, rows=6),
        # many samples of one prompt, eight heads to a KV head: the tensor cores' case
        _prefix("prefix_samples_16k", 256, 1, 64, 8, 64, 16384, 256),
        # a decode step's weights in two short sequences: latency
        _weigh("weigh_short", 2, 32, 8, 16, 1000),
        # a decode step's weights in a batch kept at a budget, older weights fading
        _weigh("weigh_step", 32, 32, 8, 64, 4224, fixed=64, decay=0.99),
        # the last 32 queries of four long prompts vote on every token
        _weigh("weigh_prompt_32k", 4, 32, 8, 64, 32768, rows=32, fresh=True),
        # a decode step of a batch kept at a budget: one token too many in each head
        _evict("evict_step", 32, 32, 8, 64, 4161, 4096, 256, fixed=64, settled=True),
        # four long prompts cut to their budget
        _evict("evict_prompt_32k", 4, 32, 8, 64, 32768, 4096, 256, fixed=4),
        # one very long prompt in small pages
        _evict("evict_prompt_128k", 1, 32, 8, 16, 131071, 8192, 1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "weigh", "evict"])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    page = rng.choice([16, 32, 64])
    batch = _log(rng, 1, 256 if op == "prefix" else 64)
    rows = rng.choice([1, 1, 1, rng.randint(1, 8)])
    if op == "prefix":
        suffix = _log(rng, 1, max(1, min(4096, (1 << 18) // (batch * hkv))))
        groups = rng.randint(1, min(batch, 6))
        most = min(32768, (1 << 28) // (batch * hkv * g * rows), (1 << 18) // (groups * hkv))
        c = _prefix("", batch, groups, hkv * g, hkv, page, _log(rng, 1, max(1, most)), suffix,
                    rows, batch > 1 and rng.random() < 0.3)
    else:
        most = max(64, (1 << 20) // (batch * hkv))
        ctx = _log(rng, 9, min(most, 131072))
        fixed = rng.choice([0, 0, 4, rng.randint(0, ctx // 2)])
        if op == "weigh":
            rows = min(rng.choice([1, 1, 8, rng.randint(1, 32)]), 128 // g, ctx)
            c = _weigh("", batch, hkv * g, hkv, page, ctx, rows, fixed, rng.choice([1.0, 0.95]), rng.random() < 0.4)
        else:
            budget = _log(rng, 1, min(8192, ctx))
            c = _evict("", batch, hkv * g, hkv, page, ctx, budget, rng.randint(0, budget), fixed, rng.random() < 0.3)
    del c["name"]
    return c


def _rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _groups(case):
    """(first sequence of each group and the batch's end, prefix pages of each group, lengths)."""
    r = _rng(case)
    batch, n, page = case["batch"], case["groups"], case["page"]
    starts = [0] + sorted(r.sample(range(1, batch), n - 1)) + [batch]
    pages = [case["prefix"] // page] + [r.randint(0, case["prefix"] // page) for _ in range(n - 1)]
    if n > 1:
        pages[-1] = 0
    lens = []
    for a, b, p in zip(starts, starts[1:], pages):
        lens += [p * page + max(case["rows"], r.randint(1, case["suffix"])) for _ in range(a, b)]
    lens[-1] = pages[-1] * page + max(case["rows"], case["suffix"])
    if case["empty"]:
        lens[0] = 0
    return starts, pages, lens


def _lens(case):
    """Cached tokens of each sequence (weigh, evict): the last one has them all."""
    if case.get("settled"):
        return [case["ctx"]] * case["batch"]
    r = _rng(case)
    lo = max(1, case.get("rows", 1), case["ctx"] * 3 // 4)
    return [r.randint(min(lo, case["ctx"]), case["ctx"]) for _ in range(case["batch"] - 1)] + [case["ctx"]]


# --------------------------------------------------------------------------
# state
# --------------------------------------------------------------------------
def _pool(blocks, hkv, page, gen, keys):
    """A pool of bf16 pages.  Keys have a few strong channels and a common part, as keys after a
    rotation do; values are nearly normal with a spread of sizes over the tokens."""
    pool = torch.empty(blocks, hkv, page, D, dtype=torch.bfloat16, device="cuda")
    loud = torch.where(torch.rand(hkv, 1, D, generator=gen, device="cuda") < 0.05, 3.0, 0.6)
    mean = torch.randn(hkv, 1, D, generator=gen, device="cuda") * 0.5
    step = max(1, (1 << 26) // (hkv * page * D))
    for a in range(0, blocks, step):
        n = min(step, blocks - a)
        x = torch.randn(n, hkv, page, D, generator=gen, device="cuda")
        if keys:
            x = x * loud + mean
        else:
            x *= torch.exp(0.5 * torch.randn(n, hkv, page, 1, generator=gen, device="cuda"))
        pool[a:a + n] = x
    return pool


def _ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)
    batch, hq, hkv, page = (case[k] for k in ("batch", "hq", "hkv", "page"))
    s = {"case": case}
    if case["op"] == "prefix":
        starts, prefix, lens = _groups(case)
        pages = max(1, max(-(-n // page) for n in lens), max(prefix))
        shared = sum(prefix)
        own_pages = [max(0, -(-n // page) - p) for a, b, p in zip(starts, starts[1:], prefix) for n in lens[a:b]]
        blocks = shared + sum(own_pages) + 3
        perm = torch.randperm(blocks, generator=gen, device="cuda").int()
        table = torch.full((batch, pages), -1, dtype=torch.int32, device="cuda")
        at, mine = 0, shared
        for a, b, p in zip(starts, starts[1:], prefix):
            table[a:b, :p] = perm[at:at + p]
            at += p
            for i in range(a, b):
                table[i, p:p + own_pages[i]] = perm[mine:mine + own_pages[i]]
                mine += own_pages[i]
        s["starts"], s["prefix"] = _ints(starts), _ints(prefix)
        s["host"] = starts, prefix, lens          # a serving program knows its batch
    else:
        lens = _lens(case)
        pages = -(-max(lens) // page)
        blocks = batch * pages + 3
        table = torch.randperm(blocks, generator=gen, device="cuda").int()[:batch * pages].reshape(batch, pages)
        s["fixed"] = _ints([case["fixed"]] * batch)
    s["table"] = table.contiguous()
    s["blocks"] = blocks
    s["k"] = _pool(blocks, hkv, page, gen, True)
    if case["op"] != "weigh":
        s["v"] = _pool(blocks, hkv, page, gen, False)
    if case["op"] != "evict":
        s["q"] = torch.randn(batch, case["rows"], hq, D, generator=gen, device="cuda").bfloat16()
        s["lens"] = _ints(lens)
    if case["op"] == "weigh":
        s["lse"] = _lse(s)
        # weights of earlier steps: a few tokens hold most
        s["weights"] = None if case["fresh"] else torch.exp(
            2 * torch.randn(blocks, hkv, page, generator=gen, device="cuda"))
        s["gone"] = torch.randint(0, 1 << 20, (batch,), generator=gen, device="cuda").int()
        s["out"] = torch.zeros(blocks, hkv, page, device="cuda")
        s["pos"] = torch.zeros(blocks, hkv, page, dtype=torch.int32, device="cuda")
    if case["op"] == "evict":
        _evict_state(s, lens, gen)
    if own:
        _handles(s)
    return s


def _evict_state(s, lens, gen):
    """Weights, positions, lengths and counts of what is gone, in one buffer: a pass works in place,
    and the next one begins with a copy of what `prepare` made."""
    case, table = s["case"], s["table"]
    batch, hkv, page = case["batch"], case["hkv"], case["page"]
    n, cap = s["blocks"] * hkv * page, table.shape[1] * page
    weights = torch.exp(2 * torch.randn(batch, hkv, cap, generator=gen, device="cuda"))
    # some tokens were never looked at: equal weights
    weights = torch.where(torch.rand(batch, hkv, cap, generator=gen, device="cuda") < 0.05, 0.0, weights)
    pos = torch.arange(cap, dtype=torch.int32, device="cuda").expand(batch, hkv, cap).contiguous()
    gone = [0] * batch
    if case["settled"]:
        # earlier steps have put later tokens into the places of evicted ones: the newest token is
        # last, the other recent ones lie anywhere behind the fixed ones
        ctx, fixed, gone = case["ctx"], case["fixed"], [1000] * batch
        u = torch.rand(batch, hkv, ctx - 1 - fixed, generator=gen, device="cuda")
        held = u.argsort(-1).int()
        old = max(0, ctx - fixed - max(case["recent"], 1))
        held = torch.where(held < old, held, held + 1000) + fixed
        pos[..., fixed:ctx - 1] = held
        pos[..., ctx - 1] = ctx + 999
    buf = torch.zeros(2 * n + 2 * batch, dtype=torch.int32, device="cuda")
    s["saved"], s["live"] = buf, torch.empty_like(buf)
    for b, x in ((0, weights.view(torch.int32)), (n, pos)):
        pool = buf[b:b + n].view(s["blocks"], hkv, page)
        pool[table.long()] = x.reshape(batch, hkv, -1, page).transpose(1, 2)
    buf[2 * n:2 * n + batch], buf[2 * n + batch:] = _ints(lens), _ints(gone)
    live = s["live"]
    s["weights"] = live[:n].view(torch.float32).view(s["blocks"], hkv, page)
    s["pos"] = live[n:2 * n].view(s["blocks"], hkv, page)
    s["lens"], s["gone"] = live[2 * n:2 * n + batch], live[2 * n + batch:]
    live.copy_(buf)


def _handles(s):
    """What a user of the library keeps: the configuration, output buffers, workspaces."""
    from sparse_paged_kv_gb300 import binding as B
    case = s["case"]
    batch, hq, hkv = case["batch"], case["hq"], case["hkv"]
    s["cfg"] = cfg = B.LocksConfig(batch=batch, n_q_heads=hq, n_kv_heads=hkv, head_dim=D, page_size=case["page"], rank=8,
                                   max_pages=s["table"].shape[1], num_blocks=s["blocks"])
    size = 0
    if case["op"] == "prefix":
        s["o"] = torch.empty(batch, case["rows"], hq, D, dtype=torch.bfloat16, device="cuda")
        s["o_lse"] = torch.empty(batch, case["rows"], hq, dtype=torch.float32, device="cuda")
        size = B.prefix_workspace_bytes(cfg, case["groups"], case["rows"])
    if case["op"] == "evict":
        size = B.evict_workspace_bytes(cfg, case["budget"])
    s["ws"] = torch.zeros(max(1, size), dtype=torch.uint8, device="cuda")


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from sparse_paged_kv_gb300 import binding as B
    case = s["case"]
    if case["op"] == "prefix":
        B.locks_prefix_decode(s["cfg"], s["q"], s["k"], s["v"], s["table"], s["lens"], s["starts"], s["prefix"], s["o"],
                              s["ws"], out_lse=s["o_lse"])
        return {"out": s["o"], "lse": s["o_lse"]}
    if case["op"] == "weigh":
        B.locks_weigh(s["cfg"], s["q"], s["lse"], s["k"], s["table"], s["lens"], s["weights"], s["out"], n_new=case["rows"],
                      decay=case["decay"], fixed=s["fixed"], positions=s["pos"], evicted=s["gone"])
        return {"weights": s["out"], "pos": s["pos"]}
    s["live"].copy_(s["saved"])
    B.locks_evict(s["cfg"], case["budget"], case["recent"], s["k"], s["v"], s["table"], s["lens"], s["weights"], s["pos"],
                  s["gone"], s["ws"], fixed=s["fixed"])
    return {n: s[n] for n in ("k", "v", "weights", "pos", "lens", "gone")}


def _run_plain(s):
    op = s["case"]["op"]
    if op == "prefix":
        return _plain_prefix(s)
    if op == "weigh":
        return _plain_weigh(s)
    s["live"].copy_(s["saved"])
    return _plain_evict(s)


def _limits(s):
    """[batch][rows]: how many slots each query sees (the last one all of them)."""
    rows = s["case"]["rows"]
    return (s["lens"].long()[:, None] - (rows - 1) + torch.arange(rows, device="cuda")).clamp(min=0)


def _queries(s):
    """float32 [batch][KV heads][rows * group][128]."""
    c = s["case"]
    q = s["q"].float().unflatten(2, (c["hkv"], -1))
    return q.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _gather(pool, table):
    """[..., KV heads, pages * page, ...] of a block table [..., pages]."""
    return pool[table.long().clamp(min=0)].transpose(-4, -3).flatten(-3, -2)


def _plain_prefix(s):
    c = s["case"]
    g = c["hq"] // c["hkv"]
    starts, prefix, lens = s["host"]
    q = _queries(s) * (1 / math.sqrt(D))
    seen = _limits(s).repeat_interleave(g, 1)                      # [batch][rows * group]
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(q.shape[:-1], device="cuda")
    for a, b, p in zip(starts, starts[1:], prefix):
        n, own_pages = b - a, max(0, -(-max(lens[a:b]) // c["page"]) - p)
        qg, lim = q[a:b], seen[a:b, None, :, None]
        parts, first = [], p * c["page"]
        shared, mine = s["table"][a, :p], s["table"][a:b, p:p + own_pages]
        if p:       # [heads][all rows of the group][prefix]
            x = torch.matmul(qg.transpose(0, 1).flatten(1, 2), _gather(s["k"], shared).float().transpose(-1, -2))
            parts.append(x.unflatten(1, (n, -1)).transpose(0, 1))
        if own_pages:
            parts.append(torch.matmul(qg, _gather(s["k"], mine).float().transpose(-1, -2)))
        if not parts:
            out[a:b], lse[a:b] = 0, -math.inf
            continue
        x = torch.cat(parts, -1)
        x = torch.where(torch.arange(x.shape[-1], device="cuda") < lim, x, -math.inf)
        m = x.amax(-1, keepdim=True)
        w = torch.exp(x - torch.where(torch.isinf(m), 0.0, m))
        total = w.sum(-1, keepdim=True)
        y = 0.0
        if p:
            y = torch.matmul(w[..., :first].transpose(0, 1).flatten(1, 2), _gather(s["v"], shared).float())
            y = y.unflatten(1, (n, -1)).transpose(0, 1)
        if own_pages:
            y = y + torch.matmul(w[..., first:], _gather(s["v"], mine).float())
        out[a:b] = (y / torch.where(total > 0, total, 1.0)).to(torch.bfloat16)
        z = (torch.log(total) + m).squeeze(-1)
        lse[a:b] = torch.where(torch.isnan(z), -math.inf, z)
    shape = (c["batch"], c["hkv"], c["rows"], g)
    return {"out": out.reshape(*shape, D).transpose(1, 2).flatten(2, 3).contiguous(),
            "lse": lse.reshape(shape).transpose(1, 2).flatten(2, 3).contiguous()}


def _lse(s):
    """log-sum-exp of every query of `weigh`, as the attention before it gave it."""
    c = s["case"]
    g = c["hq"] // c["hkv"]
    q, lim = _queries(s) * (1 / math.sqrt(D)), _limits(s).repeat_interleave(g, 1)
    got = torch.empty(q.shape[:-1], device="cuda")
    for b in range(c["batch"]):
        x = torch.matmul(q[b], _gather(s["k"], s["table"][b]).float().transpose(-1, -2))
        x = torch.where(torch.arange(x.shape[-1], device="cuda") < lim[b, :, None], x, -math.inf)
        got[b] = torch.logsumexp(x, -1)
    return got.reshape(c["batch"], c["hkv"], c["rows"], g).transpose(1, 2).flatten(2, 3).contiguous()


def _plain_weigh(s):
    c = s["case"]
    batch, hkv, page, rows = c["batch"], c["hkv"], c["page"], c["rows"]
    g = c["hq"] // hkv
    lim = _limits(s).repeat_interleave(g, 1)[:, None, :, None]
    lse = s["lse"].unflatten(2, (hkv, g)).permute(0, 2, 1, 3).flatten(2, 3).unsqueeze(-1)
    x = torch.matmul(_queries(s), _gather(s["k"], s["table"]).float().transpose(-1, -2)) * (1 / math.sqrt(D))
    slot = torch.arange(x.shape[-1], device="cuda")
    add = torch.where(slot < lim, torch.exp(x - lse), 0.0).sum(2)                     # [batch][heads][slots]
    n = s["lens"].long()[:, None, None]
    new = slot >= n - rows
    if s["weights"] is not None:
        add += torch.where(new, 0.0, _gather(s["weights"].unsqueeze(-1), s["table"]).squeeze(-1) * c["decay"])
    else:
        new = torch.ones_like(new)
    there = (slot < n) & (slot >= s["fixed"].long()[:, None, None])
    where = s["gone"].long()[:, None, None] + slot
    for pool, what, at in ((s["out"], add, there), (s["pos"], where.int(), there & new)):
        b, h, t = torch.nonzero(at.expand(batch, hkv, -1), as_tuple=True)
        pool[s["table"].long()[b, t // page], h, t % page] = what.expand(batch, hkv, -1)[b, h, t]
    return {"weights": s["out"], "pos": s["pos"]}


def _plain_evict(s):
    c = s["case"]
    page, keep = c["page"], c["budget"]
    table, n = s["table"].long(), s["lens"].long()[:, None, None]
    weights, pos = (_gather(x.unsqueeze(-1), table).squeeze(-1) for x in (s["weights"], s["pos"]))
    slot = torch.arange(weights.shape[-1], device="cuda")
    first = torch.minimum(s["fixed"].long()[:, None, None], n)
    there = (slot >= first) & (slot < n)
    recent = pos >= n + s["gone"].long()[:, None, None] - c["recent"]
    key = torch.where(recent, math.inf, weights)
    key = torch.where(there, key, -math.inf)
    rank = torch.empty_like(key, dtype=torch.long)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank.scatter_(-1, order, slot.expand_as(order))
    kept = there & (rank < keep)
    over = n - first > keep
    src = torch.nonzero(kept & over & (slot >= first + keep), as_tuple=True)
    dst = torch.nonzero(there & ~kept & over & (slot < first + keep), as_tuple=True)
    place = lambda x: (table[x[0], x[2] // page], x[1], x[2] % page)  # noqa: E731
    src, dst = place(src), place(dst)
    for pool in (s["k"], s["v"], s["weights"], s["pos"]):
        pool[dst] = pool[src]
    drop = (n - first - keep).clamp(min=0)[:, 0, 0].int()
    s["lens"] -= drop
    s["gone"] += drop
    return {x: s[x] for x in ("k", "v", "weights", "pos", "lens", "gone")}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    hq, hkv, page, batch = case["hq"], case["hkv"], case["page"], case["batch"]
    if case["op"] == "prefix":
        starts, prefix, lens = _groups(case)
        rows, tokens, pairs = case["rows"], 0, 0
        for a, b, p in zip(starts, starts[1:], prefix):
            tokens += p * page + sum(max(0, n - p * page) for n in lens[a:b])
            pairs += sum(max(0, n - i) for n in lens[a:b] for i in range(rows))
        return {"bytes": tokens * hkv * 4 * D + batch * rows * hq * (4 * D + 4) + 4 * (tokens // page) + 4 * batch,
                "flops": 4 * D * hq * pairs}
    lens = _lens(case)
    seen = [max(0, n - case["fixed"]) for n in lens]
    if case["op"] == "weigh":
        rows = case["rows"]
        held = 4 if case["fresh"] else 8
        return {"bytes": sum(seen) * hkv * (2 * D + held) + batch * rows * hq * (2 * D + 4) + 4 * (sum(seen) // page),
                "flops": 2 * D * hq * sum(max(0, n - i) for n in seen for i in range(rows))}
    keep, moved = case["budget"], 0
    for n in seen:
        if n <= keep:
            continue
        if case["settled"]:
            moved += -(-keep * (n - keep) // n)
            continue
        # of the kept tokens, the recent ones are the last; the others lie anywhere before
        late = min(case["recent"], n - keep) + max(0, keep - case["recent"]) * max(0, n - keep - case["recent"]) / max(1, n - case["recent"])
        moved += int(min(late, keep, n - keep))
    return {"bytes": sum(n for n in seen if n > keep) * hkv * 8 + moved * hkv * (8 * D + 8) + 16 * batch, "flops": 0}


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"prefix": _exact_prefix, "weigh": _exact_weigh, "evict": _exact_evict}[case["op"]](s)


def _slots(s, b, h, n, pool):
    """The first n slots of sequence b in KV head h."""
    page = s["case"]["page"]
    blk = s["table"][b, :-(-n // page)].long()
    return pool[blk, h].reshape(-1, *pool.shape[3:])[:n]


def _exact_prefix(s):
    c = s["case"]
    g = c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:-1], -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        for h in range(c["hkv"]):
            if n == 0:
                continue
            k, v = (_slots(s, b, h, n, s[x]).double() for x in "kv")
            heads = slice(h * g, h * g + g)
            z = s["q"][b, :, heads].double() @ k.T / math.sqrt(D)          # [rows][group][n]
            for r in range(c["rows"]):
                m = n - c["rows"] + r + 1
                if m > 0:
                    lse[b, r, heads] = torch.logsumexp(z[r, :, :m], -1)
                    out[b, r, heads] = torch.exp(z[r, :, :m] - lse[b, r, heads][:, None]) @ v[:m]
    return {"out": out, "lse": lse}


def _exact_weigh(s):
    c = s["case"]
    g, page = c["hq"] // c["hkv"], c["page"]
    out, pos = s["out"].double(), s["pos"].clone()
    for b, n in enumerate(s["lens"].tolist()):
        first = c["fixed"]
        if first >= n:
            continue
        t = torch.arange(first, n, device="cuda")
        blk = s["table"][b].long()[t // page]
        for h in range(c["hkv"]):
            k = _slots(s, b, h, n, s["k"]).double()[first:]
            total = torch.zeros(n - first, dtype=torch.float64, device="cuda")
            for r in range(c["rows"]):
                heads = slice(h * g, h * g + g)
                p = torch.exp(s["q"][b, r, heads].double() @ k.T / math.sqrt(D) - s["lse"][b, r, heads].double()[:, None])
                total += torch.where(t < n - c["rows"] + r + 1, p.sum(0), 0.0)
            if s["weights"] is not None:
                old = _slots(s, b, h, n, s["weights"]).double()[first:] * c["decay"]
                total += torch.where(t < n - c["rows"], old, 0.0)
                fresh = t >= n - c["rows"]
            else:
                fresh = t >= 0
            out[blk, h, t % page] = total
            pos[blk[fresh], h, t[fresh] % page] = (t[fresh] + s["gone"][b]).int()
    return {"weights": out, "pos": pos}


def _exact_evict(s):
    c = s["case"]
    page, keep = c["page"], c["budget"]
    lens, gone = s["lens"].tolist(), s["gone"].tolist()
    table = s["table"].cpu().numpy()
    weights, pos = s["weights"].cpu().numpy(), s["pos"].cpu().numpy()
    moves = [[], []]
    for b, n in enumerate(lens):
        first = min(c["fixed"], n)
        if n - first <= keep:
            continue
        t = np.arange(first, n)
        for h in range(c["hkv"]):
            at = (table[b, t // page], h, t % page)
            w = np.where(pos[at] >= n + gone[b] - c["recent"], np.inf, weights[at].astype(np.float64))
            best = np.sort(t[np.lexsort((t, -w))[:keep]])
            late = best[best >= first + keep]
            holes = np.setdiff1d(np.arange(first, first + keep), best)
            moves[0].append(np.stack([table[b, late // page], np.full(late.size, h), late % page]))
            moves[1].append(np.stack([table[b, holes // page], np.full(late.size, h), holes % page]))
        s["lens"][b] -= n - first - keep
        s["gone"][b] += n - first - keep
    if moves[0]:
        src, dst = (tuple(torch.from_numpy(np.concatenate(m, 1)).long().cuda()) for m in moves)
        for x in ("k", "v", "weights", "pos"):
            s[x][dst] = s[x][src]
    got = {x: s[x] for x in ("k", "v", "weights", "pos", "lens", "gone")}
    return {x: y.double() if y.is_floating_point() else y for x, y in got.items()}
