"""Cases for the quantised cache operators: rotary positions, writing a paged
key-value cache in 8 or 4 bits and reading it back, and the attention of one
new token over it.

Every case is one call (or the two or three calls that belong together) of a
serving program, over one attention layer: `prepare` makes what the program
has in hand before it, `run` is the pass, in elementary torch operations or,
with `own`, through the library; `exact` is the operators' definition in 64
bits, written apart from both.

The cache record of one (block, KV head) page, as include/locks.h describes
it: the token rows of codes (128 bytes, or 64 in 4 bits), their 16-byte chunks
permuted within the row, then (4 bits only) four e4m3 group scales a token,
then one float scale a token.
"""
import math
import random

import torch

own = False

D = 128                      # head dimension of the cache
FMT = {"f8": 0, "i8": 1, "i4": 2}
ROW = {"f8": 128, "i8": 128, "i4": 64}
TINY = 2.0 ** -96            # rows with no larger magnitude are stored as zeros

# Rotary scalings by name: none at the first models' base; the banded scaling of
# the Llama-3.1 layers; the ramped one (with its factor on cos and sin) for long contexts.
ROPE = {
    "none": dict(scaling="none", theta=10000.0),
    "linear": dict(scaling="linear", theta=10000.0, factor=4.0),
    "ntk": dict(scaling="ntk", theta=10000.0, factor=8.0),
    "llama3": dict(scaling="llama3", theta=500000.0, factor=8.0, low_freq_factor=1.0,
                   high_freq_factor=4.0, original_positions=8192.0),
    "yarn": dict(scaling="yarn", theta=1000000.0, factor=4.0, original_positions=32768.0,
                 beta_fast=32.0, beta_slow=1.0),
}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _rope(name, dtype, tokens, heads, total_heads, head_dim, rotary, layout, scaling, inverse, max_pos):
    return dict(name=name, op="rope", dtype=dtype, tokens=tokens, heads=heads,
                total_heads=total_heads, head_dim=head_dim, rotary=rotary, layout=layout,
                scaling=scaling, inverse=inverse, max_pos=max_pos)


def _write(name, fmt, seqs, tokens, start, hq, hkv, page, rotary, layout, scaling):
    return dict(name=name, op="write", fmt=fmt, batch=seqs, tokens=tokens, start=start, hq=hq,
                hkv=hkv, page=page, rotary=rotary, layout=layout, scaling=scaling)


def _attend(name, fmt, batch, hq, hkv, page, ctx, ragged=1.0, empty=False, k=0, window=0):
    return dict(name=name, op="attend", fmt=fmt, batch=batch, hq=hq, hkv=hkv, page=page, ctx=ctx,
                ragged=ragged, empty=empty, k=k, window=window)


def _step(name, fmt, batch, hq, hkv, page, ctx, ragged, scaling):
    return dict(name=name, op="step", fmt=fmt, batch=batch, hq=hq, hkv=hkv, page=page, ctx=ctx,
                ragged=ragged, empty=False, k=0, window=0, rotary=D, layout="half", scaling=scaling)


def listed():
    return [
        # queries and keys of one decode step of 16 sequences, taken out of the fused projection
        _rope("rope_step", "bf16", 16, 40, 48, 128, 128, "half", "llama3", False, 1 << 20),
        # a 32K prompt's queries and keys, long-context scaling
        _rope("rope_prompt", "bf16", 32768, 40, 48, 128, 128, "half", "yarn", False, 1 << 17),
        # the gradient through a partial, interleaved rotation of an odd-sized layer in float
        _rope("rope_back_f32", "f32", 2049, 17, 17, 80, 40, "interleaved", "linear", True, 1 << 14),
        # a prompt of two sequences into an 8-bit cache, and its pages read back for their summaries
        _write("write_prompt_f8", "f8", 2, 8192, 0, 32, 8, 64, 128, "half", "llama3"),
        # the later chunk of three ragged prompts into a 4-bit cache of small pages, partial rotation
        _write("write_chunk_i4", "i4", 3, 5001, 1003, 32, 8, 16, 64, "interleaved", "none"),
        # one short conversation: latency
        _attend("attend_short_f8", "f8", 1, 32, 8, 64, 1000),
        # the batch of 32K contexts that the benchmark's layer serves
        _attend("attend_32k_f8", "f8", 8, 32, 8, 64, 32768),
        # a mixed batch: lengths from nothing to 16K, small pages, 8-bit integers
        _attend("attend_mixed_i8", "i8", 16, 32, 8, 16, 16384, ragged=0.02, empty=True),
        # long contexts in 4 bits
        _attend("attend_128k_i4", "i4", 4, 32, 8, 64, 131072),
        # a million tokens
        _attend("attend_1m_f8", "f8", 1, 32, 8, 64, 1048576),
        # the pages a selection kept (budget 2048) out of 32K contexts, in 4 bits
        _attend("attend_selected_i4", "i4", 8, 32, 8, 64, 32768, k=32),
        # one whole decode step: rotate, write the token, attend; 16 ragged sequences
        _step("step_16k_f8", "f8", 16, 32, 8, 64, 16384, 0.25, "llama3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "attend", "attend", "attend", "step"])
    scaling = rng.choice(sorted(ROPE))
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    fmt, page = rng.choice(sorted(FMT)), rng.choice([16, 32, 64])
    if op == "rope":
        hd = rng.choice([64, 72, 80, 128, 192, 256])
        rot = rng.choice([hd, hd // 2])
        heads = rng.randint(1, 48)
        tokens = max(1, min(_log(rng, 1, 32768), 32768 * 40 * 128 // (heads * hd * 2)))
        c = _rope("", rng.choice(["bf16", "f16", "f32"]), tokens, heads, heads + rng.choice([0, 0, 8]),
                  hd, rot, rng.choice(["half", "interleaved"]), scaling, rng.random() < 0.3,
                  1 << rng.randint(12, 20))
    elif op == "write":
        rot = rng.choice([0, 32, 64, 96, 128, 128])
        c = _write("", fmt, rng.randint(1, 9), _log(rng, 9, 8192), rng.choice([0, rng.randint(1, 3000)]),
                   hkv * min(g, 8), hkv, page, rot, rng.choice(["half", "interleaved"]), scaling)
    else:
        batch = _log(rng, 1, 64)
        most = max(64, (1 << 20) // (batch * hkv))
        ctx = _log(rng, 1 if op == "attend" else 2, most)
        ragged = rng.choice([1.0, rng.uniform(0.0, 0.9)])
        if op == "step":
            c = _step("", fmt, batch, hkv * g, hkv, page, ctx, ragged, scaling)
        else:
            pages = -(-ctx // page)
            k = rng.choice([0, 0, min(256, rng.randint(2, max(2, pages)))])
            window = rng.choice([0, 0, 0, rng.randint(1, ctx)])
            c = _attend("", fmt, batch, hkv * g, hkv, page, ctx, ragged, batch > 1 and rng.random() < 0.3, k, window)
    del c["name"]
    return c


def _lens(case):
    """Tokens of each sequence (attend: attended; step: before the new one; write: written)."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    if case["op"] == "write":
        left, n = case["tokens"], []
        for i in range(case["batch"] - 1):
            n.append(min(left, r.randint(0, 2 * left // (case["batch"] - i))))
            left -= n[-1]
        return n + [left]
    hi = case["ctx"]
    n = [r.randint(max(1, int(case["ragged"] * hi)), hi) for _ in range(case["batch"])]
    n[-1] = hi
    if case["empty"]:
        n[0] = 0
    if case["op"] == "step":
        n = [x - 1 for x in n]
    return n


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------
def _inv_freq(rotary, scaling, theta, factor=1.0, low_freq_factor=1.0, high_freq_factor=1.0,
              original_positions=0.0, beta_fast=32.0, beta_slow=1.0):
    """(radians a position of each pair, float64; the factor on cos and sin)."""
    i = torch.arange(rotary // 2, dtype=torch.float64)
    if scaling == "ntk":
        theta = theta * factor ** (rotary / (rotary - 2))
    inv = torch.exp(-math.log(theta) * 2 * i / rotary)
    if scaling == "linear":
        inv = inv / factor
    if scaling == "llama3":
        turns = original_positions * inv / (2 * math.pi)      # full turns within the original context
        keep = ((turns - low_freq_factor) / (high_freq_factor - low_freq_factor)).clamp(0, 1)
        inv = (1 - keep) * inv / factor + keep * inv
    if scaling == "yarn":
        def at(turns):
            return rotary * math.log(original_positions / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo = max(0, math.floor(at(beta_fast)))
        hi = min(rotary - 1, math.ceil(at(beta_slow)))
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        inv = inv / factor * ramp + inv * (1 - ramp)
        return inv, 0.1 * math.log(factor) + 1.0
    return inv, 1.0


def _rotate(x, pos, inv, mscale, layout, inverse=False):
    """x [tokens][heads][dim] in float32, rotated in its first 2 * len(inv) dims."""
    a = pos.double()[:, None] * inv
    c, s = (torch.cos(a) * mscale).float()[:, None], (torch.sin(a) * mscale).float()[:, None]
    if inverse:
        s = -s
    n = inv.numel()
    if layout == "half":
        u, v = x[..., :n], x[..., n:2 * n]
        y = torch.cat([u * c - v * s, v * c + u * s], -1)
    else:
        u, v = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack([u * c - v * s, v * c + u * s], -1).flatten(-2)
    return torch.cat([y, x[..., 2 * n:]], -1)


def _quantise(x, fmt):
    """x [..., 128] float32 -> (code values float32, e4m3 group scales or None, token scales)."""
    amax = x.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(amax)
    dead = (amax < TINY) | bad
    top = {"f8": 448.0, "i8": 127.0, "i4": 7.0 * 448.0}[fmt]
    scale = amax * torch.tensor(1.0 / top, dtype=torch.float32, device=x.device)
    y = torch.where(dead, 0.0, x * torch.reciprocal(scale))
    groups = None
    if fmt == "f8":
        code = y.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    elif fmt == "i8":
        code = torch.round(y).clamp(-127, 127)
    else:
        y = y.unflatten(-1, (4, 32))
        seventh = torch.tensor(1.0 / 7.0, dtype=torch.float32, device=x.device)
        groups = (y.abs().amax(-1) * seventh).clamp(max=448).to(torch.float8_e4m3fn).float()
        g = groups.unsqueeze(-1)
        code = torch.where(g > 0, torch.round(y * torch.reciprocal(g)).clamp(-7, 7), 0.0).flatten(-2)
    scale = torch.where(bad, float("nan"), torch.where(dead, 0.0, scale)).squeeze(-1)
    return code, groups, scale


def _value(code, groups, scale):
    """The float32 values that codes and scales stand for."""
    if groups is not None:
        code = (code.unflatten(-1, (4, 32)) * groups.unsqueeze(-1)).flatten(-2)
    return code * scale.unsqueeze(-1)


def _chunks(page, fmt, device):
    """Place of 16-byte chunk c of row r, flat, in the order (r, c)."""
    r = torch.arange(page, device=device)[:, None]
    n = ROW[fmt] // 16
    c = torch.arange(n, device=device)[None]
    x = (r & 7) if n == 8 else ((r >> 1) & 3)
    return (r * n + (c ^ x)).flatten()


def _pack(code, groups, scale, page, fmt):
    """Records [..., record bytes] of pages [..., page, 128]."""
    if fmt == "f8":
        rows = code.to(torch.float8_e4m3fn).view(torch.uint8)
    elif fmt == "i8":
        rows = (code + 128).to(torch.uint8)
    else:
        n = (code + 8).to(torch.uint8)
        rows = n[..., 0::2] | (n[..., 1::2] << 4)
    lead = code.shape[:-2]
    out = torch.empty_like(rows).reshape(*lead, -1, 16)
    out[..., _chunks(page, fmt, code.device), :] = rows.reshape(*lead, -1, 16)
    parts = [out.reshape(*lead, -1)]
    if groups is not None:
        parts.append(groups.to(torch.float8_e4m3fn).view(torch.uint8).reshape(*lead, -1))
    parts.append(scale.contiguous().view(torch.uint8).reshape(*lead, -1))
    return torch.cat(parts, -1)


def _unpack(rec, page, fmt):
    """Values [..., page, 128] in float32 of records."""
    lead, n = rec.shape[:-1], page * ROW[fmt]
    rows = rec[..., :n].reshape(*lead, -1, 16)[..., _chunks(page, fmt, rec.device), :].reshape(*lead, page, -1)
    groups = None
    if fmt == "f8":
        code = rows.contiguous().view(torch.float8_e4m3fn).float()
    elif fmt == "i8":
        code = rows.float() - 128
    else:
        code = torch.stack([rows & 15, rows >> 4], -1).flatten(-2).float() - 8
        groups = rec[..., n:n + 4 * page].contiguous().view(torch.float8_e4m3fn).float().reshape(*lead, page, 4)
    scale = rec[..., -4 * page:].contiguous().view(torch.float32)
    return _value(code, groups, scale)


def _plain_attend(s, q, k_pool, v_pool):
    c = s["case"]
    page, hkv = c["page"], c["hkv"]
    g = c["hq"] // hkv
    table, lens = s["block_table"].long(), s["seq_lens"].long()
    ids = s["selected"].long() if c["k"] else torch.arange(table.shape[1], device=q.device).expand(c["batch"], hkv, -1)
    blk = torch.gather(table[:, None].expand(-1, hkv, -1), 2, ids.clamp(min=0)).clamp(min=0)
    h = torch.arange(hkv, device=q.device)[None, :, None]
    t = (ids[..., None] * page + torch.arange(page, device=q.device)).flatten(2)
    n = lens[:, None, None]
    ok = (ids >= 0).repeat_interleave(page, 2) & (t < n)
    if c["window"]:
        ok &= t >= n - c["window"]
    k = _unpack(k_pool[blk, h], page, c["fmt"]).flatten(2, 3)
    logit = torch.matmul(q.float().unflatten(1, (hkv, g)), k.transpose(-1, -2)) * (1 / math.sqrt(D))
    del k
    logit = torch.where(ok[:, :, None], logit, -math.inf)
    m = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - torch.where(torch.isinf(m), 0.0, m))
    total = p.sum(-1, keepdim=True)
    v = torch.where(ok[..., None], _unpack(v_pool[blk, h], page, c["fmt"]).flatten(2, 3), 0.0)
    out = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = (torch.log(total) + m).squeeze(-1)
    return out.flatten(1, 2).to(torch.bfloat16), torch.where(torch.isnan(lse), -math.inf, lse).flatten(1, 2)


def _plain_write(s):
    """(rotated queries bf16, code values, groups and scales of k and of v), [tokens][heads][...]."""
    q, k = s["q"].float(), s["k"].float()
    if s["inv"] is not None:
        args = (s["pos"], s["inv"], s["mscale"], s["case"]["layout"])
        q, k = _rotate(q, *args), _rotate(k, *args)
    return q.to(torch.bfloat16), _quantise(k, s["case"]["fmt"]), _quantise(s["v"].float(), s["case"]["fmt"])


def _place(s, pool, what):
    """`pool` [blocks][heads][page]... with the rows of the written tokens put in."""
    page = s["case"]["page"]
    pos = s["pos"].long()
    blk = s["block_table"].long()[s["seq"].long(), pos // page]
    pool[blk, :, pos % page] = what
    return pool


# --------------------------------------------------------------------------
# state
# --------------------------------------------------------------------------
def _table(batch, pages, extra, gen):
    """A block table over a shuffled pool."""
    perm = torch.randperm(batch * pages + extra, generator=gen, device="cuda").int()
    return perm[:batch * pages].reshape(batch, pages).contiguous(), batch * pages + extra


def _pool(blocks, hkv, page, fmt, gen, keys):
    """A pool of quantised pages.  Keys have a few strong channels and a common part, as keys
    after a rotation do; values are nearly normal with a spread of sizes over the tokens."""
    rec = page * (ROW[fmt] + (8 if fmt == "i4" else 4))
    pool = torch.empty(blocks, hkv, rec, dtype=torch.uint8, device="cuda")
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
        pool[a:a + n] = _pack(*_quantise(x.bfloat16().float(), fmt), page, fmt)
    return pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    s = {"case": case}

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    if case["op"] == "rope":
        dtype = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[case["dtype"]]
        s["x"] = randn(case["tokens"], case["total_heads"], case["head_dim"], dtype=dtype)[:, :case["heads"]]
        s["pos"] = torch.randint(0, case["max_pos"], (case["tokens"],), generator=gen, device="cuda").int()
        inv, s["mscale"] = _inv_freq(case["rotary"], **ROPE[case["scaling"]])
        s["inv"] = inv.cuda()
    else:
        lens = _lens(case)
        batch, hq, hkv, page, fmt = (case[k] for k in ("batch", "hq", "hkv", "page", "fmt"))
        start = case.get("start", 0)
        pages = max(1, -(-(start + max(lens) + (case["op"] == "step")) // page))
        s["block_table"], blocks = _table(batch, pages, 3, gen)
        tokens = 0
        if case["op"] == "write":
            tokens = sum(lens)
            s["seq"] = torch.repeat_interleave(torch.arange(batch), torch.tensor(lens)).int().cuda()
            s["pos"] = torch.cat([start + torch.arange(n) for n in lens]).int().cuda()
            used = [s["block_table"][b, start // page:-(-(start + n) // page)] for b, n in enumerate(lens) if n]
            s["blocks"] = torch.cat(used).contiguous()
            rec = page * (ROW[fmt] + (8 if fmt == "i4" else 4))
            s["k_pool"], s["v_pool"] = (torch.zeros(blocks, hkv, rec, dtype=torch.uint8, device="cuda") for _ in "kv")
        else:
            s["k_pool"], s["v_pool"] = (_pool(blocks, hkv, page, fmt, gen, keys) for keys in (True, False))
            s["seq_lens"] = torch.tensor([n + (case["op"] == "step") for n in lens], dtype=torch.int32).cuda()
            s["q"] = randn(batch, hq, D)
        if case["op"] == "step":
            tokens = batch
            s["seq"] = torch.arange(batch).int().cuda()
            s["pos"] = torch.tensor(lens, dtype=torch.int32).cuda()
        if tokens:
            qkv = randn(tokens, hq + 2 * hkv, D)     # the fused projection's output
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
            s["inv"], s["mscale"] = None, 1.0
            if case["rotary"]:
                inv, s["mscale"] = _inv_freq(case["rotary"], **ROPE[case["scaling"]])
                s["inv"] = inv.cuda()
        if case.get("k"):
            u = torch.rand(batch, hkv, pages, generator=gen, device="cuda")
            n = -(-s["seq_lens"].long() // page)[:, None, None]
            j = torch.arange(pages, device="cuda")
            u = torch.where((j == 0) | (j == n - 1), 2.0, u)        # the first and the last page are always kept
            u = torch.where(j < n, u, -1.0)
            top, at = u.topk(min(case["k"], pages), -1)
            at = torch.where(top >= 0, at, pages).sort(-1).values
            sel = torch.full((batch, hkv, case["k"]), -1, dtype=torch.int32, device="cuda")
            sel[..., :at.shape[-1]] = torch.where(at < pages, at, -1)
            s["selected"] = sel
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a user of the library keeps: configurations, rotary tables, output buffers, a workspace."""
    from sparse_paged_kv_gb300 import binding as B, runtime
    case = s["case"]
    s["rope"] = None
    if case.get("rotary"):
        s["rope"] = runtime.RopeTable(case["rotary"], layout=case["layout"], **ROPE[case["scaling"]])
    if case["op"] == "rope":
        s["out"] = torch.empty(case["tokens"], case["heads"], case["head_dim"], dtype=s["x"].dtype, device="cuda")
        return
    s["cfg"] = cfg = B.LocksKvConfig(batch=case["batch"], n_q_heads=case["hq"], n_kv_heads=case["hkv"], head_dim=D,
                                     page_size=case["page"], max_pages=s["block_table"].shape[1],
                                     num_blocks=s["k_pool"].shape[0], kv_dtype=FMT[case["fmt"]])
    s["q_out"] = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    if case["op"] == "write":
        shape = (s["blocks"].numel(), case["hkv"], case["page"], D)
        s["k_out"], s["v_out"] = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    else:
        s["out"] = torch.empty(case["batch"], case["hq"], D, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(case["batch"], case["hq"], dtype=torch.float32, device="cuda")
        s["ws"] = torch.zeros(B.kv_decode_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from sparse_paged_kv_gb300 import binding as B
    case = s["case"]
    op = case["op"]
    if op == "rope":
        B.locks_rope(s["rope"], s["x"], s["pos"], s["out"], inverse=case["inverse"])
        return s["out"]
    cfg = s["cfg"]
    if op == "write":
        B.locks_kv_write(cfg, s["k"], s["v"], s["pos"], s["k_pool"], s["v_pool"], s["block_table"],
                         token_seq=s["seq"], rope=s["rope"], q=s["q"], q_out=s["q_out"])
        B.locks_kv_read(cfg, s["k_pool"], s["v_pool"], s["blocks"], s["k_out"], s["v_out"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    q = s["q"]
    if op == "step":
        B.locks_kv_write(cfg, s["k"], s["v"], s["pos"], s["k_pool"], s["v_pool"], s["block_table"],
                         rope=s["rope"], q=s["q"], q_out=s["q_out"])
        q = s["q_out"]
    B.locks_kv_decode(cfg, q, s["k_pool"], s["v_pool"], s["block_table"], s["seq_lens"], s["out"], s["ws"],
                      selected=s.get("selected"), window=case["window"], out_lse=s["lse"])
    return {"q": q, "out": s["out"]} if op == "step" else {"out": s["out"], "lse": s["lse"]}


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "rope":
        return _rotate(s["x"].float(), s["pos"], s["inv"], s["mscale"], case["layout"], case["inverse"]).to(s["x"].dtype)
    if op == "attend":
        out, lse = _plain_attend(s, s["q"], s["k_pool"], s["v_pool"])
        return {"out": out, "lse": lse}
    q, k, v = _plain_write(s)
    if op == "write":
        shape = (s["k_pool"].shape[0], case["hkv"], case["page"], D)
        k, v = (_place(s, torch.zeros(shape, device="cuda"), _value(*x))[s["blocks"].long()].to(torch.bfloat16) for x in (k, v))
        return {"q": q, "k": k, "v": v}
    # the token's record rows are written as one-token pages, then copied to their slots
    k, v = (_plain_rows(s, pool, x) for pool, x in ((s["k_pool"], k), (s["v_pool"], v)))
    out, _ = _plain_attend(s, q, k, v)
    return {"q": q, "out": out}


def _plain_rows(s, pool, x):
    """`pool`, updated in place, with the quantised rows x of the step's tokens."""
    code, groups, scale = x
    c = s["case"]
    page, fmt = c["page"], c["fmt"]
    pos = s["pos"].long()
    blk, slot = s["block_table"].long()[s["seq"].long(), pos // page], pos % page
    rec = pool[blk]                                              # [tokens][heads][record]
    at = (slot[:, None] == torch.arange(page, device=pos.device))[:, None]
    one = lambda a, rep: a.unsqueeze(2).expand(*a.shape[:2], page, *a.shape[2:])  # noqa: E731
    new = _pack(one(code, page), None if groups is None else one(groups, page), one(scale, page).contiguous(), page, fmt)
    row = torch.arange(page, device=pos.device)
    parts = [row.repeat_interleave(ROW[fmt])] + ([row.repeat_interleave(4)] if fmt == "i4" else []) + [row.repeat_interleave(4)]
    mine = torch.gather(at.expand(-1, rec.shape[1], -1), 2, torch.cat(parts).expand(*rec.shape))
    pool[blk] = torch.where(mine, new, rec)
    return pool


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    if case["op"] == "rope":
        size = 4 if case["dtype"] == "f32" else 2
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["head_dim"] * size + 4 * case["tokens"] + 4 * case["rotary"],
                "flops": 3 * n * case["rotary"]}
    lens, hq, hkv = _lens(case), case["hq"], case["hkv"]
    row = ROW[case["fmt"]] + (8 if case["fmt"] == "i4" else 4)
    if case["op"] == "write":
        n, page, start = sum(lens), case["page"], case["start"]
        blocks = sum(-(-(start + x) // page) - start // page for x in lens if x)
        there = n * (hq * D * 4 + 2 * hkv * (2 * D + row) + 8)
        back = blocks * page * 2 * hkv * 2 * D + n * 2 * hkv * row
        return {"bytes": there + back, "flops": n * ((hq + hkv) * 3 * case["rotary"] + 8 * hkv * D)}
    extra, bytes_ = (1 if case["op"] == "step" else 0), 0
    lens = [x + extra for x in lens]
    if case["window"]:
        seen = [min(x, case["window"]) for x in lens]
    else:
        seen = lens
    if case["k"]:
        page = case["page"]
        seen = [min(x, case["k"] * page) for x in seen]
    n = sum(seen)
    bytes_ += 2 * n * hkv * row + len(lens) * hq * (4 * D + 4) + 4 * len(lens)
    bytes_ += 4 * sum(-(-x // case["page"]) for x in seen) * (hkv if case["k"] else 1)
    if extra:
        bytes_ += len(lens) * (hq * D * 4 + 2 * hkv * (2 * D + row))
    return {"bytes": bytes_, "flops": 4 * n * hq * D}


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def _exact_freq(rotary, spec):
    kind, theta, f = spec["scaling"], spec["theta"], spec.get("factor", 1.0)
    got = []
    for i in range(rotary // 2):
        w = theta ** (-2.0 * i / rotary)
        if kind == "linear":
            w /= f
        elif kind == "ntk":
            w = (theta * f ** (rotary / (rotary - 2.0))) ** (-2.0 * i / rotary)
        elif kind == "llama3":
            wave, orig = 2 * math.pi / w, spec["original_positions"]
            lo, hi = spec["low_freq_factor"], spec["high_freq_factor"]
            if wave > orig / lo:
                w /= f
            elif wave >= orig / hi:
                z = (orig / wave - lo) / (hi - lo)
                w = (1 - z) * w / f + z * w
        elif kind == "yarn":
            def place(beta):
                return rotary * math.log(spec["original_positions"] / (beta * 2 * math.pi)) / (2 * math.log(theta))
            a, b = max(0, math.floor(place(spec["beta_fast"]))), min(rotary - 1, math.ceil(place(spec["beta_slow"])))
            z = min(1.0, max(0.0, (i - a) / max(b - a, 1e-3)))
            w = w * (1 - z) + w / f * z
        got.append(w)
    return got, (0.1 * math.log(f) + 1.0 if kind == "yarn" else 1.0)


def _exact_rotate(x, pos, rotary, spec, layout, inverse=False):
    x = x.double().clone()
    freq, m = _exact_freq(rotary, spec)
    n = rotary // 2
    src = x.clone()
    for i, w in enumerate(freq):
        a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
        ang = pos.double() * w * (-1.0 if inverse else 1.0)
        c, s = (torch.cos(ang) * m)[:, None], (torch.sin(ang) * m)[:, None]
        x[..., a] = src[..., a] * c - src[..., b] * s
        x[..., b] = src[..., b] * c + src[..., a] * s
    return x


def _e4m3(x):
    """The e4m3 value nearest to x (float64), ties to even, at most 448."""
    _, e = torch.frexp(x.abs())
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _f32(x):
    """x (float64) rounded to a float, where the format's definition has one: the scales it stores, and the
    quotients that it rounds to codes.  bf16 rows meet ties of those exactly, so they are part of it."""
    return x.float().double()


def _exact_values(x, fmt):
    """What x [..., 128] in 64 bits reads back as."""
    x = _f32(x)
    top = {"f8": 448, "i8": 127, "i4": 7 * 448}[fmt]
    s = _f32(x.abs().amax(-1, keepdim=True) * float(torch.tensor(1.0 / top)))
    y = _f32(x * _f32(1 / torch.where(s > 0, s, 1.0)))
    if fmt != "i4":
        return (_e4m3(y) if fmt == "f8" else torch.round(y)) * s
    got = torch.zeros_like(x)
    for a in range(0, D, 32):
        part = y[..., a:a + 32]
        g = _e4m3(_f32(part.abs().amax(-1, keepdim=True) * float(torch.tensor(1.0 / 7.0))))
        code = torch.round(_f32(part * _f32(1 / torch.where(g > 0, g, 1.0)))).clamp(-7, 7)
        got[..., a:a + 32] = code * g * s
    return got


def _exact_rows(rec, page, fmt):
    """Values [pages][page][128] in 64 bits of the records of one head."""
    r = torch.arange(page, device=rec.device)[:, None]
    d = torch.arange(D, device=rec.device)[None]
    if fmt == "i4":
        byte = rec[:, r * 64 + 16 * ((d // 32) ^ ((r // 2) % 4)) + (d % 32) // 2].int()
        code = ((byte >> (4 * (d % 2))) & 15).double() - 8
        e = rec[:, page * 64 + 4 * r + d // 32].int()
        code *= _exact_e4m3_bits(e)
        at = page * 68
    else:
        byte = rec[:, r * 128 + 16 * ((d // 16) ^ (r % 8)) + d % 16].int()
        code = _exact_e4m3_bits(byte) if fmt == "f8" else byte.double() - 128
        at = page * 128
    bits = rec[:, at:at + 4 * page].reshape(-1, page, 4).long()
    bits = bits[..., 0] + (bits[..., 1] << 8) + (bits[..., 2] << 16) + (bits[..., 3] << 24)
    e = (bits >> 23) & 255
    scale = torch.where(e > 0, ((bits & 0x7FFFFF) + 0x800000).double() * torch.exp2(e.double() - 150), 0.0)
    return code * scale[..., None]


def _exact_e4m3_bits(b):
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9)
    return torch.where(b >= 128, -mag, mag)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "rope":
        return _exact_rotate(s["x"], s["pos"], case["rotary"], ROPE[case["scaling"]], case["layout"], case["inverse"])
    page, hkv, fmt = case["page"], case["hkv"], case["fmt"]
    if op in ("write", "step"):
        q, k = s["q"].double(), s["k"].double()
        if case["rotary"]:
            args = (s["pos"], case["rotary"], ROPE[case["scaling"]], case["layout"])
            q, k = _exact_rotate(q, *args), _exact_rotate(k, *args)
        k, v = _exact_values(k, fmt), _exact_values(s["v"].double(), fmt)
    if op == "write":
        got = []
        where = {int(b): i for i, b in enumerate(s["blocks"].tolist())}
        table, seq, pos = s["block_table"].tolist(), s["seq"].tolist(), s["pos"].tolist()
        at = torch.tensor([where[table[b][p // page]] * page + p % page for b, p in zip(seq, pos)], device="cuda")
        for x in (k, v):
            flat = torch.zeros(len(where) * page, hkv, D, dtype=torch.float64, device="cuda")
            flat[at] = x
            got.append(flat.reshape(len(where), page, hkv, D).transpose(1, 2).contiguous())
        return {"q": q, "k": got[0], "v": got[1]}
    if op == "attend":
        q = s["q"].double()
    g = case["hq"] // hkv
    out = torch.zeros(case["batch"], case["hq"], D, dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], case["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    qa = q.to(torch.bfloat16).double() if op == "step" else q      # the query is handed on in bf16
    for b, n in enumerate(s["seq_lens"].tolist()):
        for h in range(hkv):
            ids = s["selected"][b, h].tolist() if case["k"] else list(range(-(-n // page)))
            ids = [j for j in ids if j >= 0]
            if not ids:
                continue
            blk = s["block_table"][b].long()[torch.tensor(ids, device="cuda")]
            t = (torch.tensor(ids, device="cuda")[:, None] * page + torch.arange(page, device="cuda")).flatten()
            first = max(0, n - case["window"]) if case["window"] else 0
            seen = ((t >= first) & (t < n)).nonzero().flatten()
            if not seen.numel():
                continue
            kk, vv = (_exact_rows(pool[blk, h], page, fmt).reshape(-1, D)[seen] for pool in (s["k_pool"], s["v_pool"]))
            if op == "step":
                kk[t[seen] == n - 1], vv[t[seen] == n - 1] = k[b, h], v[b, h]
            a = slice(h * g, h * g + g)
            z = qa[b, a] @ kk.T / math.sqrt(D)
            lse[b, a] = torch.logsumexp(z, -1)
            out[b, a] = torch.exp(z - lse[b, a][:, None]) @ vv
    return {"q": q, "out": out} if op == "step" else {"out": out, "lse": lse}
