"""Serving one attention layer from a quantised paged cache, from prompt to decode.

Two ragged prompts are rotated and written into 4-bit (or 8-bit) pages, their
complete pages are summarised, and a few decode steps each write a token,
select pages under the token budget and attend them in codes.  Random rows
stand in for a model's projections.

    python examples/quantised_cache.py [f8|i8|i4] [steps]
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

FORMATS = {"f8": 0, "i8": 1, "i4": 2}


def main(fmt="i4", steps=4, prompts=(3000, 1234), hq=32, hkv=8, page=64, budget=1024):
    import numpy as np
    import torch

    from sparse_paged_kv_gb300 import binding as B
    from sparse_paged_kv_gb300 import runtime

    gen = torch.Generator(device="cuda").manual_seed(0)
    d, batch = 128, len(prompts)
    max_pages = -(-(max(prompts) + steps) // page)
    cfg = B.LocksKvConfig(batch=batch, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=page,
                          max_pages=max_pages, num_blocks=batch * max_pages, kv_dtype=FORMATS[fmt])
    table = np.random.default_rng(0).permutation(cfg.num_blocks).reshape(batch, max_pages)
    rope = runtime.RopeTable(d, theta=500000.0, scaling="llama3", factor=8.0)
    cache = runtime.QuantCache(cfg, table, rope=rope, budget_tokens=budget)

    def project(n):                       # the fused projection's output: queries, keys, values
        qkv = torch.randn(n, hq + 2 * hkv, d, generator=gen, device="cuda").bfloat16()
        return qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]

    # the prompts, in one ragged call
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(prompts)]).int().cuda()
    pos = torch.cat([torch.arange(n) for n in prompts]).int().cuda()
    q, k, v = project(sum(prompts))
    q_rotated = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")   # for the prompt's own attention
    cache.write(q, k, v, seq, pos, q_out=q_rotated)
    cache.build(torch.cat([cache.block_table[b, :n // page] for b, n in enumerate(prompts)]))

    outs = []
    for _ in range(steps):
        cache.step(*project(batch))
        cache.build_completed()           # pages this token completed, for the next step
        outs.append(cache.out.clone())
    torch.cuda.synchronize()
    if cache.status.item():
        raise RuntimeError(f"device status {cache.status.item():#x}")
    bf16 = 2 * 2 * cfg.num_blocks * hkv * page * d
    print(f"{fmt}: lengths {cache.seq_lens.tolist()}, {cache.selected.shape[-1]} pages a step, "
          f"cache {2 * cache.k_pool.nbytes / 1e6:.1f} MB (bf16 {bf16 / 1e6:.1f} MB), "
          f"|out| {outs[-1].float().abs().mean().item():.4f}")
    return cache, outs


if __name__ == "__main__":
    main(*(sys.argv[1:2] or ["i4"]), *(int(x) for x in sys.argv[2:3]))
