"""One attention layer that serves a batch behind a shared prompt: the prompt's
pages are cached once and read once a step for all sequences; each sequence's own
tokens are kept within a budget, the least attended evicted first.

    python examples/shared_prefix.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from sparse_paged_kv_gb300 import binding as B  # noqa: E402
from sparse_paged_kv_gb300 import build_lib, runtime  # noqa: E402


def main(batch: int = 4, prefix_tokens: int = 1024, prompt: int = 200, steps: int = 70, budget: int = 128):
    build_lib.build()
    torch.manual_seed(0)
    page, hq, hkv, d = 64, 32, 8, 128
    shared = prefix_tokens // page
    own = -(-(prompt + steps) // page)                 # pages of a sequence's own
    blocks = np.random.default_rng(0).permutation(shared + batch * own)
    table = np.concatenate([np.tile(blocks[:shared], (batch, 1)), blocks[shared:].reshape(batch, own)], 1)
    cfg = B.LocksConfig(batch=batch, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=page, rank=8,
                        max_pages=shared + own, num_blocks=blocks.size)
    cache = runtime.BatchCache(cfg, table, group_starts=[0, batch], prefix_pages=[shared], budget_tokens=budget,
                               recent_tokens=32, max_rows=16)
    rope = runtime.RopeTable(d, theta=500000.0, scaling="llama3", factor=8.0)

    def rows(n, heads):
        return torch.randn(n, heads, d, device="cuda").bfloat16()

    def rotated(x, positions):
        B.locks_rope(rope, x, positions, x)
        return x

    # the shared prompt once, then each sequence's own: rotated keys and values, a page at a time
    def fill(row, first, n):
        at = torch.arange(first, first + n, dtype=torch.int32, device="cuda")
        k, v = rotated(rows(n, hkv), at), rows(n, hkv)
        blk = cache.block_table[row].long()[at.long() // page]
        cache.k_cache[blk, :, at.long() % page], cache.v_cache[blk, :, at.long() % page] = k, v

    fill(0, 0, prefix_tokens)
    for b in range(batch):
        fill(b, prefix_tokens, prompt)
    cache.seq_lens.fill_(prefix_tokens + prompt)

    # the prompts' last 16 tokens attend, vote on every own token, and the least are evicted
    last = torch.arange(prefix_tokens + prompt - 16, prefix_tokens + prompt, dtype=torch.int32, device="cuda")
    q = rotated(rows(batch * 16, hq), last.repeat(batch)).view(batch, 16, hq, d)
    cache.observe(q)
    print("after the prompts:", cache.seq_lens.tolist(), "tokens, next positions", cache.next_positions().tolist())

    q1, k1, v1 = rows(batch, hq), rows(batch, hkv), rows(batch, hkv)
    graph = cache.capture_step(q1, k1, v1)
    for _ in range(steps):
        for x, heads in ((q1, hq), (k1, hkv)):
            x.copy_(rotated(rows(batch, heads), cache.next_positions()))
        v1.copy_(rows(batch, hkv))
        graph.replay()
    torch.cuda.synchronize()
    print(f"after {steps} steps:", cache.seq_lens.tolist(), "tokens, next positions", cache.next_positions().tolist())
    assert int(cache.status) == 0 and torch.isfinite(cache.out.float()).all()
    return cache


if __name__ == "__main__":
    main()
