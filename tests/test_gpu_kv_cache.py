"""The quantised cache as a serving program uses it (runtime.QuantCache): a
ragged prompt, summaries of its pages, decode steps that complete pages, the
captured step and the example, against the NumPy reference on the records
that the pools hold."""
import importlib.util
import os

import numpy as np
import pytest

from tests import kv_ref as R
from tests.test_gpu_kv import attend_tol, rope_tol, BF16_HALF

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    from sparse_paged_kv_gb300 import binding, build_lib
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    binding.load_library(build_lib.build())


def make(fmt, page, batch, hq, hkv, pages, budget=0, rot=128, **rope):
    from sparse_paged_kv_gb300 import binding as B
    from sparse_paged_kv_gb300 import runtime
    cfg = B.LocksKvConfig(batch=batch, n_q_heads=hq, n_kv_heads=hkv, head_dim=128, page_size=page,
                          max_pages=pages, num_blocks=batch * pages + 1, kv_dtype=fmt)
    table = np.random.default_rng(page + fmt).permutation(cfg.num_blocks)[:batch * pages].reshape(batch, pages)
    return runtime.QuantCache(cfg, table, rope=runtime.RopeTable(rot, **rope), budget_tokens=budget)


def rows(n, heads, seed):
    import torch
    return torch.randn(n, heads, 128, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def check_attention(cache, selected=None, window=0):
    """self.out against the reference over what the pools hold."""
    c = cache.cfg
    G = c.n_q_heads // c.n_kv_heads
    kp, vp = cache.k_pool.cpu().numpy(), cache.v_pool.cpu().numpy()
    table, lens = cache.block_table.cpu().numpy(), cache.seq_lens.tolist()
    q, out = cache.q.double().cpu().numpy(), cache.out.double().cpu().numpy()
    lse = cache.out_lse.double().cpu().numpy()
    for b, n in enumerate(lens):
        for h in range(c.n_kv_heads):
            ids = np.arange(-(-n // c.page_size)) if selected is None else selected[b, h][selected[b, h] >= 0]
            t = (ids[:, None] * c.page_size + np.arange(c.page_size)).ravel()
            ok = (t < n) & (t >= n - window if window else True)
            blk = table[b, ids]
            k, v = (R.values(*R.unpack(p[blk, h], c.kv_dtype, c.page_size), c.kv_dtype).reshape(-1, 128)[ok]
                    for p in (kp, vp))
            a = slice(h * G, h * G + G)
            o, l, bounds = R.attend(q[b, a], k, v)
            to, tl = attend_tol(o, l, bounds, int(ok.sum()))
            assert (np.abs(out[b, a] - o) <= to).all() and (np.abs(lse[b, a] - l) <= tl).all(), (b, h)


@pytest.mark.parametrize("name,fmt", sorted(R.FORMATS.items()))
def test_prompt_then_steps(name, fmt):
    """Chunked ragged prompts, then steps that cross page borders; keys as the reference
    rotates and quantises them, queries, lengths, completions, attention."""
    import torch
    page, hq, hkv, prompts, steps = 32, 6, 2, (70, 31, 1), 3
    kw = dict(theta=500000.0, scaling="llama3", factor=8.0)
    cache = make(fmt, page, 3, hq, hkv, 4, **kw)
    n = sum(prompts)
    qkv = rows(n, hq + 2 * hkv, 1)
    seq = torch.cat([torch.full((m,), b) for b, m in enumerate(prompts)]).int().cuda()
    pos = torch.cat([torch.arange(m) for m in prompts]).int().cuda()
    q_out = torch.empty(n, hq, 128, dtype=torch.bfloat16, device="cuda")
    for part in (slice(0, 50), slice(50, n)):                       # two chunks
        cache.write(qkv[part, :hq], qkv[part, hq:hq + hkv], qkv[part, hq + hkv:], seq[part].contiguous(),
                    pos[part].contiguous(), q_out=q_out[part])
    assert cache.seq_lens.tolist() == list(prompts)
    w, m = R.frequencies(128, **kw)
    want, tol = rope_tol(qkv.double().cpu().numpy(), pos.cpu().numpy(), w, m, "half", BF16_HALF)
    assert (np.abs(q_out.double().cpu().numpy() - want[:, :hq]) <= tol[:, :hq]).all()
    lens = list(prompts)
    for s in range(steps):
        x = rows(3, hq + 2 * hkv, 100 + s)
        cache.step(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:])
        want, tol = rope_tol(x.double().cpu().numpy(), np.array(lens), w, m, "half", BF16_HALF)
        assert (np.abs(cache.q.double().cpu().numpy() - want[:, :hq]) <= tol[:, :hq]).all()
        table = cache.block_table.cpu().numpy()
        done = [int(table[b, t // page]) if (t + 1) % page == 0 else -1 for b, t in enumerate(lens)]
        assert cache.completed.tolist() == done
        lens = [t + 1 for t in lens]
        assert cache.seq_lens.tolist() == lens
        check_attention(cache)
        cache.attend(window=20)
        check_attention(cache, window=20)
    assert cache.status.item() == 0
    # the values written, read back: the definition's, bit for bit
    for b, t in enumerate(prompts):
        ids = cache.block_table[b, :-(-t // page)].contiguous()
        _, v = cache.read(ids)
        src = qkv[(seq == b).nonzero().flatten(), hq + hkv:].float().cpu().numpy()
        code, groups, scale = R.quantise(src, fmt)
        exp = (R.values(code, groups, np.ones_like(scale), fmt).astype(np.float32) * scale[..., None])
        got = v.transpose(1, 2).reshape(-1, hkv, 128)[:t].cpu()
        assert torch.equal(got, torch.from_numpy(exp.astype(np.float32)).bfloat16())


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("name,fmt", sorted(R.FORMATS.items()))
def test_selected_steps(name, fmt, page):
    """With a budget: the selection is the one that a LocksLayer makes over the pages read
    back, also right after a page completes; attention is over it."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    hq, hkv, prompt, pages = 8, 2, 20 * page - 2, 22
    cache = make(fmt, page, 1, hq, hkv, pages, budget=6 * page)
    qkv = rows(prompt, hq + 2 * hkv, 7)
    pos = torch.arange(prompt).int().cuda()
    cache.write(None, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], torch.zeros_like(pos), pos)
    cache.build(cache.block_table[0, :prompt // page].contiguous(), pages_at_once=7)
    for s in range(5):
        x = rows(1, hq + 2 * hkv, 200 + s)
        cache.step(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:])
        n = int(cache.seq_lens.item())
        ids = cache.block_table[0, :n // page].contiguous()
        keys = torch.zeros(cache.cfg.num_blocks, hkv, page, 128, dtype=torch.bfloat16, device="cuda")
        keys[ids.long()] = cache.read(ids, values=False)
        fresh = torch.zeros_like(cache.summaries[:-1])
        B.locks_build_summaries(cache.locks_cfg, keys, ids, fresh)
        ws = torch.zeros_like(cache.ws_select)
        sel = torch.full_like(cache.selected, -7)
        B.locks_select(cache.locks_cfg, cache.q, fresh, cache.block_table, cache.seq_lens, cache.budget, sel, ws)
        assert torch.equal(sel, cache.selected)
        assert n > prompt + 2 or sel.max().item() == -(-n // page) - 1
        check_attention(cache, selected=cache.selected.cpu().numpy())
        cache.build_completed()
    assert cache.status.item() == 0


def test_captured_step_follows_the_lengths():
    """Replays advance the lengths and give the bits of steps run one by one."""
    import torch
    page, hq, hkv = 16, 8, 2
    a, b = (make(R.I8, page, 2, hq, hkv, 6) for _ in range(2))
    x = rows(2, hq + 2 * hkv, 0)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    graph = a.capture_step(q, k, v)
    for s in range(2 * page + 1):
        x.copy_(rows(2, hq + 2 * hkv, 300 + s))
        graph.replay()
        b.step(q, k, v)
        assert a.seq_lens.tolist() == b.seq_lens.tolist() == [s + 1, s + 1]
        assert torch.equal(a.out, b.out) and torch.equal(a.out_lse, b.out_lse) and torch.equal(a.q, b.q)
        assert torch.equal(a.completed, b.completed)
    check_attention(a)
    assert torch.equal(a.k_pool, b.k_pool) and torch.equal(a.v_pool, b.v_pool)


def test_steps_on_another_stream():
    import torch
    page, hq, hkv = 64, 8, 2
    a, b = (make(R.F8, page, 2, hq, hkv, 4, budget=2 * page) for _ in range(2))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in range(3):
        x = rows(2, hq + 2 * hkv, 400 + s)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        a.step(q, k, v)
        a.build_completed()
        side.wait_stream(torch.cuda.current_stream())
        b.step(q, k, v, stream=side)
        b.build_completed(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert torch.equal(a.out, b.out) and torch.equal(a.k_pool, b.k_pool)


@pytest.mark.parametrize("fmt", ["f8", "i4"])
def test_example(fmt):
    spec = importlib.util.spec_from_file_location("quantised_cache", os.path.join(ROOT, "examples", "quantised_cache.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    cache, outs = m.main(fmt, steps=3, prompts=(700, 127), hq=8, hkv=2)
    assert cache.seq_lens.tolist() == [703, 130]
    check_attention(cache, selected=cache.selected.cpu().numpy())
