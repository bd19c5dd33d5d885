"""Edges of the quantised cache's calls on the GPU: batches with nothing to attend,
block ids outside the pool, the captured step, raw stream handles."""
import numpy as np
import pytest

from tests import kv_ref as R
from tests.test_gpu_kv import Cache

pytestmark = pytest.mark.gpu

FMTS = sorted(R.FORMATS.items())


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    from sparse_paged_kv_gb300 import binding, build_lib
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    binding.load_library(build_lib.build())


def decode(c, lens, selected=None, window=0):
    """One call with these lengths, which lie in a longer array: (out, lse, status)."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    batch = c.cfg.batch
    n = torch.full((batch + 64,), 1, dtype=torch.int32, device="cuda")
    n[:batch] = torch.tensor(lens, dtype=torch.int32)
    out = torch.full((batch, c.hq, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((batch, c.hq), 9.0, device="cuda")
    ws = torch.zeros(B.kv_decode_workspace_bytes(c.cfg), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.from_numpy(c.q).bfloat16().cuda()
    table = torch.from_numpy(c.table).cuda()
    if selected is not None:
        selected = torch.from_numpy(selected).cuda()
    B.locks_kv_decode(c.cfg, q, c.dev[0], c.dev[1], table, n[:batch], out, ws, selected=selected,
                      window=window, out_lse=lse, status=status)
    return out, lse, status.item()


@pytest.mark.parametrize("how", ["dense", "listed", "window"])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (1, 1), (32, 2)])
@pytest.mark.parametrize("batch", [1, 3, 200])
@pytest.mark.parametrize("name,fmt", FMTS)
def test_a_batch_of_empty_sequences(name, fmt, batch, hq, hkv, how):
    """Every length 0: zeros and -inf in every row, whatever the form of the call."""
    c = Cache(fmt, 16, [0] * batch, hq, hkv, seed=batch)
    sel = np.zeros((batch, hkv, 5), np.int32) if how == "listed" else None
    out, lse, status = decode(c, [0] * batch, selected=sel, window=7 if how == "window" else 0)
    assert status == 0
    assert (out == 0).all() and (lse == float("-inf")).all()


@pytest.mark.parametrize("batch", [1, 40])
def test_a_batch_of_negative_lengths(batch):
    """They count as 0, with a flag."""
    from sparse_paged_kv_gb300 import binding as B
    c = Cache(R.F8, 64, [0] * batch, 8, 2, seed=1)
    out, lse, status = decode(c, [-3] * batch)
    assert status == B.LOCKS_DEV_BAD_SEQ_LEN
    assert (out == 0).all() and (lse == float("-inf")).all()


def test_attention_over_a_cache_that_holds_nothing_yet():
    """A new QuantCache attends nothing; after a token it attends that one."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    from sparse_paged_kv_gb300 import runtime
    cfg = B.LocksKvConfig(batch=2, n_q_heads=4, n_kv_heads=2, head_dim=128, page_size=16, max_pages=2,
                          num_blocks=4, kv_dtype=R.I8)
    cache = runtime.QuantCache(cfg, np.arange(4).reshape(2, 2))
    cache.attend()
    assert (cache.out == 0).all() and (cache.out_lse == float("-inf")).all()
    x = torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    cache.step(x[:, :4], x[:, 4:6], x[:, 6:])
    want = cache.read(cache.block_table[:, 0].contiguous())[1][:, :, 0].repeat_interleave(2, 1)
    # one token: its weight is 1 (2^-11 in f16, 2^-20 from the exponential) and the result rounds to
    # bf16, as the value read back does
    assert ((cache.out.float() - want.float()).abs() <= want.float().abs() * (2 * 2.0 ** -8 + 2.0 ** -10)).all()
    assert cache.status.item() == 0


@pytest.mark.parametrize("name,fmt", FMTS)
def test_build_skips_block_ids_outside_the_pool(name, fmt):
    """Flagged; the other summaries are those of a build without them, and no other changes."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    from sparse_paged_kv_gb300 import runtime
    page, hkv, blocks = 16, 2, 7
    cfg = B.LocksKvConfig(batch=1, n_q_heads=4, n_kv_heads=hkv, head_dim=128, page_size=page, max_pages=6,
                          num_blocks=blocks, kv_dtype=fmt)
    caches = [runtime.QuantCache(cfg, np.arange(6).reshape(1, 6), budget_tokens=4 * page) for _ in range(2)]
    x = torch.randn(6 * page, 2 * hkv, 128, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    pos = torch.arange(6 * page).int().cuda()
    for c, ids in zip(caches, ([3, 0, 5], [-1, 3, blocks, 0, blocks + 5, 2 ** 31 - 1, 5, -2 ** 31])):
        c.write(None, x[:, :hkv], x[:, hkv:], torch.zeros_like(pos), pos)
        c.summaries.fill_(99)
        c.build(torch.tensor(ids, dtype=torch.int32).cuda())
    a, b = caches
    assert a.status.item() == 0 and b.status.item() == B.LOCKS_DEV_BAD_BLOCK_ID
    assert torch.equal(a.summaries[:blocks], b.summaries[:blocks])
    assert (b.summaries[[1, 2, 4, 6]] == 99).all() and (b.summaries[0] != 99).any()


def _budgeted(lens, page=16, pages=8, hq=4, hkv=2, budget=3 * 16):
    """A cache with a budget, its prompts written and their complete pages summarised."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    from sparse_paged_kv_gb300 import runtime
    batch = len(lens)
    cfg = B.LocksKvConfig(batch=batch, n_q_heads=hq, n_kv_heads=hkv, head_dim=128, page_size=page,
                          max_pages=pages, num_blocks=batch * pages, kv_dtype=R.I8)
    cache = runtime.QuantCache(cfg, np.arange(batch * pages).reshape(batch, pages), rope=runtime.RopeTable(128),
                               budget_tokens=budget)
    n = sum(lens)
    x = torch.randn(n, 2 * hkv, 128, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    seq = torch.cat([torch.full((m,), b) for b, m in enumerate(lens)]).int().cuda()
    pos = torch.cat([torch.arange(m) for m in lens]).int().cuda()
    cache.write(None, x[:, :hkv], x[:, hkv:], seq, pos)
    cache.build(torch.cat([cache.block_table[b, :m // page] for b, m in enumerate(lens)]))
    return cache


def _token(batch, seed, hq=4, hkv=2):
    import torch
    return torch.randn(batch, hq + 2 * hkv, 128, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def test_capture_takes_back_what_its_first_step_wrote():
    """Lengths, completed pages, the query and the outputs are what they were before."""
    import torch
    cache = _budgeted([79, 90])
    x = _token(2, 1)
    cache.step(x[:, :4], x[:, 4:6], x[:, 6:])                # sequence 0 completes page 4
    names = ("seq_lens", "completed", "positions", "q", "out", "out_lse", "selected", "summaries")
    before = {n: getattr(cache, n).clone() for n in names}
    assert before["completed"].tolist() == [4, -1]
    x.copy_(_token(2, 2))
    cache.capture_step(x[:, :4], x[:, 4:6], x[:, 6:])
    torch.cuda.synchronize()
    for n in names:
        assert torch.equal(getattr(cache, n), before[n]), n


@pytest.mark.parametrize("lens", [[79, 95], [80, 94]])
def test_captured_budgeted_steps_equal_single_ones(lens):
    """From one below a page border and from just behind it, the captured step with the summaries of
    completed pages built before and between its replays gives the bits of steps run one by one."""
    import torch
    a, b = _budgeted(lens), _budgeted(lens)
    x = _token(2, 0)
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    for c in (a, b):
        c.step(q, k, v)                                     # may complete a page, not summarised yet
    x.copy_(_token(2, 50))
    graph = a.capture_step(q, k, v)
    for s in range(18):
        a.build_completed()
        b.build_completed()
        x.copy_(_token(2, 100 + s))
        graph.replay()
        b.step(q, k, v)
        for n in ("seq_lens", "completed", "selected", "q", "out", "out_lse", "summaries", "k_pool", "v_pool"):
            assert torch.equal(getattr(a, n), getattr(b, n)), (s, n)
    assert a.status.item() == 0 and b.status.item() == 0


def test_calls_take_a_raw_stream_handle():
    """An integer cudaStream_t wherever a stream is taken, the default stream's 0 too."""
    import torch
    a, b = _budgeted([79, 30]), _budgeted([79, 30])
    side = torch.cuda.Stream()
    for handle in (side.cuda_stream, 0):
        torch.cuda.synchronize()
        for s in range(3):
            x = _token(2, 700 + s)
            q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
            a.step(q, k, v)
            a.build_completed()
            torch.cuda.synchronize()
            b.step(q, k, v, stream=handle)
            b.build_completed(stream=handle)
            b.attend(stream=handle)
            page = b.read(b.block_table[0, :2].contiguous(), stream=handle)
            torch.cuda.synchronize()
            a.attend()
            want = a.read(a.block_table[0, :2].contiguous())
            assert torch.equal(page[0], want[0]) and torch.equal(page[1], want[1])
            for n in ("out", "out_lse", "summaries", "k_pool", "v_pool", "completed"):
                assert torch.equal(getattr(a, n), getattr(b, n)), (handle, s, n)
