"""runtime.QuantCache and the binding on the host: what they hand to the kernels, with the kernels
replaced by recorders (no GPU)."""
import numpy as np
import pytest

from sparse_paged_kv_gb300 import binding as B
from sparse_paged_kv_gb300 import build_lib, runtime


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.load_library(build_lib.build())


def make(blocks=6, budget=64, page=16, batch=2, hq=4, hkv=2):
    cfg = B.LocksKvConfig(batch=batch, n_q_heads=hq, n_kv_heads=hkv, head_dim=128, page_size=page,
                          max_pages=3, num_blocks=blocks, kv_dtype=B.LOCKS_KV_I4)
    table = np.arange(batch * 3).reshape(batch, 3) % blocks
    return runtime.QuantCache(cfg, table, budget_tokens=budget, device="cpu")


def fake_kernels(monkeypatch):
    """locks_kv_read and locks_build_completed on the CPU: a page holds its block's number, a
    summary the page's number + 1 in every byte; entries outside the pool are skipped and flagged."""
    def read(cfg, k_pool, v_pool, block_ids, k_out, v_out, status=None, stream=None):
        for i, b in enumerate(block_ids.tolist()):
            if b >= cfg.num_blocks:
                status |= B.LOCKS_DEV_BAD_BLOCK_ID
            elif b >= 0:
                k_out[i] = float(b)

    def build(cfg, pages, completed, summaries, **kw):
        assert pages.shape[0] == cfg.num_blocks == summaries.shape[0]
        for i, slot in enumerate(completed.tolist()):
            assert -1 <= slot < cfg.num_blocks
            if slot >= 0:
                summaries[slot] = int(pages[slot, 0, 0, 0].item()) + 1

    monkeypatch.setattr(B, "locks_kv_read", read)
    monkeypatch.setattr(B, "locks_build_completed", build)


@pytest.mark.parametrize("at_once", [1, 2, 1024])
def test_build_skips_block_ids_outside_the_pool(monkeypatch, at_once):
    """They are flagged, as in every call, and touch no summary (the spare row included)."""
    import torch
    fake_kernels(monkeypatch)
    cache = make()
    cache.summaries.fill_(99)
    ids = torch.tensor([4, -1, 6, 1, 11, 2 ** 31 - 1, -2 ** 31, 0], dtype=torch.int32)
    cache.build(ids, pages_at_once=at_once)
    assert cache.status.item() == B.LOCKS_DEV_BAD_BLOCK_ID
    assert [int(cache.summaries[b].unique()) for b in (0, 1, 4)] == [1, 2, 5]
    assert (cache.summaries[[2, 3, 5]] == 99).all()


def test_build_of_valid_blocks_flags_nothing(monkeypatch):
    import torch
    fake_kernels(monkeypatch)
    cache = make()
    cache.build(torch.tensor([5, 3, -1], dtype=torch.int32))
    assert cache.status.item() == 0
    assert [int(cache.summaries[b].unique()) for b in (3, 5)] == [4, 6]


@pytest.mark.parametrize("how", ["pickle", "copy", "deepcopy"])
def test_configurations_can_be_copied_and_sent(how):
    """To another process, say: the copy is equal, works, and has a C structure of its own."""
    import copy
    import dataclasses
    import pickle
    again = {"pickle": lambda x: pickle.loads(pickle.dumps(x)), "copy": copy.copy,
             "deepcopy": copy.deepcopy}[how]
    cache = make()
    c = cache.cfg
    assert c.pool_bytes > 0                                # (kept in the instance from here on)
    d = again(c)
    assert d == c and hash(d) == hash(c) and type(d) is type(c)
    assert d.c() is not c.c() and bytes(d.c()) == bytes(c.c())
    assert B.kv_record_bytes(d) == B.kv_record_bytes(c) and d.pool_bytes == c.pool_bytes
    assert dataclasses.replace(d, batch=5).c().batch == 5
    assert again(cache.locks_cfg) == cache.locks_cfg


def test_a_first_call_in_another_thread_finds_the_types(monkeypatch):
    """Torch is published once its types are there: a thread that comes in between checks the
    same tensor as the one that loads it."""
    import threading

    import torch
    errors = []

    def check():
        try:
            B._typed(torch.zeros(1, dtype=torch.int32), "int32", "x")
        except Exception as e:
            errors.append(e)

    class Types(dict):
        def update(self, *a, **kw):                       # the moment at which they are filled in
            if not self.entered:
                self.entered = True
                other = threading.Thread(target=check)
                other.start()
                other.join(10)
            super().update(*a, **kw)

    types = Types()
    types.entered = False
    monkeypatch.setattr(B, "_torch", None)
    monkeypatch.setattr(B, "_DTYPES", types)
    check()
    assert errors == [] and types.entered and B._torch is torch

FAKE = 0x10000   # never dereferenced: every call below returns before a launch


@pytest.mark.parametrize("hq,hkv,with_q", [(1 << 23, 1 << 22, True), (1 << 16, 1 << 16, False),
                                           ((1 << 15) + 1, (1 << 15) + 1, False), (7 << 13, 1 << 13, True)])
def test_write_refuses_more_rows_a_token_than_it_can_number(hq, hkv, with_q):
    """2^16 rows of a token (its key, its value and, where they are passed, its query heads), less
    than any of these has."""
    c = B.LocksKvConfig(batch=1, n_q_heads=hq, n_kv_heads=hkv, head_dim=128, page_size=64, max_pages=4,
                        num_blocks=1, kv_dtype=B.LOCKS_KV_F8)
    q, q_out = (FAKE, FAKE + 16) if with_q else (None, None)
    assert B.kv_record_bytes(c) > 0                        # (the other calls take it)
    assert B.load_library().locks_kv_write(
        c.ref, FAKE, hkv * 128, FAKE, hkv * 128, q, hq * 128, q_out, FAKE, FAKE, 2, None, FAKE, FAKE, FAKE,
        None, None, None, None) == B.LOCKS_ERR_UNSUPPORTED


def test_rope_refuses_more_heads_than_it_can_number():
    """2^24 heads: the strides between a thread's heads stay far from 32 bits."""
    import ctypes
    table = ctypes.byref(B.locks_rope_table_t(FAKE, 2, 0, 1.0))
    for heads in ((1 << 24) + 1, (1 << 31) - 1):
        assert B.load_library().locks_rope(table, B.LOCKS_BF16, 2, FAKE, heads * 2, 2, FAKE, 1, heads, FAKE,
                                           heads * 2, 2, 0, None) == B.LOCKS_ERR_UNSUPPORTED


def test_summaries_without_a_budget_are_refused_by_name():
    import torch
    cache = make(budget=0)
    with pytest.raises(ValueError, match="budget_tokens"):
        cache.build(torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="budget_tokens"):
        cache.build_completed()


@pytest.mark.parametrize("budget", [-64, 1, 16, 257 * 16])
def test_a_budget_that_the_selection_refuses_is_refused_at_once(budget):
    """And not by a step that has written its token already: 2 to 256 pages."""
    with pytest.raises(B.LocksError):
        make(budget=budget)


@pytest.mark.parametrize("budget,k", [(17, 2), (256 * 16, 256)])
def test_the_smallest_and_the_largest_budget(budget, k):
    assert make(budget=budget).selected.shape == (2, 2, k)


@pytest.mark.parametrize("over", [dict(page=32, budget=128), dict(hq=6), dict(hq=32)])
def test_shapes_that_the_selection_refuses_are_refused_with_a_budget_only(over):
    """Pages of 32, groups of 3 and of 16 heads."""
    with pytest.raises(B.LocksError):
        make(**over)
    assert make(**{**over, "budget": 0}).selected is None
