"""The operators of a batch that shares prefixes and lives within a budget, on the GPU, where their inputs
are unusual: prefixes that nobody sees whole, rows without weight, recent tokens, many long heads, other streams."""
import numpy as np
import pytest

from tests import batch_ref as R
from tests.test_gpu_batch import Batch, _lib, cache  # noqa: F401

pytestmark = pytest.mark.gpu

INSIDE = [
    # lens, hq, hkv, page, starts, prefix pages, rows
    ([40, 30], 8, 2, 32, [0, 2], [2], 1),                       # in the last page of the prefix
    ([100, 70], 4, 1, 64, [0, 2], [4], 1),                      # a stage before its end
    ([300, 130, 5, 0], 6, 2, 64, [0, 4], [20], 1),              # many stages before it
    ([0, 0, 50], 4, 1, 32, [0, 2], [3], 1),                     # nobody sees any of it
    ([700, 690, 30, 20], 4, 1, 16, [0, 2, 4], [40, 4], 3),      # one group past its prefix, one within
    ([200 - i for i in range(40)], 8, 1, 64, [0, 40], [9], 1),  # 320 rows: a pair of tiles and a lone one
    ([90 - i % 50 for i in range(210)], 2, 1, 16, list(range(0, 211, 3)), [8] * 70, 1),   # many groups
    ([150, 0, 20] * 25, 4, 1, 64, list(range(76)), [2, 1, 1] * 25, 2),                     # one sequence each
]


@pytest.mark.parametrize("lens,hq,hkv,page,starts,prefix,rows", INSIDE)
def test_prefix_that_nobody_sees_whole(lens, hq, hkv, page, starts, prefix, rows):
    """Sequences end inside their group's prefix: what none of them sees may hold NaN and infinities, and its
    pages may have no block yet."""
    import torch
    b = Batch(lens, hq, hkv, page, starts, prefix, rows, seed=len(lens))
    used = torch.zeros(b.k.shape[:3], dtype=torch.bool)
    for i, n in enumerate(lens):
        t = np.arange(n)
        used[b.table[i, t // page], :, t % page] = True
    for pool in (b.k, b.v):
        pool[~used.cuda()] = torch.tensor([float("nan"), float("inf")] * 64, device="cuda").bfloat16()
    table = b.table.copy()
    for a, z in zip(starts, starts[1:]):
        for i in range(a, z):
            table[i, -(-max(lens[a:z]) // page):] = -1
    b.block_table = b.ints(table)
    b.ws = torch.full_like(b.ws, 255)
    b.attend().check()


def test_observe_on_another_stream():
    """observe() and steps on a busy side stream, their results dropped while the current stream takes memory
    and writes it: the bits of the same run on one stream."""
    import torch
    runs = []
    for side in (None, torch.cuda.Stream()):
        c, gen = cache([200, 130, 64], 4, 60, 8, seed=3)
        q = torch.randn(3, 4, 8, 128, generator=gen).bfloat16().cuda()
        rows = [[torch.randn(3, h, 128, generator=gen).bfloat16().cuda() for h in (8, 2, 2)] for _ in range(5)]
        drafted = torch.randn(3, 2, 8, 128, generator=gen).bfloat16().cuda()
        if side is not None:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                big = torch.ones(8192, 8192, device="cuda", dtype=torch.bfloat16)
                for _ in range(20):
                    big @ big
        c.observe(q, stream=side)
        taken = [torch.full_like(q, float("nan")), torch.full(q.shape[:-1], -1e30, device="cuda")]
        for r in rows:
            c.step(*r, stream=side)
        out, lse = c.attend(drafted, stream=side)
        taken += [torch.full_like(drafted, float("nan")), torch.full(drafted.shape[:-1], -1e30, device="cuda")]
        nxt = c.next_positions(stream=side)
        torch.cuda.synchronize()
        runs.append([out, lse, nxt, c.out, c.k_cache, c.v_cache, c.weights, c.positions, c.seq_lens, c.evicted, c.status])
        del taken
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_steps_with_room_for_one_token():
    """A budget that leaves one slot of a sequence's pages: every step appends, evicts one and goes on."""
    import torch
    c, gen = cache([384, 100, 383], 4, 319, 8, seed=5)          # 384 slots: 64 of a prefix, 319 and one
    c.observe(torch.randn(3, 4, 8, 128, generator=gen).bfloat16().cuda())
    nxt = c.next_positions().tolist()
    assert nxt == [384, 100, 383]
    for step in range(1, 301):
        c.step(*(torch.randn(3, h, 128, generator=gen).bfloat16().cuda() for h in (8, 2, 2)))
        if step in (1, 2, 283, 284, 300):
            assert c.next_positions().tolist() == [n + step for n in nxt]
            assert c.seq_lens.tolist() == [383, min(383, 100 + step), 383]
            for b in range(3):                                  # what is held: the newest 8, nothing twice
                n = int(c.seq_lens[b])
                for h in range(2):
                    pos = R.slots(c.positions.cpu().numpy(), c.block_table.cpu().numpy()[b], h, n)[64:]
                    assert np.unique(pos).size == pos.size and (np.sort(pos)[-8:] == nxt[b] + step - 8 + np.arange(8)).all()
    assert c.status.item() == 0
