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


def _running():
    """A batch of which sequences 0 and 3 have lost tokens, and queries for its newest rows."""
    import torch
    c, gen = cache([200, 100, 80, 150], 4, 60, 8, seed=9)
    c.observe(torch.randn(4, 4, 8, 128, generator=gen).bfloat16().cuda())
    for _ in range(6):
        c.step(*(torch.randn(4, h, 128, generator=gen).bfloat16().cuda() for h in (8, 2, 2)))
    assert c.evicted.tolist() == [82, 0, 0, 32]
    return c, torch.randn(4, 4, 8, 128, generator=gen).bfloat16().cuda()


def _held(c, b):
    import torch
    n, page = int(c.seq_lens[b]), c.cfg.page_size
    at = torch.arange(n, device="cuda")
    blk = c.block_table[b].long()[at // page]
    return [x[blk, :, at % page].clone() for x in (c.k_cache, c.v_cache, c.weights, c.positions)]


def test_observe_keeps_the_order_of_sequences_that_lost_tokens():
    import torch
    c, q = _running()
    before = [_held(c, b) for b in range(4)]
    c.observe(q)
    for b in (0, 3):
        assert all(torch.equal(x, y) for x, y in zip(_held(c, b), before[b]))
    for b, n in ((1, 106), (2, 86)):
        now = _held(c, b)
        assert (now[3][64:] == torch.arange(64, n, device="cuda")[:, None]).all()
        # four rows of four heads hand out one each, and what was gathered before is gone
        assert (now[2][64:].sum(0) <= 16 * (1 + 1e-5)).all() and not torch.equal(now[2][64:], before[b][2][64:])
    assert c.evicted.tolist() == [82, 0, 0, 32] and c.status.item() == 0


@pytest.mark.parametrize("on_device", [False, True])
def test_a_sequence_that_joins_is_observed_alone(on_device):
    """Its tokens as in a batch of its own; those of the others as they were."""
    import torch
    c, q = _running()
    gen = torch.Generator().manual_seed(1)
    n, page = 170, c.cfg.page_size
    at = torch.arange(64, n, device="cuda")
    blk = c.block_table[3].long()[at // page]
    for pool in (c.k_cache, c.v_cache):
        pool[blk, :, at % page] = torch.randn(n - 64, 2, 128, generator=gen).bfloat16().cuda()
    c.seq_lens[3], c.evicted[3] = n, 0
    whole = [x[c.block_table[3].long()[torch.arange(n, device="cuda") // page], :, torch.arange(n, device="cuda") % page].double()
             .cpu().numpy() for x in (c.k_cache, c.v_cache)]
    before = [_held(c, b) for b in range(3)]
    joins = torch.tensor([0, 0, 0, 1], device="cuda").bool() if on_device else [False, False, False, True]
    lse = c.observe(q, sequences=joins)[1]
    for b in range(3):
        assert all(torch.equal(x, y) for x, y in zip(_held(c, b), before[b]))
    assert c.seq_lens.tolist() == [124, 106, 86, 124] and c.evicted.tolist() == [82, 0, 0, 46]
    k, v, w, pos = (x.cpu() for x in _held(c, 3))
    for h in range(2):
        a = slice(4 * h, 4 * h + 4)
        want, bound = R.weigh(q[3, :, a].double().cpu().numpy(), lse[3, :, a].double().cpu().numpy(), whole[0][:, h], n, 64,
                              None, 0, 1.0)
        t = pos[64:, h].numpy()
        assert np.unique(t).size == 60 and t.min() >= 64 and (np.sort(t)[-8:] == np.arange(n - 8, n)).all()
        assert (np.abs(w[64:, h].double().numpy() - want[t - 64]) <= bound[t - 64]).all()
        for x, y in ((k, whole[0]), (v, whole[1])):
            assert (x[64:, h].double().numpy() == y[t, h]).all()
        lost = np.setdiff1d(np.arange(64, n - 8), t)
        kept = np.setdiff1d(t, np.arange(n - 8, n))
        assert want[lost - 64].max() <= want[kept - 64].min() + 2 * bound.max()
    with pytest.raises(ValueError):
        c.observe(q, sequences=[True])
    assert c.status.item() == 0


def test_steps_of_a_prompt_that_was_not_observed():
    """Its newest tokens count as recent all the same."""
    import torch
    c, gen = cache([200, 160, 90], 4, 60, 40, seed=11)
    for step in range(1, 4):
        c.step(*(torch.randn(3, h, 128, generator=gen).bfloat16().cuda() for h in (8, 2, 2)))
        assert c.next_positions().tolist() == [200 + step, 160 + step, 90 + step]
        for b, n in enumerate((200, 160, 90)):
            pos = _held(c, b)[3][64:].sort(0).values
            for h in range(2):
                assert pos[:, h].unique().numel() == pos.shape[0] == min(60, n + step - 64)
                held = min(pos.shape[0], 40)
                assert pos[-held:, h].tolist() == list(range(n + step - held, n + step))


@pytest.mark.parametrize("hq,hkv,rows", [(4, 1, 4), (8, 2, 2), (16, 1, 16)])
def test_weigh_rows_that_are_off_may_hold_anything(hq, hkv, rows):
    """Query rows whose log-sum-exp is -inf, NaN and infinities in them: no weight.  A row that counts and
    holds a NaN gives one to what it sees."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    lens, g = [200, 1, 0, 150], hq // hkv
    b = Batch(lens, hq, hkv, 32, rows=rows, seed=rows).attend()
    q = b.q.double().cpu().numpy()
    b.lse[0, rows - 1, 1], b.lse[0, 0] = -float("inf"), -float("inf")       # (the one token of sequence 1 has the last row)
    b.q[0, rows - 1, 1], b.q[0, 0], b.q[1, :rows - 1] = float("nan"), float("inf"), -float("inf")
    out = torch.zeros(b.cfg.num_blocks, hkv, 32, device="cuda")
    B.locks_weigh(b.cfg, b.q, b.lse, b.k, b.block_table, b.seq_lens, None, out, status=b.status)
    got, lse = out.double().cpu().numpy(), b.lse.double().cpu().numpy()
    for i, n in enumerate(lens):
        for h in range(hkv):
            a = slice(h * g, h * g + g)
            want, bound = R.weigh(q[i, :, a], lse[i, :, a], b.rows_of(i, h)[0], n, 0, None, 0, 1.0)
            assert (np.abs(R.slots(got, b.table[i], h, n) - want) <= bound).all(), (i, h)
    b.q[3, rows - 1, g - 1, 5] = float("nan")
    B.locks_weigh(b.cfg, b.q, b.lse, b.k, b.block_table, b.seq_lens, None, out, status=b.status)
    now = out.double().cpu().numpy()
    assert np.isnan(R.slots(now, b.table[3], 0, 150)).all()
    for i, h in [(i, h) for i in range(4) for h in range(hkv) if (i, h) != (3, 0)]:
        assert (R.slots(now, b.table[i], h, lens[i]) == R.slots(got, b.table[i], h, lens[i])).all()
    assert b.status.item() == 0


# --------------------------------------------------------------------------
# eviction whose recent tokens lie among many others
# --------------------------------------------------------------------------
RECENT = [
    # lens, hkv, page, budget, recent, fixed
    ([5000, 4990], 1, 64, 1000, 300, 3),                        # a block a head
    ([40000], 2, 16, 3000, 500, 7),                             # clusters
    ([40000], 2, 16, 39995, 500, 6),                            # none to evict
    ([40000, 39998], 2, 16, 39990, 500, 6),                     # a few
    ([30001], 1, 64, 15000, 15000, 0),                          # nothing but recent ones
    ([700000], 1, 16, 5000, 100, 3),                            # chunks of the keys
    ([30000], 8, 16, 4000, 300, 5),                             # eight heads on one large cluster each
    ([33000, 32900], 8, 64, 2000, 100, 4),                      # sixteen heads of two blocks an SM
]


def run_evict(lens, hkv, page, budget, recent, fixed, w, pos, gone):
    """One call on heads whose n slots have weights and positions w, pos [sequence][head][n], against the plain form."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    batch, pages = len(lens), max(-(-n // page) for n in lens)
    rng = np.random.default_rng(batch + budget)
    blocks = batch * pages + 2
    table = rng.permutation(blocks)[:batch * pages].reshape(batch, pages).astype(np.int32)
    pools = [np.full((blocks, hkv, page), 123.0, np.float32), np.full((blocks, hkv, page), -5, np.int32)]
    gen = torch.Generator(device="cuda").manual_seed(budget)
    kv = [torch.randn(blocks, hkv, page, 128, generator=gen, device="cuda").bfloat16() for _ in "kv"]
    for b, n in enumerate(lens):
        t = np.arange(n)
        for h in range(hkv):
            for pool, x in zip(pools, (w, pos)):
                pool[table[b, t // page], h, t % page] = x[b][h]
    want, want_kv = [x.copy() for x in pools], [x.clone() for x in kv]
    for b, n in enumerate(lens):
        for h in range(hkv):
            holes, movers = R.evict(w[b][h], pos[b][h], n, fixed, gone, budget, recent)
            for pool, old in zip(want, pools):
                pool[table[b, holes // page], h, holes % page] = old[table[b, movers // page], h, movers % page]
            src, dst = ([torch.from_numpy(x.astype(np.int64)).cuda() for x in (table[b, y // page], y % page)]
                        for y in (movers, holes))
            for pool, old in zip(want_kv, kv):
                pool[dst[0], h, dst[1]] = old[src[0], h, src[1]]
    cfg = B.LocksConfig(batch=batch, n_q_heads=hkv, n_kv_heads=hkv, head_dim=128, page_size=page, rank=8,
                        max_pages=pages, num_blocks=blocks)
    dev = [torch.from_numpy(x).cuda() for x in pools]
    seq_lens, evicted, status = Batch.ints(lens), Batch.ints([gone] * batch), Batch.ints([0])
    ws = torch.zeros(B.evict_workspace_bytes(cfg, budget), dtype=torch.uint8, device="cuda")
    B.locks_evict(cfg, budget, recent, *kv, Batch.ints(table), seq_lens, *dev, evicted, ws, fixed=Batch.ints([fixed] * batch),
                  status=status)
    after = [min(n, fixed + budget) for n in lens]
    assert seq_lens.tolist() == after and status.item() == 0
    assert evicted.tolist() == [gone + n - m for n, m in zip(lens, after)]
    for got, x in zip(dev, want):
        assert (got.cpu().numpy().view(np.int32) == x.view(np.int32)).all()
    for got, x in zip(kv, want_kv):
        assert torch.equal(got.view(torch.int16), x.view(torch.int16))


@pytest.mark.parametrize("lens,hkv,page,budget,recent,fixed", RECENT)
@pytest.mark.parametrize("distinct", [0, 5])
def test_evict_recent_tokens_of_long_heads(lens, hkv, page, budget, recent, fixed, distinct):
    """The newest positions lie anywhere and stay, the lightest of all among them."""
    rng = np.random.default_rng(budget + recent)
    gone, w, pos = 777, [], []
    for n in lens:
        w.append(rng.random((hkv, n), np.float32))
        if distinct:
            w[-1] = np.floor(w[-1] * distinct)
        pos.append(np.empty((hkv, n), np.int32))
        for h in range(hkv):
            held = rng.choice(n + gone - recent - fixed, n - fixed - recent, replace=False) + fixed
            held = np.concatenate([held, np.arange(n + gone - recent, n + gone)])
            pos[-1][h, :fixed], pos[-1][h, fixed:] = np.arange(fixed), rng.permutation(held)
            newest = pos[-1][h] >= n + gone - recent
            assert newest.sum() == recent > 0
            light = newest & (rng.random(n) < 0.5)
            assert light.any()
            w[-1][h, light] = -1.0                              # below every other: only their positions keep them
    run_evict(lens, hkv, page, budget, recent, fixed, w, pos, gone)


@pytest.mark.parametrize("lens,budget", [([40000], 3000), ([300], 40), ([700000], 5000)])
def test_evict_more_recent_tokens_than_the_budget(lens, budget):
    """Positions that occur twice: of equal ones the lower slots stay."""
    rng = np.random.default_rng(budget)
    w = [rng.random((1, n), np.float32) for n in lens]
    pos = [rng.integers(n - budget, n, (1, n)).astype(np.int32) for n in lens]
    pos[0][0, ::3] = 0
    assert (pos[0] >= lens[0] - budget).sum() > budget
    run_evict(lens, 1, 16, budget, budget, 2, w, pos, 0)
