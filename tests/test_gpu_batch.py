"""The operators of a batch that shares prefixes and lives within a budget, on the GPU, against their plain
64-bit forms: attention of the newest tokens, weights of cached tokens, eviction, a run of them together."""
import importlib.util
import os

import numpy as np
import pytest

from tests import batch_ref as R

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    from sparse_paged_kv_gb300 import binding, build_lib
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    binding.load_library(build_lib.build())


class Batch:
    """Random pools, a block table in which groups share their prefix, queries."""

    def __init__(self, lens, hq, hkv, page, starts=(), prefix=(), rows=1, seed=0, scale=1.0, spare=2, pages=None):
        import torch
        from sparse_paged_kv_gb300 import binding as B
        rng = np.random.default_rng(seed)
        self.lens, self.hq, self.hkv, self.page, self.rows = list(lens), hq, hkv, page, rows
        self.starts, self.prefix, self.g = list(starts), list(prefix), hq // hkv
        batch = len(self.lens)
        pages = pages or max(1, max([-(-n // page) for n in self.lens] + self.prefix))
        blocks = batch * pages + spare
        self.table = rng.permutation(blocks)[:batch * pages].reshape(batch, pages).astype(np.int32)
        for a, z, n in zip(self.starts, self.starts[1:], self.prefix):
            self.table[a:z, :n] = self.table[a, :n]
        gen = torch.Generator().manual_seed(seed)

        def bf16(*shape, size=1.0):
            return (torch.randn(*shape, generator=gen) * size).bfloat16().cuda()

        self.k, self.v = bf16(blocks, hkv, page, 128), bf16(blocks, hkv, page, 128)
        self.q = bf16(batch, rows, hq, 128, size=scale)
        self.cfg = B.LocksConfig(batch=batch, n_q_heads=hq, n_kv_heads=hkv, head_dim=128, page_size=page, rank=8,
                                 max_pages=pages, num_blocks=blocks)
        self.seq_lens, self.block_table = self.ints(self.lens), self.ints(self.table)
        self.status = self.ints([0])
        n = len(self.prefix)
        self.ws = torch.zeros(B.prefix_workspace_bytes(self.cfg, n, rows), dtype=torch.uint8, device="cuda")
        self.out = torch.full_like(self.q, 7.0)
        self.lse = torch.full((batch, rows, hq), 7.0, device="cuda")
        self.gs, self.pp = (self.ints(self.starts), self.ints(self.prefix)) if n else (None, None)

    @staticmethod
    def ints(x):
        import torch
        return torch.from_numpy(np.asarray(x, np.int32)).cuda()

    def attend(self, **kw):
        from sparse_paged_kv_gb300 import binding as B
        B.locks_prefix_decode(self.cfg, self.q, self.k, self.v, self.block_table, self.seq_lens, self.gs, self.pp,
                              self.out, self.ws, out_lse=self.lse, status=self.status, **kw)
        return self

    def rows_of(self, b, h):
        """(keys, values) in 64 bits of what sequence b holds in head h."""
        import torch
        blk = torch.from_numpy(self.table[b, :-(-self.lens[b] // self.page)].astype(np.int64)).cuda()
        return [x[blk, h].reshape(-1, 128)[:self.lens[b]].double().cpu().numpy() for x in (self.k, self.v)]

    def check(self, status=0, sequences=None):
        q, out, lse = (x.double().cpu().numpy() for x in (self.q, self.out, self.lse))
        for b in sequences if sequences is not None else range(len(self.lens)):
            for h in range(self.hkv):
                a = slice(h * self.g, h * self.g + self.g)
                k, v = self.rows_of(b, h)
                for r in range(self.rows):
                    n = R.limit(self.lens[b], self.rows, r)
                    o, l, bo, bl = R.attend(q[b, r, a], k[:n], v[:n])
                    if n == 0:
                        assert (out[b, r, a] == 0).all() and np.isneginf(lse[b, r, a]).all()
                        continue
                    assert (np.abs(out[b, r, a] - o) <= bo).all(), (b, h, r, np.abs(out[b, r, a] - o).max())
                    assert (np.abs(lse[b, r, a] - l) <= bl).all(), (b, h, r)
        assert self.status.item() == status
        return self


PREFIX = [
    # lens, hq, hkv, page, starts, prefix pages, rows
    ([1], 4, 1, 64, [], [], 1),
    ([129], 1, 1, 16, [], [], 1),
    ([0, 5, 128], 8, 2, 32, [], [], 1),
    ([200, 130, 129, 128], 8, 2, 64, [0, 4], [2], 1),
    ([70, 0, 40, 64, 65], 6, 2, 32, [0, 5], [2], 1),                       # some end inside the prefix
    ([300] * 9 + [77] * 3, 16, 1, 16, [0, 9, 12], [18, 0], 1),             # 144 rows: two tiles
    ([1000 + i for i in range(33)], 8, 2, 64, [0, 33], [15], 1),           # 132 rows: a pair of tiles
    ([260 + i for i in range(70)], 8, 1, 16, [0, 3, 70], [3, 16], 1),      # 268 rows and a lone tile
    ([513, 600, 2, 700], 4, 1, 64, [0, 4], [8], 7),                        # drafted tokens
    ([400, 390], 5, 1, 32, [0, 2], [12], 50),                              # 2 * 25 tokens of 5 heads: two tiles
    ([100, 33], 1, 1, 16, [], [], 256),
    ([90, 17], 48, 3, 64, [0, 2], [0], 16),
    ([3000], 32, 8, 64, [0, 1], [20], 1),
    ([1, 2, 3, 4], 2, 2, 16, [1, 3], [0], 1),                              # groups that leave sequences out
    ([64] * 700, 1, 1, 64, [0, 350, 700], [1, 0], 1),                      # more entries than threads
]


@pytest.mark.parametrize("lens,hq,hkv,page,starts,prefix,rows", PREFIX)
def test_prefix_attention(lens, hq, hkv, page, starts, prefix, rows):
    n = len(lens)
    Batch(lens, hq, hkv, page, starts, prefix, rows, seed=n).attend().check(
        sequences=None if n < 100 else [0, 1, 349, 350, 698, 699])


@pytest.mark.parametrize("scale", [1e-3, 8.0, 40.0])
def test_prefix_scales_of_logits(scale):
    """Flat rows, and rows that one token dominates, whose maximum moves from stage to stage."""
    Batch([900, 640, 641], 8, 1, 64, [0, 3], [10], 2, seed=3, scale=scale).attend().check()


def test_prefix_long():
    """A list longer than the blocks: one unit in many pieces, and pieces of many stages."""
    Batch([40000, 40001, 39937], 4, 2, 64, [0, 3], [624], 1, seed=5).attend().check()
    Batch([70000], 2, 1, 16, [], [], 3, seed=6).attend().check()


def test_prefix_masked_places_may_hold_anything():
    """NaN and infinities behind the sequences' ends, in free blocks and in a padded sequence's pages."""
    import torch
    b = Batch([130, 0, 97, 64], 8, 2, 32, [0, 4], [2], 1, seed=7)
    used = torch.zeros(b.k.shape[:3], dtype=torch.bool, device="cuda")
    for i, n in enumerate(b.lens):
        for t in range(n):
            used[int(b.table[i, t // 32]), :, t % 32] = True
    for pool in (b.k, b.v):
        pool[~used] = torch.tensor([float("nan"), float("inf")] * 64, device="cuda").bfloat16()
    b.attend().check()


def test_prefix_attended_nan_reaches_its_sequence_only():
    import torch
    b = Batch([300, 290, 310], 4, 1, 64, [0, 3], [4], 1, seed=8)
    b.k[int(b.table[1, 4]), 0, 3] = float("nan")           # a token of sequence 1's own
    b.v[int(b.table[2, 4]), 0, 0, 5] = float("inf")
    b.attend()
    assert torch.isnan(b.out[1].float()).all() and torch.isnan(b.lse[1]).all()
    assert torch.isinf(b.out[2, 0, :, 5].float()).all() and torch.isfinite(b.out[2, 0, :, :5].float()).all()
    b.check(sequences=[0])


def test_prefix_bad_blocks_and_groups():
    from sparse_paged_kv_gb300 import binding as B
    b = Batch([300, 300], 4, 1, 64, [0, 2], [2], 1, seed=9)
    b.table[1, 2] = b.cfg.num_blocks                        # of sequence 1's own pages
    b.block_table = b.ints(b.table)
    b.attend().check(status=B.LOCKS_DEV_BAD_BLOCK_ID, sequences=[0])
    k, v = (np.delete(x, np.s_[128:192], 0) for x in (lambda t: [p[t].reshape(-1, 128)[:300] for p in (
        b.k[:, 0].double().cpu().numpy(), b.v[:, 0].double().cpu().numpy())])(np.minimum(b.table[1], b.cfg.num_blocks - 1)))
    o, l, bo, bl = R.attend(b.q[1, 0].double().cpu().numpy(), k, v)
    assert (np.abs(b.out[1, 0].double().cpu().numpy() - o) <= bo).all()
    assert (np.abs(b.lse[1, 0].double().cpu().numpy() - l) <= bl).all()
    # lengths past the table and groups out of order are clamped and flagged; nothing is read out of range
    b = Batch([300, 300], 4, 1, 64, [0, 2], [2], 1, seed=9)
    b.seq_lens.copy_(b.ints([300, 10 ** 6]))
    b.attend().check(status=B.LOCKS_DEV_BAD_SEQ_LEN, sequences=[0])
    b = Batch([200, 200], 4, 1, 64, [0, 2], [2], 1, seed=9)
    for starts, pages in (([0, 3], [2]), ([-1, 2], [2]), ([0, 2], [99]), ([0, 2], [-1]), ([2, 0], [1])):
        b.status.zero_()
        b.gs.copy_(b.ints(starts))
        b.pp.copy_(b.ints(pages))
        b.attend()
        assert b.status.item() & B.LOCKS_DEV_BAD_GROUP
        if pages != [99]:                                   # every sequence through its own row, whole
            b.check(status=B.LOCKS_DEV_BAD_GROUP)
    # many groups out of order that claim every sequence again and again
    b = Batch([200 + i for i in range(80)], 4, 1, 64, [0] + [79, 0] * 39 + [79], [2] * 79, 1, seed=10)
    b.attend().check(status=B.LOCKS_DEV_BAD_GROUP, sequences=[0, 41, 79])


def test_prefix_is_deterministic_and_replays():
    """Twice the same bits, with other calls between; captured and replayed with other lengths and queries;
    a workspace that two captured calls share; calls on other streams with workspaces of their own."""
    import torch
    a = Batch([700, 650, 641, 0], 8, 2, 64, [0, 4], [10], 1, seed=11)
    b = Batch([1000 + i for i in range(40)], 8, 2, 64, [0, 40], [15], 1, seed=12)
    first = [x.attend().out.clone() for x in (a, b)]
    shared = torch.zeros(max(a.ws.numel(), b.ws.numel()), dtype=torch.uint8, device="cuda")
    shared.fill_(255)                                       # (it needs no zeros)
    a.ws = b.ws = shared
    graphs = []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.attend()
        graphs.append(g)
    for _ in range(3):
        for x, g, want in zip((a, b), graphs, first):
            x.out.fill_(3.0)
            g.replay()
            assert torch.equal(x.out, want)
    a.lens = [642, 700, 0, 650]
    a.seq_lens.copy_(a.ints(a.lens))
    a.q.copy_(torch.randn(a.q.shape, generator=torch.Generator().manual_seed(1)).bfloat16())
    graphs[0].replay()
    a.check()
    a.ws, b.ws = torch.zeros_like(shared), torch.zeros_like(shared)
    want = [a.attend().out.clone(), first[1]]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for x, s in zip((a, b), streams):
            x.attend(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])


def test_prefix_against_dense_decode():
    """With nothing shared it is the library's dense decode of the same cache."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    b = Batch([500, 64, 1, 333], 8, 2, 64, seed=13).attend()
    out, lse = torch.empty(4, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(4, 8, device="cuda")
    ws = torch.zeros(B.decode_workspace_bytes(b.cfg, b.cfg.max_pages), dtype=torch.uint8, device="cuda")
    B.locks_dense_decode(b.cfg, b.q[:, 0].contiguous(), b.k, b.v, b.block_table, b.seq_lens, out, ws, out_lse=lse)
    b.check()
    # each within its own bf16 roundings of the same number: of the weights and of the output
    assert (b.out[:, 0].float() - out.float()).abs().max() <= 4 * R.HALF_BF16 * b.v.float().abs().max()
    assert (b.lse[:, 0] - lse).abs().max() < 1e-4


def test_far_offsets():
    """Rows that begin more than 2^31 elements into their pool."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    blocks, hkv, page = 33000, 8, 64
    n = 200
    k = torch.zeros(blocks, hkv, page, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = np.array([[blocks - 1, blocks - 3, blocks - 2, blocks - 4]], np.int32)
    gen = torch.Generator(device="cuda").manual_seed(0)
    for pool in (k, v):
        pool[-4:] = torch.randn(4, hkv, page, 128, generator=gen, device="cuda").bfloat16()
    assert k[-4].storage_offset() > 1 << 31
    b = Batch([n], 8, 8, page, seed=2)
    b.k, b.v, b.table, b.block_table = k, v, table, b.ints(table)
    b.cfg = B.LocksConfig(batch=1, n_q_heads=8, n_kv_heads=8, head_dim=128, page_size=page, rank=8, max_pages=4,
                          num_blocks=blocks)
    b.ws = torch.zeros(B.prefix_workspace_bytes(b.cfg, 0), dtype=torch.uint8, device="cuda")
    b.attend().check()
    w = torch.zeros(blocks, hkv, page, device="cuda")
    pos = torch.zeros(blocks, hkv, page, dtype=torch.int32, device="cuda")
    gone = b.ints([0])
    B.locks_weigh(b.cfg, b.q, b.lse, k, b.block_table, b.seq_lens, None, w, positions=pos, evicted=gone)
    total = w.sum().item()
    assert abs(total - 8) < 1e-3 and w[:-4].abs().sum().item() == 0
    ws = torch.zeros(B.evict_workspace_bytes(b.cfg, 100), dtype=torch.uint8, device="cuda")
    before = [p[-4:].clone() for p in (k, w, pos)]
    B.locks_evict(b.cfg, 100, 10, k, v, b.block_table, b.seq_lens, w, pos, gone, ws)
    assert b.seq_lens.item() == 100 and gone.item() == 100
    for h in range(hkv):
        flat = before[1][[3, 1, 2, 0], h].reshape(-1)[:n].cpu().numpy()
        where = before[2][[3, 1, 2, 0], h].reshape(-1)[:n].cpu().numpy()
        holes, movers = R.evict(flat, where, n, 0, 0, 100, 10)
        got = k[[blocks - 1, blocks - 3], h].reshape(-1, 128)
        assert torch.equal(got[holes], before[0][[3, 1, 2, 0], h].reshape(-1, 128)[movers])


# --------------------------------------------------------------------------
# weights
# --------------------------------------------------------------------------
WEIGH = [
    # lens, hq, hkv, page, rows, fixed, n_new, decay, old
    ([1], 1, 1, 16, 1, None, 1, 1.0, True),
    ([130, 0, 64], 8, 2, 64, 1, None, 1, 0.5, True),
    ([300, 257, 128], 6, 2, 32, 1, [3, 100, 128], 1, 1.0, True),
    ([300, 5, 77], 16, 1, 16, 3, [0, 5, 64], 3, 0.9, True),
    ([200, 31], 4, 1, 64, 32, None, 0, 1.0, False),
    ([400, 399], 5, 1, 32, 50, [17, 33], 7, 1.0, True),
    ([100, 90], 1, 1, 16, 256, None, 0, 1.0, False),
    ([1000] * 40, 2, 2, 16, 2, None, 2, 0.0, True),
    ([9000, 40], 48, 3, 64, 16, [64, 0], 16, 1.0, True),
]


@pytest.mark.parametrize("lens,hq,hkv,page,rows,fixed,n_new,decay,old", WEIGH)
@pytest.mark.parametrize("in_place", [False, True])
def test_weigh(lens, hq, hkv, page, rows, fixed, n_new, decay, old, in_place):
    import torch
    from sparse_paged_kv_gb300 import binding as B
    if in_place and not old:
        pytest.skip("nothing to be in place of")
    b = Batch(lens, hq, hkv, page, rows=rows, seed=len(lens) + rows).attend()
    shape = (b.cfg.num_blocks, hkv, page)
    gen = torch.Generator().manual_seed(4)
    was = torch.rand(shape, generator=gen).cuda() * 3 if old else None
    out = was.clone() if in_place else torch.full(shape, -5.0, device="cuda")
    before = out.clone()
    pos = torch.full(shape, -7, dtype=torch.int32, device="cuda")
    gone = b.ints([11 * i for i in range(len(lens))])
    B.locks_weigh(b.cfg, b.q, b.lse, b.k, b.block_table, b.seq_lens, out if in_place else was, out, n_new=n_new,
                  decay=decay, fixed=None if fixed is None else b.ints(fixed), positions=pos, evicted=gone,
                  status=b.status)
    got, p = out.double().cpu().numpy(), pos.cpu().numpy()
    q, lse = b.q.double().cpu().numpy(), b.lse.double().cpu().numpy()
    touched = np.zeros(shape, bool)
    for i, n in enumerate(lens):
        first = 0 if fixed is None else fixed[i]
        t = np.arange(min(first, n), n)
        blk = b.table[i, t // page]
        touched[blk, :, t % page] = True
        for h in range(hkv):
            a = slice(h * b.g, h * b.g + b.g)
            held = None if was is None else R.slots(was.double().cpu().numpy(), b.table[i], h, n)
            want, bound = R.weigh(q[i, :, a], lse[i, :, a], b.rows_of(i, h)[0], n, min(first, n), held, n_new, decay)
            assert (np.abs(got[blk, h, t % page] - want) <= bound).all(), (i, h)
            fresh = (t >= n - n_new) | (not old)
            assert (p[blk, h, t % page] == np.where(fresh, t + 11 * i, -7)).all()
    assert (got[~touched] == before.double().cpu().numpy()[~touched]).all() and (p[~touched] == -7).all()
    assert b.status.item() == 0


def test_weigh_masked_places_and_rows():
    """Keys behind the end may hold anything; a row whose log-sum-exp is -inf adds nothing; an infinite
    one nothing either; bad blocks are left out and flagged."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    b = Batch([70, 100], 4, 1, 32, rows=2, seed=5).attend()
    b.k[int(b.table[0, 2]), :, 6:] = float("nan")
    b.lse[0, 0, 1], b.lse[0, 1, 2] = -float("inf"), float("inf")
    out = torch.zeros(b.cfg.num_blocks, 1, 32, device="cuda")
    bad = b.table.copy()
    bad[1, 1] = -1
    B.locks_weigh(b.cfg, b.q, b.lse, b.k, b.ints(bad), b.seq_lens, None, out, status=b.status)
    lse = b.lse.double().cpu().numpy()
    lse[np.isinf(lse)] = -np.inf                              # (either way a row without weight)
    for i, n in ((0, 70), (1, 100)):
        want, bound = R.weigh(b.q[i].double().cpu().numpy(), lse[i], b.rows_of(i, 0)[0], n, 0, None, 0, 1.0)
        got = R.slots(out.double().cpu().numpy(), b.table[i], 0, n)
        if i == 1:
            assert (got[32:64] == 0).all()
            want[32:64] = 0
        assert (np.abs(got - want) <= bound).all()
    assert b.status.item() == B.LOCKS_DEV_BAD_BLOCK_ID


# --------------------------------------------------------------------------
# eviction
# --------------------------------------------------------------------------
EVICT = [
    # lens, hkv, page, budget, recent, fixed, distinct weights (0: all), odd values every so many
    ([20], 1, 16, 5, 0, None, 0, 0),
    ([20, 33, 0], 2, 16, 5, 2, [0, 4, 0], 0, 0),
    ([9, 10], 1, 64, 1, 1, None, 2, 0),
    ([300, 299], 2, 64, 298, 10, [1, 0], 3, 0),                # one and one: found as least keys
    ([308, 305, 304], 1, 32, 300, 100, None, 1, 0),            # up to eight
    ([309, 320], 2, 32, 300, 300, None, 4, 5),                 # more
    ([1000, 999, 31], 1, 32, 500, 100, [0, 600, 31], 3, 0),
    ([5000], 1, 64, 1000, 0, None, 2, 7),
    ([40000], 2, 16, 3000, 500, [7], 5, 0),                    # clusters
    ([40000], 2, 16, 39995, 500, [6], 0, 0),
    ([30001], 1, 64, 15000, 500, None, 1, 0),
    ([700000], 1, 16, 5000, 100, [3], 50, 0),                  # chunks of the keys
    ([30000], 8, 16, 4000, 300, [5], 0, 0),                    # eight heads on one large cluster each
]


@pytest.mark.parametrize("lens,hkv,page,budget,recent,fixed,distinct,odd", EVICT)
def test_evict(lens, hkv, page, budget, recent, fixed, distinct, odd):
    import torch
    from sparse_paged_kv_gb300 import binding as B
    seed = len(lens) + budget
    rng = np.random.default_rng(seed)
    batch, pages = len(lens), max(-(-n // page) for n in lens)
    blocks = batch * pages + 2
    table = rng.permutation(blocks)[:batch * pages].reshape(batch, pages).astype(np.int32)
    w = rng.random((blocks, hkv, page), np.float32)
    if distinct:
        w = np.floor(w * distinct)
    if odd:
        for i, x in enumerate((np.nan, -0.0, np.inf, -np.inf, -3.0)):
            w.reshape(-1)[i::odd] = x
    pos = rng.integers(0, 1000, (blocks, hkv, page)).astype(np.int32)
    gone = rng.integers(0, 500, batch).astype(np.int32)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn(blocks, hkv, page, 128, generator=gen, device="cuda").bfloat16() for _ in "kv")
    kk, vv, ww, pp = k.clone(), v.clone(), w.copy(), pos.copy()
    first = [0] * batch if fixed is None else fixed
    lens_after, gone_after = np.array(lens, np.int32), gone.copy()
    for b, n in enumerate(lens):
        if n - min(first[b], n) > budget:
            lens_after[b], gone_after[b] = first[b] + budget, gone[b] + n - first[b] - budget
        for h in range(hkv):
            holes, movers = R.evict(R.slots(w, table[b], h, n), R.slots(pos, table[b], h, n), n, first[b], int(gone[b]),
                                    budget, recent)
            src, dst = ((table[b, x // page], h, x % page) for x in (movers, holes))
            ww[dst], pp[dst] = w[src], pos[src]
            src, dst = ([torch.from_numpy(np.asarray(x, np.int64)).cuda() if i != 1 else h for i, x in enumerate(y)]
                        for y in (src, dst))
            kk[dst[0], h, dst[2]], vv[dst[0], h, dst[2]] = k[src[0], h, src[2]], v[src[0], h, src[2]]
    cfg = B.LocksConfig(batch=batch, n_q_heads=hkv, n_kv_heads=hkv, head_dim=128, page_size=page, rank=8,
                        max_pages=pages, num_blocks=blocks)
    dev = [torch.from_numpy(x).cuda() for x in (w, pos, np.array(lens, np.int32), gone, table)]
    ws = torch.zeros(B.evict_workspace_bytes(cfg, budget), dtype=torch.uint8, device="cuda")
    status = Batch.ints([0])
    for _ in range(2):                                         # (a second call finds nothing to do)
        B.locks_evict(cfg, budget, recent, k, v, dev[4], dev[2], dev[0], dev[1], dev[3], ws,
                      fixed=None if fixed is None else Batch.ints(fixed), status=status)
        assert dev[2].tolist() == lens_after.tolist() and dev[3].tolist() == gone_after.tolist()
        assert (dev[0].cpu().numpy().view(np.int32) == ww.view(np.int32)).all()
        assert (dev[1].cpu().numpy() == pp).all()
        assert torch.equal(k.view(torch.int16), kk.view(torch.int16))
        assert torch.equal(v.view(torch.int16), vv.view(torch.int16))
    assert status.item() == 0


def test_evict_bad_blocks():
    """A page outside the pool holds the least of all; moves into it are left out and flagged."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    cfg = B.LocksConfig(batch=1, n_q_heads=1, n_kv_heads=1, head_dim=128, page_size=16, rank=8, max_pages=4, num_blocks=4)
    w = torch.arange(64, dtype=torch.float32, device="cuda").view(4, 1, 16)
    pos = torch.arange(64, dtype=torch.int32, device="cuda").view(4, 1, 16)
    k = torch.randn(4, 1, 16, 128, device="cuda").bfloat16()
    before = k.clone()
    lens, gone, status = Batch.ints([64]), Batch.ints([0]), Batch.ints([0])
    for budget in (40, 60):                                    # many and few
        ws = torch.zeros(B.evict_workspace_bytes(cfg, budget), dtype=torch.uint8, device="cuda")
        lens.fill_(64), gone.zero_(), status.zero_()
        B.locks_evict(cfg, budget, 0, k, k.clone(), Batch.ints([[0, 9, 2, 3]]), lens, w, pos, gone, ws, status=status)
        assert status.item() == B.LOCKS_DEV_BAD_BLOCK_ID and lens.item() == budget and gone.item() == 64 - budget
        assert torch.equal(k[1], before[1])                    # (a block that nobody named)


def test_evict_workspace_of_several_budgets():
    """One workspace for falling budgets, on a stream of its own: each call finds its counters ready."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    batch, hkv, page, pages = 3, 2, 32, 10
    cfg = B.LocksConfig(batch=batch, n_q_heads=hkv, n_kv_heads=hkv, head_dim=128, page_size=page, rank=8,
                        max_pages=pages, num_blocks=batch * pages)
    gen = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn(batch * pages, hkv, page, 128, generator=gen, device="cuda").bfloat16() for _ in "kv")
    w = torch.rand(batch * pages, hkv, page, generator=gen, device="cuda")
    heaviest = w.view(batch, pages, hkv, page).transpose(1, 2).reshape(batch, hkv, -1).sort(-1, descending=True).values
    pos = torch.arange(pages * page, dtype=torch.int32, device="cuda").view(pages, 1, page).repeat(batch, hkv, 1)
    table = torch.arange(batch * pages, dtype=torch.int32, device="cuda").view(batch, pages)
    lens, gone, status = Batch.ints([pages * page] * batch), Batch.ints([0] * batch), Batch.ints([0])
    budgets = (200, 197, 60, 59, 1)
    ws = torch.zeros(max(B.evict_workspace_bytes(cfg, n) for n in budgets), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for n in budgets:
        B.locks_evict(cfg, n, 0, k, v, table, lens, w, pos, gone, ws, status=status, stream=side)
        side.synchronize()
        assert lens.tolist() == [n] * batch and gone.tolist() == [pages * page - n] * batch
        left = w.view(batch, pages, hkv, page).transpose(1, 2).reshape(batch, hkv, -1)[..., :n]
        assert torch.equal(left.sort(-1, descending=True).values, heaviest[..., :n])
    assert status.item() == 0


def test_prefix_on_two_streams_at_once():
    """Two batches on two streams, a workspace each: the bits of the calls one after the other."""
    import torch
    batches = [Batch([900 + 7 * i for i in range(12)], 16, 2, 32, [0, 6, 12], [20, 3], rows=2, seed=seed)
               for seed in (1, 2)]
    want = []
    for b in batches:
        b.attend()
        want.append((b.out.clone(), b.lse.clone()))
        b.out.zero_(), b.lse.zero_()
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    for _ in range(4):
        for b, s in zip(batches, streams):
            with torch.cuda.stream(s):
                b.attend()
    torch.cuda.synchronize()
    for b, (out, lse) in zip(batches, want):
        assert torch.equal(b.out, out) and torch.equal(b.lse, lse) and b.status.item() == 0


# --------------------------------------------------------------------------
# together
# --------------------------------------------------------------------------
def cache(lens, prefix, budget, recent, rows=4, decay=1.0, seed=0, page=16, hq=8, hkv=2, pages=24):
    import torch
    from sparse_paged_kv_gb300 import binding as B
    from sparse_paged_kv_gb300 import runtime
    rng = np.random.default_rng(seed)
    batch = len(lens)
    table = rng.permutation(batch * pages).reshape(batch, pages)
    table[:, :prefix] = table[0, :prefix]
    cfg = B.LocksConfig(batch=batch, n_q_heads=hq, n_kv_heads=hkv, head_dim=128, page_size=page, rank=8, max_pages=pages,
                        num_blocks=batch * pages)
    c = runtime.BatchCache(cfg, table, [0, batch], [prefix], budget_tokens=budget, recent_tokens=recent, decay=decay,
                           max_rows=rows)
    gen = torch.Generator().manual_seed(seed)
    for pool in (c.k_cache, c.v_cache):
        pool.copy_(torch.randn(pool.shape, generator=gen).bfloat16())
    c.seq_lens.copy_(Batch.ints(lens))
    return c, gen


def test_run_together_against_reference():
    """A prompt's end, then steps: every output, weight, position and length against the 64-bit forms run on
    what the cache held before each call."""
    import torch
    c, gen = cache([200, 100, 64, 90], 4, 60, 8, decay=0.9)
    page, hkv, g = 16, 2, 4
    table = c.block_table.cpu().numpy()

    def rows(*shape):
        return torch.randn(*shape, 128, generator=gen).bfloat16().cuda()

    def held(pool, b, h, n):
        return R.slots(pool, table[b], h, n)

    def check(q, out, lse, n_new, fresh, state):
        k, v, w, pos, lens, gone = state
        q, out, lse = (x.double().cpu().numpy().reshape(4, -1, 8, 128 if x.dtype == torch.bfloat16 else 1)
                       for x in (q, out, lse))
        lse = lse[..., 0]
        for b in range(4):
            n = int(lens[b])
            for h in range(hkv):
                a = slice(h * g, h * g + g)
                kk, vv = held(k, b, h, n), held(v, b, h, n)
                for r in range(q.shape[1]):
                    m = R.limit(n, q.shape[1], r)
                    o, l, bo, bl = R.attend(q[b, r, a], kk[:m], vv[:m])
                    assert (np.abs(out[b, r, a] - o) <= bo).all() and (np.abs(lse[b, r, a] - l) <= bl).all()
                want, bound = R.weigh(q[b, :, a], lse[b, :, a], kk, n, min(64, n), None if fresh else held(w, b, h, n),
                                      n_new, 0.9)
                # what was kept carries its weight along: the tokens now in the cache are among the old
                now_n = int(c.seq_lens[b])
                now_pos = held(c.positions.cpu().numpy(), b, h, now_n)[64:]
                now_w = held(c.weights.double().cpu().numpy(), b, h, now_n)[64:]
                old_pos = held(pos, b, h, n)[64:].copy()
                if fresh:
                    old_pos = np.arange(64, n)
                elif n_new:
                    old_pos[-n_new:] = np.arange(n - n_new, n) + gone[b]
                at = {p: i for i, p in enumerate(old_pos)}
                assert len(set(now_pos)) == now_pos.size and all(p in at for p in now_pos)
                idx = np.array([at[p] for p in now_pos], int)
                assert (np.abs(now_w - want[idx]) <= bound[idx]).all()
                if n - 64 > 60:
                    assert now_n == 124
                    lost = np.setdiff1d(np.arange(want.size), idx)
                    newest = old_pos >= n + gone[b] - 8
                    assert newest[idx].sum() == 8 and not newest[lost].any()
                    keep = idx[~newest[idx]]
                    assert (want[lost].max() <= want[keep].min() + bound.max() * 2) if lost.size else True
                kept_k = held(c.k_cache.double().cpu().numpy(), b, h, now_n)[64:]
                assert (kept_k == kk[64:][idx]).all()

    def state():
        return [x.double().cpu().numpy() if x.is_floating_point() else x.cpu().numpy().copy()
                for x in (c.k_cache, c.v_cache, c.weights, c.positions, c.seq_lens, c.evicted)]

    before = state()
    q = rows(4, 4, 8)
    out, lse = c.observe(q)
    check(q, out, lse, 0, True, before)
    for step in range(5):
        q, k, v = rows(4, 8), rows(4, 2), rows(4, 2)
        nxt = c.next_positions().tolist()
        c.append(k, v)
        before = state()
        c.attend(q)
        c.weigh(q, c.out_lse, 1)
        c.evict()
        check(q, c.out, c.out_lse, 1, False, before)
        assert c.next_positions().tolist() == [x + 1 for x in nxt]
    assert c.seq_lens.tolist() == [124, 105, 69, 95] and c.status.item() == 0
    # the shared pages are as they were
    assert (state()[0][table[0, :4]] == before[0][table[0, :4]]).all()


def test_captured_step_is_the_step():
    import torch
    runs = []
    for graph in (False, True):
        c, gen = cache([200, 130, 64], 4, 60, 8, seed=3)
        q, k, v = (torch.zeros(3, h, 128, dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2))
        c.observe(torch.randn(3, 4, 8, 128, generator=gen).bfloat16().cuda())
        held = [x.clone() for x in (c.k_cache, c.weights, c.positions, c.seq_lens, c.evicted, c.status)]
        step = c.capture_step(q, k, v).replay if graph else lambda: c.step(q, k, v)
        for x, y in zip(held, (c.k_cache, c.weights, c.positions, c.seq_lens, c.evicted, c.status)):
            assert torch.equal(x, y)                          # (a capture leaves the cache as it was)
        outs = []
        for _ in range(70):
            for x in (q, k, v):
                x.copy_(torch.randn(x.shape, generator=gen).bfloat16())
            step()
            outs.append(c.out.clone())
        runs.append(outs + [c.k_cache, c.v_cache, c.weights, c.positions, c.seq_lens, c.evicted, c.status])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_example():
    path = os.path.join(ROOT, "examples", "shared_prefix.py")
    spec = importlib.util.spec_from_file_location("shared_prefix", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    c = mod.main(batch=2, prefix_tokens=128, prompt=90, steps=20, budget=64)
    assert c.seq_lens.tolist() == [192, 192] and c.next_positions().tolist() == [238, 238]
