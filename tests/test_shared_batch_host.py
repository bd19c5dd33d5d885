"""The operators of a batch that shares prefixes and lives within a budget, on the host: sizes, refusals
before any launch, the runtime's own checks, and the reference's own checks (no GPU)."""
import copy
import ctypes
import pickle

import numpy as np
import pytest

from sparse_paged_kv_gb300 import binding as B
from sparse_paged_kv_gb300 import build_lib, runtime
from tests import batch_ref as R

FAKE = 0x10000   # never dereferenced: every call below returns before a launch


@pytest.fixture(scope="module")
def lib():
    return B.load_library(build_lib.build())


def cfg(**kw):
    base = dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, page_size=64, rank=8, max_pages=64, num_blocks=200)
    base.update(kw)
    return B.LocksConfig(**base)


BAD_CFG = [
    (dict(batch=-1), B.LOCKS_ERR_INVALID_ARG), (dict(n_q_heads=7), B.LOCKS_ERR_INVALID_ARG),
    (dict(n_kv_heads=0), B.LOCKS_ERR_INVALID_ARG), (dict(max_pages=0), B.LOCKS_ERR_INVALID_ARG),
    (dict(num_blocks=0), B.LOCKS_ERR_INVALID_ARG), (dict(page_size=0), B.LOCKS_ERR_INVALID_ARG),
    (dict(head_dim=64), B.LOCKS_ERR_UNSUPPORTED), (dict(page_size=8), B.LOCKS_ERR_UNSUPPORTED),
    (dict(page_size=128), B.LOCKS_ERR_UNSUPPORTED), (dict(n_q_heads=34), B.LOCKS_ERR_UNSUPPORTED),
    (dict(max_pages=1 << 24), B.LOCKS_ERR_UNSUPPORTED), (dict(num_blocks=1 << 30), B.LOCKS_ERR_UNSUPPORTED),
    (dict(batch=1 << 22), B.LOCKS_ERR_UNSUPPORTED),
]


def prefix(lib, c, rows=1, groups=1, wsb=1 << 40, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, bt=FAKE, sl=FAKE, gs=FAKE, pp=FAKE, out=FAKE, ws=FAKE)
    a.update(over)
    return lib.locks_prefix_decode(c.ref, a["q"], rows, a["k"], a["v"], a["bt"], a["sl"], a["gs"], a["pp"], groups,
                                   a["out"], None, a["ws"], wsb, None, None)


def weigh(lib, c, rows=1, n_new=1, decay=1.0, **over):
    a = dict(q=FAKE, lse=FAKE, k=FAKE, bt=FAKE, sl=FAKE, out=FAKE)
    a.update(over)
    return lib.locks_weigh(c.ref, a["q"], rows, a["lse"], a["k"], a["bt"], a["sl"], None, None, a["out"], n_new,
                           decay, None, None, None, None)


def evict(lib, c, budget=64, recent=0, wsb=1 << 40, **over):
    a = dict(k=FAKE, v=FAKE, bt=FAKE, sl=FAKE, w=FAKE, p=FAKE, ev=FAKE, ws=FAKE)
    a.update(over)
    return lib.locks_evict(c.ref, budget, recent, a["k"], a["v"], a["bt"], a["sl"], None, a["w"], a["p"], a["ev"],
                           a["ws"], wsb, None, None)


@pytest.mark.parametrize("kw,code", BAD_CFG)
def test_refused_configurations(lib, kw, code):
    c = cfg(**kw)
    assert prefix(lib, c) == code and weigh(lib, c) == code and evict(lib, c) == code
    assert B.prefix_workspace_bytes(c, 0) == 0 and B.evict_workspace_bytes(c, 64) == 0


def test_refused_arguments(lib):
    c, bad = cfg(), B.LOCKS_ERR_INVALID_ARG
    for name in ("q", "k", "v", "bt", "sl", "gs", "pp", "out", "ws"):
        assert prefix(lib, c, **{name: None}) == bad, name
    for name in ("q", "k", "v", "out", "ws"):
        assert prefix(lib, c, **{name: FAKE + 8}) == bad, name
    assert prefix(lib, c, rows=0) == bad and prefix(lib, c, rows=-1) == bad
    assert prefix(lib, c, groups=-1) == bad and prefix(lib, c, groups=3) == bad
    assert prefix(lib, c, rows=65) == B.LOCKS_ERR_UNSUPPORTED                  # 2 floor(128 / 4) = 64
    assert prefix(lib, c, wsb=B.prefix_workspace_bytes(c, 1) - 1) == B.LOCKS_ERR_WORKSPACE
    for name in ("q", "lse", "k", "bt", "sl", "out"):
        assert weigh(lib, c, **{name: None}) == bad, name
    for name in ("q", "k"):
        assert weigh(lib, c, **{name: FAKE + 2}) == bad, name
    assert weigh(lib, c, n_new=-1) == bad and weigh(lib, c, decay=-0.5) == bad
    assert weigh(lib, c, decay=float("nan")) == bad and weigh(lib, c, decay=float("inf")) == bad
    assert weigh(lib, c, rows=0) == bad and weigh(lib, c, rows=65) == B.LOCKS_ERR_UNSUPPORTED
    for name in ("k", "v", "bt", "sl", "w", "p", "ev", "ws"):
        assert evict(lib, c, **{name: None}) == bad, name
    for name in ("k", "v", "w", "p", "ws"):
        assert evict(lib, c, **{name: FAKE + 4}) == bad, name
    assert evict(lib, c, budget=0) == bad and evict(lib, c, recent=-1) == bad and evict(lib, c, recent=65) == bad
    assert evict(lib, c, wsb=B.evict_workspace_bytes(c, 64) - 1) == B.LOCKS_ERR_WORKSPACE
    for fn in (lib.locks_prefix_workspace_bytes, lib.locks_evict_workspace_bytes):
        assert fn(None, *([1] * (len(fn.argtypes) - 1))) == 0


def test_nothing_to_do(lib):
    c = cfg(batch=0)
    assert prefix(lib, c, groups=0, q=None, ws=None, wsb=0) == B.LOCKS_OK
    assert weigh(lib, c, q=None) == B.LOCKS_OK and evict(lib, c, ws=None, wsb=0) == B.LOCKS_OK


def test_limits_of_sizes(lib):
    # rows a sequence by the group size, any number of groups up to the batch, counts of the list in an int
    for hq, most in ((2, 256), (6, 84), (8, 64), (16, 32), (32, 16)):
        c = cfg(n_q_heads=hq)
        assert B.prefix_workspace_bytes(c, 2, most) > B.prefix_workspace_bytes(c, 0, 1) > 0
        assert B.prefix_workspace_bytes(c, 0, most + 1) == 0
    assert B.prefix_workspace_bytes(cfg(), 3) == 0
    assert B.prefix_workspace_bytes(cfg(batch=1, max_pages=(1 << 24) - 1, n_q_heads=1, n_kv_heads=1, num_blocks=1 << 24), 0) > 0
    assert B.prefix_workspace_bytes(cfg(batch=1000, max_pages=(1 << 24) - 1, n_q_heads=1, n_kv_heads=1), 0) == 0
    assert prefix(lib, cfg(batch=1000, max_pages=(1 << 24) - 1), groups=0) == B.LOCKS_ERR_UNSUPPORTED
    assert weigh(lib, cfg(batch=1000, max_pages=(1 << 24) - 1)) == B.LOCKS_ERR_UNSUPPORTED
    # a list of moves for every head: at most half of the slots
    c = cfg(max_pages=10)
    assert B.evict_workspace_bytes(c, 1 << 30) == B.evict_workspace_bytes(c, 320) > B.evict_workspace_bytes(c, 10)


def test_configuration_is_copied_and_sent():
    c = cfg(rank=5)
    assert isinstance(c.ref, type(ctypes.byref(ctypes.c_int())))
    for other in (copy.copy(c), copy.deepcopy(c), pickle.loads(pickle.dumps(c))):
        assert other == c and "ref" not in vars(other) and other.ref is not c.ref


def test_binding_checks(lib):
    import torch
    c = cfg()
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    pool = torch.zeros(200, 2, 64, 128, dtype=torch.bfloat16)
    ints = torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(ValueError):                    # one of a pair
        B.locks_prefix_decode(c, q, pool, pool, ints, ints, ints, None, q, ws)
    with pytest.raises(ValueError):                    # neither one row nor several
        B.locks_prefix_decode(c, q[0], pool, pool, ints, ints, None, None, q, ws)
    with pytest.raises(ValueError):                    # shapes and types
        B.locks_prefix_decode(c, q.float(), pool, pool, ints, ints, None, None, q, ws)
    with pytest.raises(ValueError):                    # host tensors
        B.locks_prefix_decode(c, q, pool, pool, ints, ints, None, None, q, ws)
    with pytest.raises(ValueError):
        B.locks_weigh(c, q, ints, pool, ints, ints, None, pool)
    with pytest.raises(ValueError):
        B.locks_evict(c, 64, 0, pool, pool, ints, ints, pool, pool, ints, ws)


def test_batch_cache_checks(lib):
    table = np.arange(8).reshape(2, 4)
    c = cfg(max_pages=4, num_blocks=8)
    shared = table.copy()
    shared[1, :2] = shared[0, :2]

    def make(t=table, **kw):
        return runtime.BatchCache(c, t, device="cpu", **kw)

    ok = make(shared, group_starts=[0, 2], prefix_pages=[2], budget_tokens=64, recent_tokens=8)
    assert ok.fixed.tolist() == [128, 128] and ok.next_positions().tolist() == [0, 0]
    assert make().weights is None
    for kw in (dict(t=table[:1]), dict(group_starts=[0, 2]), dict(group_starts=[0, 2], prefix_pages=[2]),
               dict(group_starts=[0, 1], prefix_pages=[1, 1]), dict(group_starts=[2, 0], prefix_pages=[0]),
               dict(group_starts=[0, 3], prefix_pages=[0]), dict(group_starts=[0, 2], prefix_pages=[5]),
               dict(t=shared, group_starts=[0, 2], prefix_pages=[2], fixed=[100, 128]), dict(fixed=[1]),
               dict(budget_tokens=-1), dict(budget_tokens=8, recent_tokens=9), dict(recent_tokens=1)):
        with pytest.raises(ValueError):
            make(**kw)
    with pytest.raises(B.LocksError):
        make(max_rows=65)
    for call in (lambda x: x.weigh(None, None, 1), lambda x: x.evict()):
        with pytest.raises(ValueError):
            call(make())
    import torch
    with pytest.raises(ValueError):
        ok.attend(torch.zeros(2, 2, 8, 128, dtype=torch.bfloat16))


def test_reference_attention_and_weights():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(3, 128)), rng.normal(size=(40, 128)), rng.normal(size=(40, 128))
    out, lse, bo, bl = R.attend(q, k, v)
    for g in range(3):
        p = np.exp(k @ q[g] / np.sqrt(128))
        assert np.allclose(out[g], p @ v / p.sum()) and np.isclose(lse[g], np.log(p.sum()))
    assert (bo > 0).all() and (bo < 0.05).all() and (bl > 0).all() and (bl < 1e-3).all()
    # the weights a full window gives: each row hands out one
    qr = rng.normal(size=(4, 3, 128))
    lses = np.stack([R.attend(qr[r], k[:R.limit(40, 4, r)], v[:R.limit(40, 4, r)])[1] for r in range(4)])
    w, b = R.weigh(qr, lses, k, 40, 0, None, 0, 1.0)
    assert np.isclose(w.sum(), 12.0) and (b < 1e-4).all()
    w2, _ = R.weigh(qr, lses, k, 40, 10, np.ones(40), 4, 0.5)
    assert np.allclose(w2[:26], w[10:36] + 0.5) and np.allclose(w2[26:], w[36:])


def test_reference_eviction():
    w = np.array([5, 1, 1, 3, np.nan, 0, 9, 1], float)
    pos = np.array([0, 1, 2, 3, 4, 20, 6, 7])
    # budget 4 of the 7 behind slot 0, position 20 recent: NaN, 9, 3 and the recent one stay
    holes, movers = R.evict(w, pos, 8, 1, 13, 4, 1)
    assert holes.tolist() == [1, 2] and movers.tolist() == [5, 6]
    # ties go to the lower slot
    holes, movers = R.evict(np.ones(6), np.zeros(6), 6, 0, 0, 4, 0)
    assert holes.size == movers.size == 0
    assert R.evict(w, pos, 4, 0, 0, 4, 0)[0].size == 0
