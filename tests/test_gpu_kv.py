"""The quantised cache on the GPU against its NumPy reference in 64 bits:
rotary positions, writes, reads and decode attention, over formats, page
sizes, head groups, lengths, masks, strides and streams."""
import math

import numpy as np
import pytest

import workloads as W
from tests import kv_ref as R

pytestmark = pytest.mark.gpu

BF16_HALF = 2.0 ** -8            # half a step of bf16, relative
HALF_STEP = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11, "float32": 2.0 ** -24}
F16_LEAST = 2.0 ** -25           # half a step of f16 below its normal range, absolute
# one rotated element from its float32 inputs: the angle is exact to 2^-25 half-turns (9.4e-8
# rad), sine and cosine to 2 units of 2^-24, and mscale, the two products and their sum round
# once each: below 8 x 2^-24 of |u| + |v|
ROT = 2.0 ** -21


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    from sparse_paged_kv_gb300 import binding, build_lib
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    binding.load_library(build_lib.build())


def _table(rot, **kw):
    from sparse_paged_kv_gb300 import runtime
    return runtime.RopeTable(rot, **kw)


# --------------------------------------------------------------------------
# locks_rope
# --------------------------------------------------------------------------
def rope_tol(x, pos, w, mscale, layout, half):
    """Tolerance of each rotated element, and the exact result."""
    y = R.rotate(x, pos, w, mscale, layout)
    n = len(w)
    size = np.zeros_like(y)
    i = np.arange(n)
    u, v = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    size[..., u] = size[..., v] = mscale * (np.abs(x[..., u]) + np.abs(x[..., v]))
    # the reference's own angle, position * w in 64 bits, is off by 2^-52 of it
    ang = 2.0 ** -52 * np.abs(np.asarray(pos, np.float64)).max()
    return y, np.abs(y) * half + size * (ROT + ang)


ROPE_CASES = [
    # tokens, heads, head_dim, rotary, layout, scaling
    (1, 1, 2, 2, "half", {}), (5, 3, 6, 6, "half", {}), (7, 2, 64, 64, "half", {}),
    (33, 5, 128, 128, "half", dict(scaling="llama3", theta=500000.0, factor=8.0)),
    (9, 4, 128, 128, "interleaved", dict(scaling="yarn", theta=1e6, factor=4.0, original_positions=32768.0)),
    (130, 3, 80, 40, "interleaved", dict(scaling="linear", factor=4.0)),
    (17, 3, 80, 32, "half", dict(scaling="ntk", factor=8.0)), (4, 2, 72, 72, "half", {}),
    (3, 9, 256, 256, "interleaved", {}), (2, 3, 512, 510, "half", {}), (600, 40, 128, 64, "half", {}),
    (21, 2, 24, 8, "interleaved", {}),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("case", ROPE_CASES, ids=lambda c: "x".join(map(str, c[:5])))
def test_rope(case, dtype):
    import torch
    from sparse_paged_kv_gb300 import binding as B
    tokens, heads, dim, rot, layout, kw = case
    gen = torch.Generator().manual_seed(tokens * 7 + heads * 5 + dim + rot)
    x = torch.randn(tokens, heads, dim, generator=gen).to(getattr(torch, dtype))
    pos = torch.randint(0, 1 << 20, (tokens,), generator=gen).int()
    pos[0] = 0
    w, m = R.frequencies(rot, **kw)
    want, tol = rope_tol(x.double().numpy(), pos.numpy(), w, m, layout, HALF_STEP[dtype])
    tol += F16_LEAST if dtype == "float16" else 0.0
    table = _table(rot, layout=layout, **kw)
    xd, pd = x.cuda(), pos.cuda()
    out = torch.full_like(xd, float("nan"))
    B.locks_rope(table, xd, pd, out)
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all()
    assert np.array_equal(got[..., rot:], x.double().numpy()[..., rot:])    # copied dims, bit for bit
    # in place, the same bits
    B.locks_rope(table, xd, pd, xd)
    assert torch.equal(xd, out)


@pytest.mark.parametrize("pad,off", [(0, 0), (8, 8), (1, 0), (3, 1)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_strides(layout, pad, off):
    """Slices with any token and head stride, aligned and not; nothing else is written."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    tokens, heads, dim, rot = 19, 3, 64, 48
    gen = torch.Generator().manual_seed(3)
    big = torch.randn(tokens, heads + 2, dim + pad + off, generator=gen).bfloat16().cuda()
    x = big[:, 1:1 + heads, off:off + dim]
    pos = torch.arange(tokens).int().cuda() * 1000 - 5000            # negative ones too
    w, m = R.frequencies(rot)
    want, tol = rope_tol(x.double().cpu().numpy(), pos.cpu().numpy(), w, m, layout, BF16_HALF)
    keep = big.clone()
    out = torch.zeros(heads, tokens, dim + pad, dtype=torch.bfloat16, device="cuda").transpose(0, 1)[..., :dim]
    B.locks_rope(_table(rot, layout=layout), x, pos, out)
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    assert torch.equal(big, keep)
    B.locks_rope(_table(rot, layout=layout), x, pos, x)
    assert torch.equal(x, out)
    keep[:, 1:1 + heads, off:off + dim] = out
    assert torch.equal(big, keep)


@pytest.mark.parametrize("pos", [2 ** 31 - 1, -2 ** 31, 123456789])
def test_rope_far_positions(pos):
    import torch
    from sparse_paged_kv_gb300 import binding as B
    x = torch.randn(1, 2, 128, generator=torch.Generator().manual_seed(1))
    w, m = R.frequencies(128)
    want, tol = rope_tol(x.double().numpy(), np.array([pos]), w, m, "half", HALF_STEP["float32"])
    # w itself has 53 bits in both: another 2^-53 of the angle
    out = torch.empty_like(x, device="cuda")
    B.locks_rope(_table(128), x.cuda(), torch.tensor([pos], dtype=torch.int32).cuda(), out)
    assert (np.abs(out.double().cpu().numpy() - want) <= tol + 2.0 ** -52 * abs(pos) * np.abs(x.numpy()).max()).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,rot", [(64, 48), (80, 40), (10, 6)])
def test_rope_inverse_is_the_gradient(layout, dim, rot):
    """Against the formula's transpose, and against differences of the forward call."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    kw = dict(scaling="yarn", theta=1e4, factor=4.0, original_positions=64.0)
    table = _table(rot, layout=layout, **kw)
    w, m = R.frequencies(rot, **kw)
    gen = torch.Generator().manual_seed(11)
    tokens, heads = 6, 2
    pos = torch.randint(0, 5000, (tokens,), generator=gen).int()
    gy = torch.randn(tokens, heads, dim, generator=gen)
    got = torch.empty_like(gy, device="cuda")
    B.locks_rope(table, gy.cuda(), pos.cuda(), got, inverse=True)
    got = got.double().cpu().numpy()
    want = R.rotate(gy.numpy(), pos.numpy(), w, m, layout, inverse=True)
    tol = 2.0 ** -24 * np.abs(want) + 2 * m * np.abs(gy.numpy()).max() * ROT
    assert (np.abs(got - want) <= tol).all()
    # differences: the map is linear, so a step of 1 along each dim gives the Jacobian's columns
    x = torch.randn(tokens, heads, dim, generator=gen).cuda()
    base, out = torch.empty_like(x), torch.empty_like(x)
    B.locks_rope(table, x, pos.cuda(), base)
    grad = np.zeros((tokens, heads, dim))
    for e in range(dim):
        step = x.clone()
        step[..., e] += 1.0
        B.locks_rope(table, step, pos.cuda(), out)
        moved = (step - x).double().cpu().numpy()[..., e]
        d = (out.double() - base.double()).cpu().numpy() / moved[..., None]
        grad[..., e] = (d * gy.double().numpy()).sum(-1)
    # each difference of two outputs of size up to 6: their roundings, times the sum over dims
    assert np.abs(grad - got).max() <= dim * np.abs(gy.numpy()).max() * 12 * m * (ROT + 2.0 ** -23)


# --------------------------------------------------------------------------
# locks_kv_write, locks_kv_read
# --------------------------------------------------------------------------
def make_cfg(fmt, page, batch, hq, hkv, max_pages, blocks):
    from sparse_paged_kv_gb300 import binding as B
    return B.LocksKvConfig(batch=batch, n_q_heads=hq, n_kv_heads=hkv, head_dim=128, page_size=page,
                           max_pages=max_pages, num_blocks=blocks, kv_dtype=fmt)


def bf16(a):
    import torch
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16()


FMTS = sorted(R.FORMATS.items())


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("name,fmt", FMTS)
def test_write_without_rotation_is_the_definition_bit_for_bit(name, fmt, page):
    """Ragged tokens, padding, odd rows; every byte outside the written rows keeps its value."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    hq, hkv, batch, max_pages, blocks = 6, 2, 3, 5, 17
    cfg = make_cfg(fmt, page, batch, hq, hkv, max_pages, blocks)
    rng = np.random.default_rng(page * 10 + fmt)
    table = rng.permutation(blocks)[:batch * max_pages].reshape(batch, max_pages).astype(np.int32)
    where = [(0, t) for t in range(3, 2 * page + 5)] + [(1, 0)] + [(2, 5 * page - 1)] + [(-1, 7)]
    order = rng.permutation(len(where))
    seq = np.array([where[i][0] for i in order], np.int32)
    pos = np.array([where[i][1] for i in order], np.int32)
    n = len(where)
    raw = rng.standard_normal((n, hq + 2 * hkv, 128)) * np.exp(rng.standard_normal((n, 1, 1)) * 3)
    raw[0] = 0
    raw[1, hq:] *= 1e-30                                  # below the smallest row that is kept
    raw[2, hq:] *= 1e33
    raw[3, hq, 100] = np.inf
    raw[4, hq + 1, 0] = np.nan
    raw[5, hq + 2, 127] = -np.inf
    qkv = bf16(raw).cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    rec = R.record_bytes(fmt, page)
    kp, vp = (torch.full((blocks, hkv, rec), 0xAB, dtype=torch.uint8, device="cuda") for _ in "kv")
    q_out = torch.full((n, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([page, 5, 1], dtype=torch.int32).cuda()
    done = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    B.locks_kv_write(cfg, k, v, dev(pos), kp, vp, dev(table), token_seq=dev(seq), q=q, q_out=q_out,
                     seq_lens=lens, completed=done, status=status)
    assert status.item() == 0
    assert lens.tolist() == [2 * page + 5, 5, 5 * page]
    pad = seq < 0
    assert torch.equal(q_out.cpu()[torch.from_numpy(~pad)].view(torch.int16),
                       q.cpu()[torch.from_numpy(~pad)].contiguous().view(torch.int16))
    assert (q_out.cpu()[torch.from_numpy(pad)] == 7.0).all()
    want_done = [table[s, p // page] if s >= 0 and (p + 1) % page == 0 else -1 for s, p in zip(seq, pos)]
    assert done.tolist() == [int(x) for x in want_done] and sum(x >= 0 for x in want_done) >= 3
    for pool, x in ((kp, k), (vp, v)):
        codes, groups, scales = R.quantise(x.float().cpu().numpy(), fmt)
        want = np.full((blocks, hkv, rec), 0xAB, np.uint8)
        mine = np.zeros((blocks, hkv, rec), bool)
        for i in range(n):
            if seq[i] < 0:
                continue
            blk, slot = table[seq[i], pos[i] // page], pos[i] % page
            sel = np.zeros((1, page), bool)
            sel[0, slot] = True
            one = R.pack(np.broadcast_to(codes[i][:, None], (hkv, page, 128)),
                         None if groups is None else np.broadcast_to(groups[i][:, None], (hkv, page, 4)),
                         np.broadcast_to(scales[i][:, None], (hkv, page)), fmt)
            at = np.zeros(rec, bool)
            at[R.byte_of(fmt, page)[slot]] = True
            at[rec - 4 * page + 4 * slot:rec - 4 * page + 4 * slot + 4] = True
            if fmt == R.I4:
                at[page * 64 + 4 * slot:page * 64 + 4 * slot + 4] = True
            want[blk][:, at] = one[:, at]
            mine[blk][:, at] = True
        got = pool.cpu().numpy()
        nan = np.zeros_like(mine)                          # a NaN scale's payload is free
        sc = np.ascontiguousarray(want[..., -4 * page:]).view(np.float32)
        nan[..., -4 * page:] = np.repeat(np.isnan(sc), 4, axis=-1) & mine[..., -4 * page:]
        assert np.array_equal(got[~nan], want[~nan])
        assert np.isnan(np.ascontiguousarray(got[..., -4 * page:]).view(np.float32)
                        [np.isnan(sc) & mine[..., -4 * page:].reshape(*sc.shape, 4).all(-1)]).all()


@pytest.mark.parametrize("layout,rot,kw", [
    ("half", 128, dict(scaling="llama3", theta=500000.0, factor=8.0)), ("half", 64, {}),
    ("interleaved", 128, {}), ("half", 96, {}), ("interleaved", 48, dict(scaling="linear", factor=2.0)),
    ("half", 16, {})])
@pytest.mark.parametrize("name,fmt", FMTS)
def test_write_with_rotation(name, fmt, layout, rot, kw):
    """Queries within bf16 rounding; keys within half a step of their codes."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    page, hq, hkv, batch, max_pages = 32, 7, 1, 2, 8
    blocks = batch * max_pages
    cfg = make_cfg(fmt, page, batch, hq, hkv, max_pages, blocks)
    gen = torch.Generator().manual_seed(rot + fmt)
    n = 70
    qkv = torch.randn(n, hq + 2, 128, generator=gen).bfloat16().cuda()
    pos = torch.cat([torch.arange(35), torch.arange(100, 135)]).int()
    seq = torch.cat([torch.zeros(35), torch.ones(35)]).int()
    table = torch.arange(blocks - 1, -1, -1).int().reshape(batch, max_pages)
    rec = R.record_bytes(fmt, page)
    kp, vp = (torch.zeros(blocks, hkv, rec, dtype=torch.uint8, device="cuda") for _ in "kv")
    q_out = torch.empty(n, hq, 128, dtype=torch.bfloat16, device="cuda")
    B.locks_kv_write(cfg, qkv[:, hq:hq + 1], qkv[:, hq + 1:], pos.cuda(), kp, vp, table.cuda(),
                     token_seq=seq.cuda(), rope=_table(rot, layout=layout, **kw), q=qkv[:, :hq], q_out=q_out)
    w, m = R.frequencies(rot, **kw)
    x = qkv.double().cpu().numpy()
    want, tol = rope_tol(x, pos.numpy(), w, m, layout, BF16_HALF)
    assert (np.abs(q_out.double().cpu().numpy() - want[:, :hq]) <= tol[:, :hq]).all()
    blk = table[seq.long(), (pos // page).long()].numpy()
    slot = (pos % page).numpy()
    k = R.read(kp.cpu().numpy(), fmt, page)[blk, 0, slot].astype(np.float64)
    v = R.read(vp.cpu().numpy(), fmt, page)[blk, 0, slot].astype(np.float64)
    kx, vx = want[:, hq], x[:, hq + 1]
    vcode = R.quantise(vx.astype(np.float32), fmt)
    assert np.array_equal(v, (R.values(vcode[0], vcode[1], np.ones_like(vcode[2]), fmt).astype(np.float32)
                              * vcode[2][..., None]).astype(np.float64))
    amax = np.abs(kx).max(-1, keepdims=True)
    err = (np.abs(x[:, hq]).max() * 2 * m) * ROT         # of the rotated key itself
    if fmt == R.F8:
        half = np.maximum(np.abs(kx) * 2.0 ** -4, amax / 448 * 2.0 ** -10)
    elif fmt == R.I8:
        half = np.broadcast_to(amax / 254, kx.shape)
    else:
        g = kx.reshape(n, 4, 32)
        gm = np.abs(g).max(-1, keepdims=True)
        # the e4m3 scale of a group is within 2^-4 of gm / 7: half a step, and what clipping loses
        half = np.maximum(gm / 14 * (1 + 2.0 ** -4), np.abs(g) - gm * (1 - 2.0 ** -4)).reshape(n, 128)
        half = np.maximum(half, amax / 3136 * 2.0 ** -10 * 7)        # scales below e4m3's normal range
    assert (np.abs(k - kx) <= half * (1 + 2.0 ** -20) + 4 * err).all()


def test_write_rotates_the_query_in_place_and_on_another_stream():
    import torch
    from sparse_paged_kv_gb300 import binding as B
    cfg = make_cfg(R.F8, 64, 4, 8, 2, 2, 8)
    gen = torch.Generator().manual_seed(2)
    qkv = torch.randn(4, 12, 128, generator=gen).bfloat16().cuda()
    q = qkv[:, :8].contiguous()
    pos = torch.tensor([0, 63, 64, 127], dtype=torch.int32).cuda()
    table = torch.arange(8).int().reshape(4, 2).cuda()
    t = _table(128)
    pools = [torch.zeros(8, 2, R.record_bytes(R.F8, 64), dtype=torch.uint8, device="cuda") for _ in range(4)]
    q_out = torch.empty_like(q)
    B.locks_kv_write(cfg, qkv[:, 8:10], qkv[:, 10:], pos, pools[0], pools[1], table, rope=t, q=q, q_out=q_out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.locks_kv_write(cfg, qkv[:, 8:10], qkv[:, 10:], pos, pools[2], pools[3], table, rope=t, q=q, q_out=q,
                     stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(q, q_out) and torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    assert int(pools[0].count_nonzero()) > 0


def test_write_flags_what_it_cannot_place():
    """Positions and sequences out of range, blocks outside the pool: nothing is written but the query."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    from sparse_paged_kv_gb300.binding import (LOCKS_DEV_BAD_BLOCK_ID, LOCKS_DEV_BAD_PAGE_ID,
                                               LOCKS_DEV_BAD_SEQ_LEN)
    cfg = make_cfg(R.I4, 16, 2, 2, 1, 2, 3)
    table = torch.tensor([[0, 3], [-1, 2]], dtype=torch.int32).cuda()
    for seq, pos, flag in ((0, 32, LOCKS_DEV_BAD_SEQ_LEN), (0, -1, LOCKS_DEV_BAD_SEQ_LEN),
                           (1, 2 ** 31 - 1, LOCKS_DEV_BAD_SEQ_LEN), (2, 0, LOCKS_DEV_BAD_PAGE_ID),
                           (0, 16, LOCKS_DEV_BAD_BLOCK_ID), (1, 15, LOCKS_DEV_BAD_BLOCK_ID),
                           (1, 16, 0)):
        x = torch.randn(1, 4, 128).bfloat16().cuda()
        kp, vp = (torch.zeros(3, 1, R.record_bytes(R.I4, 16), dtype=torch.uint8, device="cuda") for _ in "kv")
        lens = torch.tensor([4, 4], dtype=torch.int32).cuda()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        done = torch.full((1,), -9, dtype=torch.int32, device="cuda")
        q_out = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device="cuda")
        one = lambda a: torch.tensor([a], dtype=torch.int32).cuda()  # noqa: E731
        B.locks_kv_write(cfg, x[:, 2:3], x[:, 3:], one(pos), kp, vp, table, token_seq=one(seq), q=x[:, :2],
                         q_out=q_out, seq_lens=lens, completed=done, status=status)
        assert status.item() == flag, (seq, pos)
        assert torch.equal(q_out, x[:, :2])
        if flag:
            assert not kp.any() and not vp.any() and lens.tolist() == [4, 4] and done.item() == -1
        else:
            assert kp[2].any() and vp[2].any() and lens.tolist() == [4, 17]


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("name,fmt", FMTS)
def test_read(name, fmt, page):
    """Any bytes read as the values they stand for (one float32 product, one rounding to bf16)."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    hkv, blocks = 3, 9
    cfg = make_cfg(fmt, page, 1, 3, hkv, 4, blocks)
    rng = np.random.default_rng(fmt * 100 + page)
    x = rng.standard_normal((2, blocks, hkv, page, 128)).astype(np.float32)
    x[:, 1] *= 1e20
    x[:, 2, 0, 5] = np.inf
    x[:, 3] = 0
    recs = [R.pack(*R.quantise(a, fmt), fmt) for a in x]
    kp, vp = (torch.from_numpy(a).cuda() for a in recs)
    ids = np.array([4, -1, 1, 2, 8, 3, 4, blocks, -5], np.int32)
    outs = [torch.full((len(ids), hkv, page, 128), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    idd = torch.from_numpy(ids).cuda()
    B.locks_kv_read(cfg, kp, vp, idd, outs[0], outs[1], status=status)
    assert status.item() == B.LOCKS_DEV_BAD_BLOCK_ID
    B.locks_kv_read(cfg, kp, None, idd, outs[2], None)
    B.locks_kv_read(cfg, None, vp, idd, None, outs[3])
    for i, rec in ((0, recs[0]), (1, recs[1]), (2, recs[0]), (3, recs[1])):
        got = outs[i].cpu()
        for j, b in enumerate(ids.tolist()):
            if not 0 <= b < blocks:
                assert (got[j] == 3.0).all()
                continue
            want = torch.from_numpy(R.read(rec[b], fmt, page)).bfloat16()
            assert torch.equal(torch.nan_to_num(got[j], nan=12345.0), torch.nan_to_num(want, nan=12345.0))


# --------------------------------------------------------------------------
# locks_kv_decode
# --------------------------------------------------------------------------
def attend_tol(out, lse, bounds, n):
    """Tolerances of a unit's outputs: logits are float32 sums of exact products, off by 2^-18 of
    the sum of |q k| (sixteen partial sums, truncated at 2^-22 each) and 2^-20 for the exponential;
    a weight is rounded to f16 (2^-11, or 2^-31 of the largest where it is tiny), its products
    summed in float32 (2^-16 in all); the result is rounded to bf16."""
    pv, size, vmax = bounds
    delta = (size * 2.0 ** -18 + 2.0 ** -20)[:, None]
    tol = BF16_HALF * np.abs(out) + (2.0 ** -11 + 2 * delta + 2.0 ** -16) * pv + n * 2.0 ** -31 * vmax
    finite = np.where(np.isfinite(lse), np.abs(lse), 0)
    return tol, delta[:, 0] + 2.0 ** -18 + 2.0 ** -22 * finite


class Cache:
    """A quantised cache in NumPy and on the device, unused slots and blocks poisoned."""

    def __init__(self, fmt, page, lens, hq, hkv, seed=0, extra=2, kmul=1.0, vmul=None, headroom=0):
        import torch
        self.fmt, self.page, self.lens, self.hq, self.hkv = fmt, page, list(lens), hq, hkv
        rng = self.rng = np.random.default_rng(seed)
        batch = len(self.lens)
        self.max_pages = max(1, max(-(-n // page) for n in self.lens)) + headroom
        need = sum(-(-n // page) for n in self.lens)
        self.blocks = need + extra
        perm = rng.permutation(self.blocks)
        self.table = np.full((batch, self.max_pages), -1, np.int32)
        self.k, self.v = [], []
        rec = R.record_bytes(fmt, page)
        # poison: codes and scales of all ones bits (an e4m3 NaN, a NaN scale)
        self.pools = [np.full((self.blocks, hkv, rec), 0xFF, np.uint8) for _ in "kv"]
        at = 0
        for b, n in enumerate(self.lens):
            pages = -(-n // page)
            self.table[b, :pages] = perm[at:at + pages]
            at += pages
            pair = []
            for which, pool in enumerate(self.pools):
                x = rng.standard_normal((pages, hkv, page, 128))
                x = x * (kmul if which == 0 else (1.0 if vmul is None else vmul(rng, (pages, hkv, page, 1))))
                x = W.bf16_bits_to_f32(W.f32_to_bf16_bits(x.astype(np.float32)))
                c, g, s = R.quantise(x, fmt)
                full = R.pack(c, g, s, fmt)
                keep = np.broadcast_to((np.arange(pages * page) < n).reshape(pages, 1, page), (pages, hkv, page))
                mask = np.zeros((pages, hkv, rec), bool)
                mask[..., R.byte_of(fmt, page)] = keep[..., None]
                mask[..., -4 * page:] = np.repeat(keep, 4, -1)
                if fmt == R.I4:
                    mask[..., page * 64:page * 68] = np.repeat(keep, 4, -1)
                idx = self.table[b, :pages]
                pool[idx] = np.where(mask, full, pool[idx])
                val = R.values(c, g, s, fmt).transpose(1, 0, 2, 3).reshape(hkv, pages * page, 128)[:, :n]
                pair.append(val)
            self.k.append(pair[0])
            self.v.append(pair[1])
        q = rng.standard_normal((batch, hq, 128)).astype(np.float32)
        self.q = W.bf16_bits_to_f32(W.f32_to_bf16_bits(q))
        self.dev = [torch.from_numpy(p).cuda() for p in self.pools]
        self.cfg = make_cfg(fmt, page, batch, hq, hkv, self.max_pages, self.blocks)

    def run(self, selected=None, window=0, stream=None, ws=None, status=None, lens=None):
        import torch
        from sparse_paged_kv_gb300 import binding as B
        dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        batch = len(self.lens)
        out = torch.full((batch, self.hq, 128), 9.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((batch, self.hq), 9.0, device="cuda")
        if ws is None:
            ws = torch.zeros(B.kv_decode_workspace_bytes(self.cfg), dtype=torch.uint8, device="cuda")
        st = status if status is not None else torch.zeros(1, dtype=torch.int32, device="cuda")
        n = torch.tensor(self.lens if lens is None else lens, dtype=torch.int32).cuda()
        B.locks_kv_decode(self.cfg, bf16(self.q).cuda(), self.dev[0], self.dev[1], dev(self.table), n, out, ws,
                          selected=dev(selected), window=window, out_lse=lse, status=st, stream=stream)
        if status is None:
            assert st.item() == 0, hex(st.item())
        return out, lse

    def check(self, got, selected=None, window=0, skip=lambda b, j: False):
        out, lse = (x.double().cpu().numpy() for x in got)
        G = self.hq // self.hkv
        for b, n in enumerate(self.lens):
            for h in range(self.hkv):
                t = np.arange(n)
                ok = t >= n - window if window else np.ones(n, bool)
                if selected is not None:
                    ok &= np.isin(t // self.page, [j for j in selected[b, h] if j >= 0])
                ok &= ~np.array([skip(b, j) for j in range(-(-n // self.page))], bool)[t // self.page] if n else ok
                a = slice(h * G, h * G + G)
                o, l, bounds = R.attend(self.q[b, a].astype(np.float64), self.k[b][h, ok], self.v[b][h, ok])
                to, tl = attend_tol(o, l, bounds, int(ok.sum()))
                assert (np.abs(out[b, a] - o) <= to).all(), (b, h, np.abs(out[b, a] - o).max())
                if ok.any():
                    assert (np.abs(lse[b, a] - l) <= tl).all(), (b, h, np.abs(lse[b, a] - l).max())
                else:
                    assert (lse[b, a] == -np.inf).all()


LENS = [[1], [0, 3, 0], [15, 16, 17], [63, 64, 65, 1], [200, 0, 31, 128, 129], [1000, 77, 4096 + 37]]


@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("name,fmt", FMTS)
def test_decode(name, fmt, page, lens):
    c = Cache(fmt, page, lens, 8, 2, seed=sum(lens) + page + fmt, headroom=1)
    c.check(c.run())


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (10, 2), (7, 1), (8, 8), (16, 2), (9, 1), (15, 1), (32, 2)])
@pytest.mark.parametrize("name,fmt", FMTS)
def test_decode_groups(name, fmt, hq, hkv):
    c = Cache(fmt, 64, [333, 70], hq, hkv, seed=hq * 3 + fmt)
    c.check(c.run())


@pytest.mark.parametrize("window", [1, 15, 16, 64, 100, 333, 10000])
@pytest.mark.parametrize("page", [16, 64])
def test_decode_window(page, window):
    c = Cache(R.I8, page, [333, 0, 64, 1], 8, 2, seed=window)
    c.check(c.run(window=window), window=window)


@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("name,fmt", FMTS)
def test_decode_selected(name, fmt, page, window):
    """Lists with holes, of one page, of none."""
    c = Cache(fmt, page, [page * 9 + 5, page * 3, 40, 0], 8, 2, seed=page + fmt)
    k = 6
    sel = np.full((4, 2, k), -1, np.int32)
    sel[0, 0] = [0, 2, 3, 7, 8, 9]
    sel[0, 1] = [-1, 9, -1, 4, -1, -1]
    sel[1, 0, :2] = [0, 2]
    sel[1, 1, 5] = 1
    sel[2, 0, 0] = 0                                     # [2, 1] and sequence 3: nothing
    c.check(c.run(selected=sel, window=window), selected=sel, window=window)


def test_decode_flags_bad_pages_and_lengths():
    import torch
    from sparse_paged_kv_gb300 import binding as B
    c = Cache(R.F8, 16, [100, 50], 4, 1, seed=3)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    keep = c.table.copy()
    c.table[0, 2], c.table[1, 0] = c.blocks, -7
    got = c.run(status=st)
    assert st.item() == B.LOCKS_DEV_BAD_BLOCK_ID
    c.check(got, skip=lambda b, j: (b, j) in ((0, 2), (1, 0)))
    c.table = keep
    st.zero_()
    sel = np.array([[[0, 99, 3]], [[2 ** 31 - 1, 1, -1]]], np.int32)
    got = c.run(selected=sel, status=st)
    assert st.item() == B.LOCKS_DEV_BAD_PAGE_ID
    c.check(got, selected=sel)
    st.zero_()
    got = c.run(status=st, lens=[c.max_pages * 16 + 1, -3])      # clamped to the table's row; to nothing
    assert st.item() == B.LOCKS_DEV_BAD_SEQ_LEN
    assert (got[1][1] == float("-inf")).all() and (got[0][1] == 0).all()


@pytest.mark.parametrize("name,fmt", FMTS)
def test_decode_sharp_and_flat_logits(name, fmt):
    """One token that takes nearly all the weight over a long flat tail, and large logits."""
    for mul, seed in ((0.01, 1), (8.0, 2), (60.0, 3)):
        c = Cache(fmt, 64, [2000, 130], 8, 2, seed=seed, kmul=mul)
        c.check(c.run())
    c = Cache(fmt, 64, [20000], 4, 1, seed=4, kmul=0.02)
    c.q[:] = c.q[:, :1]                                   # all heads alike, then one key along them
    x = (c.q[0, 0] * 0.9 * 128 ** 0.5 / np.linalg.norm(c.q[0, 0]) ** 2 * 9.0).astype(np.float32)
    code, g, s = R.quantise(x[None], fmt)
    blk, slot = c.table[0, 77 // 64], 77 % 64
    at = R.byte_of(fmt, 64)[slot]
    one = R.pack(np.broadcast_to(code, (64, 128)), None if g is None else np.broadcast_to(g, (64, 4)),
                 np.broadcast_to(s, (64,)), fmt)
    rec = c.pools[0][blk, 0]
    rec[at] = one[at]
    rec[len(rec) - 256 + 4 * slot:len(rec) - 252 + 4 * slot] = one[-256 + 4 * slot:len(one) - 252 + 4 * slot]
    if fmt == R.I4:
        rec[64 * 64 + 4 * slot:64 * 64 + 4 * slot + 4] = one[64 * 64 + 4 * slot:64 * 64 + 4 * slot + 4]
    import torch
    c.dev[0] = torch.from_numpy(c.pools[0]).cuda()
    c.k[0][0, 77] = R.values(code, g, s, fmt)[0]
    c.check(c.run())


@pytest.mark.parametrize("name,fmt", FMTS)
def test_decode_value_scales_of_every_size(name, fmt):
    """Tokens whose values differ by 2^40 in size; small and large queries."""
    c = Cache(fmt, 32, [700, 90], 6, 2, seed=8, vmul=lambda r, s: 2.0 ** r.integers(-20, 20, s))
    c.check(c.run())
    c.q *= 2.0 ** -30
    c.check(c.run())
    c = Cache(fmt, 32, [700, 90], 6, 2, seed=9, kmul=2.0 ** -40)
    c.q *= 2.0 ** 36
    c.check(c.run())


def test_decode_non_finite_rows_are_seen():
    """A row written with a NaN or an infinity makes its unit's output NaN, and only that unit's."""
    c = Cache(R.I8, 16, [100, 60], 4, 2, seed=5)
    import torch
    blk = c.table[0, 2]
    rec = c.pools[0][blk, 1]
    rec[16 * 128 + 4 * 3:16 * 128 + 4 * 3 + 4] = np.frombuffer(np.float32(np.nan).tobytes(), np.uint8)
    c.dev[0] = torch.from_numpy(c.pools[0]).cuda()
    out, lse = c.run()
    assert torch.isnan(out[0, 2:]).all() and torch.isnan(lse[0, 2:]).all()
    assert not torch.isnan(out[0, :2]).any() and not torch.isnan(out[1]).any()


@pytest.mark.parametrize("name,fmt", FMTS)
def test_decode_is_the_same_every_time(name, fmt):
    """One workspace over many calls, two streams, a graph: the same bits."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    c = Cache(fmt, 64, [5000, 0, 700, 64, 3000], 8, 2, seed=6)
    ws = torch.zeros(B.kv_decode_workspace_bytes(c.cfg), dtype=torch.uint8, device="cuda")
    first = c.run(ws=ws)
    c.check(first)
    for _ in range(5):
        again = c.run(ws=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        again = c.run(ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    q, table = bf16(c.q).cuda(), torch.from_numpy(c.table).cuda()
    n = torch.tensor(c.lens, dtype=torch.int32).cuda()
    out, lse = torch.zeros_like(first[0]), torch.zeros_like(first[1])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        B.locks_kv_decode(c.cfg, q, c.dev[0], c.dev[1], table, n, out, ws, out_lse=lse)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first[0], out) and torch.equal(first[1], lse)


@pytest.mark.parametrize("batch,hkv", [(300, 1), (41, 8), (700, 2)])
def test_decode_many_sequences(batch, hkv):
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, 150, batch)
    lens[5] = 2500
    c = Cache(R.I4, 32, lens.tolist(), hkv * 4, hkv, seed=batch)
    c.check(c.run())


@pytest.mark.parametrize("hq,hkv,page", [(8, 4, 64), (12, 4, 16), (48, 3, 32)])
@pytest.mark.parametrize("name,fmt", FMTS)
def test_decode_long(name, fmt, hq, hkv, page):
    """Enough tokens that every block goes round its ring of stages several times."""
    c = Cache(fmt, page, [40000, 25001, 17], hq, hkv, seed=hq + fmt)
    c.check(c.run())


def test_pools_past_four_gigabytes():
    """Blocks whose byte offsets pass 32 bits: written, read back and attended."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    page, hkv, hq = 64, 8, 8
    rec = R.record_bytes(R.F8, page)
    blocks = (1 << 32) // (rec * hkv) + 40
    cfg = make_cfg(R.F8, page, 1, hq, hkv, 3, blocks)
    kp, vp = (torch.zeros(blocks, hkv, rec, dtype=torch.uint8, device="cuda") for _ in "kv")
    n = 150
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(n, hq + 2 * hkv, 128, generator=gen).bfloat16().cuda()
    table = torch.tensor([[blocks - 1, blocks - 30, blocks - 2]], dtype=torch.int32).cuda()
    pos = torch.arange(n).int().cuda()
    seq = torch.zeros(n).int().cuda()
    B.locks_kv_write(cfg, x[:, hq:hq + hkv], x[:, hq + hkv:], pos, kp, vp, table, token_seq=seq)
    ids = table.flatten().contiguous()
    ko, vo = (torch.zeros(3, hkv, page, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    B.locks_kv_read(cfg, kp, vp, ids, ko, vo)
    ok, ov = (o.transpose(1, 2).reshape(3 * page, hkv, 128)[:n] for o in (ko, vo))
    for got, want in ((ok, x[:, hq:hq + hkv]), (ov, x[:, hq + hkv:])):
        # a code is off by 2^-4 of the value or 2^-10 of the scale, and bf16 rounds once more
        w = want.float()
        tol = torch.maximum(w.abs() * 2.0 ** -4, w.abs().amax(-1, keepdim=True) / 448 * 2.0 ** -10)
        assert ((got.float() - w).abs() <= tol * 1.01 + w.abs() * 2.0 ** -8 * 1.07).all()
    out = torch.empty(1, hq, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(B.kv_decode_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    q = x[:1, :hq].contiguous()
    B.locks_kv_decode(cfg, q, kp, vp, table, torch.tensor([n], dtype=torch.int32).cuda(), out, ws)
    for h in range(hkv):
        k, v = (R.read(pool[ids.long(), h].cpu().numpy(), R.F8, page).astype(np.float64).reshape(-1, 128)[:n]
                for pool in (kp, vp))
        o, l, bounds = R.attend(q[0, h:h + 1].double().cpu().numpy(), k, v)
        tol, _ = attend_tol(o, l, bounds, n)
        assert (np.abs(out[0, h:h + 1].double().cpu().numpy() - o) <= tol).all()


@pytest.mark.parametrize("batch,hkv,n", [(16, 8, 500), (1, 8, 1000), (4, 2, 777), (19, 8, 130), (3, 1, 20000),
                                         (76, 2, 90), (1, 1, 64), (38, 4, 65)])
@pytest.mark.parametrize("name,fmt", FMTS)
def test_decode_equal_lengths(name, fmt, batch, hkv, n):
    """Sequences of one length, whose units are cut in equal parts, with and without empty ones."""
    c = Cache(fmt, 32, [n] * batch, hkv * 2, hkv, seed=n + fmt)
    c.check(c.run())
    lens = [n] * batch
    lens[0] = 0
    lens[batch // 2] = 0
    c = Cache(fmt, 32, lens, hkv * 2, hkv, seed=n)
    c.check(c.run())


def test_decode_shapes_share_a_workspace():
    """Calls of other batches, groups and formats in between change nothing."""
    import torch
    from sparse_paged_kv_gb300 import binding as B
    shapes = [(R.F8, 64, [5000, 300], 8, 2), (R.I4, 16, [700] * 60, 4, 1), (R.I8, 32, [9000], 32, 2),
              (R.I4, 64, [3, 0, 20000], 16, 4)]
    caches = [Cache(f, p, n, hq, hkv, seed=i) for i, (f, p, n, hq, hkv) in enumerate(shapes)]
    ws = torch.zeros(max(B.kv_decode_workspace_bytes(c.cfg) for c in caches), dtype=torch.uint8, device="cuda")
    first = [c.run(ws=ws) for c in caches]
    for c, got in zip(caches, first):
        c.check(got)
    for i in (2, 0, 3, 1, 0, 2, 1, 3, 3, 1):
        again = caches[i].run(ws=ws)
        assert torch.equal(again[0], first[i][0]) and torch.equal(again[1], first[i][1])
