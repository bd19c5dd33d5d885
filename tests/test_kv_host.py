"""The quantised cache on the host: sizes, refusals before any launch, the
rotary frequencies, and the reference's own checks (no GPU)."""
import ctypes

import numpy as np
import pytest

from sparse_paged_kv_gb300 import binding as B
from sparse_paged_kv_gb300 import build_lib
from tests import kv_ref as R

FAKE = 0x10000   # never dereferenced: every call below returns before a launch


@pytest.fixture(scope="module")
def lib():
    return B.load_library(build_lib.build())


def cfg(**kw):
    base = dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, page_size=64, max_pages=64,
                num_blocks=200, kv_dtype=B.LOCKS_KV_F8)
    base.update(kw)
    return B.LocksKvConfig(**base)


def test_struct_layouts():
    assert ctypes.sizeof(B.locks_kv_cfg_t) == 8 * 4
    assert ctypes.sizeof(B.locks_rope_spec_t) == 8 + 7 * 8
    assert ctypes.sizeof(B.locks_rope_table_t) == 24


@pytest.mark.parametrize("page", [16, 32, 64])
def test_record_bytes(lib, page):
    for fmt in (R.F8, R.I8, R.I4):
        n = B.kv_record_bytes(cfg(page_size=page, kv_dtype=fmt))
        assert n == R.record_bytes(fmt, page) and n % 16 == 0
        at = R.byte_of(fmt, page)                       # a permutation of the code bytes
        assert sorted(set(at.ravel().tolist())) == list(range(page * R.row_bytes(fmt)))


BAD_CFG = [
    (dict(batch=-1), B.LOCKS_ERR_INVALID_ARG), (dict(n_q_heads=7), B.LOCKS_ERR_INVALID_ARG),
    (dict(n_kv_heads=0), B.LOCKS_ERR_INVALID_ARG), (dict(kv_dtype=3), B.LOCKS_ERR_INVALID_ARG),
    (dict(kv_dtype=-1), B.LOCKS_ERR_INVALID_ARG), (dict(max_pages=0), B.LOCKS_ERR_INVALID_ARG),
    (dict(head_dim=64), B.LOCKS_ERR_UNSUPPORTED), (dict(page_size=8), B.LOCKS_ERR_UNSUPPORTED),
    (dict(page_size=128), B.LOCKS_ERR_UNSUPPORTED), (dict(n_q_heads=34), B.LOCKS_ERR_UNSUPPORTED),
    (dict(max_pages=1 << 24), B.LOCKS_ERR_UNSUPPORTED),
    (dict(num_blocks=1 << 30), B.LOCKS_ERR_UNSUPPORTED),
    (dict(batch=1 << 23), B.LOCKS_ERR_UNSUPPORTED),
]


def _decode(lib, c, k=0, window=0, wsb=1 << 30, **over):
    a = dict(q=FAKE, kp=FAKE, vp=FAKE, bt=FAKE, sl=FAKE, sel=None, out=FAKE, ws=FAKE)
    a.update(over)
    return lib.locks_kv_decode(c.ref, a["q"], a["kp"], a["vp"], a["bt"], a["sl"], a["sel"], k,
                               window, a["out"], None, a["ws"], wsb, None, None)


def _table(rot=128, layout=0, turns=FAKE, mscale=1.0):
    return ctypes.byref(B.locks_rope_table_t(turns, rot, layout, mscale))


def _write(lib, c, n=2, rope=None, ks=256, vs=256, qs=1024, **over):
    a = dict(k=FAKE, v=FAKE, q=None, qo=None, seq=FAKE, pos=FAKE, kp=FAKE, vp=FAKE, bt=FAKE, sl=None)
    a.update(over)
    return lib.locks_kv_write(c.ref, a["k"], ks, a["v"], vs, a["q"], qs, a["qo"], a["seq"], a["pos"],
                              n, rope, a["kp"], a["vp"], a["bt"], a["sl"], None, None, None)


def _read(lib, c, n=2, **over):
    a = dict(kp=FAKE, vp=FAKE, ids=FAKE, ko=FAKE, vo=FAKE)
    a.update(over)
    return lib.locks_kv_read(c.ref, a["kp"], a["vp"], a["ids"], n, a["ko"], a["vo"], None, None)


def _rope(lib, rope, dtype=0, dim=128, n=4, heads=2, x=FAKE, pos=FAKE, out=FAKE):
    return lib.locks_rope(rope, dtype, dim, x, heads * dim, dim, pos, n, heads, out, heads * dim,
                          dim, 0, None)


@pytest.mark.parametrize("over,want", BAD_CFG)
def test_every_call_refuses_a_bad_configuration(lib, over, want):
    c = cfg(**over)
    assert B.kv_record_bytes(c) == 0 and B.kv_decode_workspace_bytes(c) == 0
    assert _decode(lib, c) == _write(lib, c) == _read(lib, c) == want


def test_no_configuration(lib):
    assert lib.locks_kv_record_bytes(None) == 0
    assert lib.locks_kv_decode(None, *([FAKE] * 5), None, 0, 0, FAKE, None, FAKE, 1 << 30, None,
                               None) == B.LOCKS_ERR_INVALID_ARG


def test_decode_refusals(lib):
    c = cfg()
    for name in ("q", "kp", "vp", "bt", "sl", "out", "ws"):
        assert _decode(lib, c, **{name: None}) == B.LOCKS_ERR_INVALID_ARG, name
    for name in ("q", "kp", "vp", "out", "ws"):
        assert _decode(lib, c, **{name: FAKE + 8}) == B.LOCKS_ERR_INVALID_ARG, name
    assert _decode(lib, c, window=-1) == B.LOCKS_ERR_INVALID_ARG
    assert _decode(lib, c, sel=FAKE, k=0) == B.LOCKS_ERR_INVALID_ARG
    assert _decode(lib, c, wsb=B.kv_decode_workspace_bytes(c) - 1) == B.LOCKS_ERR_WORKSPACE
    wide = cfg(batch=1 << 16, max_pages=1 << 20, num_blocks=1 << 20)     # 2^37 stages of 64 tokens
    assert _decode(lib, wide) == B.LOCKS_ERR_UNSUPPORTED
    assert _decode(lib, wide, sel=FAKE, k=1 << 20) == B.LOCKS_ERR_UNSUPPORTED
    assert _decode(lib, c, sel=FAKE, k=1 << 24) == B.LOCKS_ERR_UNSUPPORTED
    assert _decode(lib, cfg(batch=0)) == B.LOCKS_OK


def test_write_refusals(lib):
    c = cfg()
    for name in ("k", "v", "pos", "kp", "vp", "bt"):
        assert _write(lib, c, **{name: None}) == B.LOCKS_ERR_INVALID_ARG, name
    for name in ("k", "v", "kp", "vp"):
        assert _write(lib, c, **{name: FAKE + 2}) == B.LOCKS_ERR_INVALID_ARG, name
    assert _write(lib, c, q=FAKE) == B.LOCKS_ERR_INVALID_ARG                 # q without q_out
    assert _write(lib, c, qo=FAKE) == B.LOCKS_ERR_INVALID_ARG
    assert _write(lib, c, q=FAKE, qo=FAKE, qs=1536) == B.LOCKS_ERR_INVALID_ARG   # in place, strided
    assert _write(lib, c, q=FAKE, qo=FAKE + 16, qs=1028) == B.LOCKS_ERR_INVALID_ARG
    assert _write(lib, c, ks=260) == B.LOCKS_ERR_INVALID_ARG
    assert _write(lib, c, n=-1) == B.LOCKS_ERR_INVALID_ARG
    assert _write(lib, c, seq=None, n=3) == B.LOCKS_ERR_INVALID_ARG          # more tokens than sequences
    assert _write(lib, c, sl=FAKE) == B.LOCKS_ERR_INVALID_ARG                # lengths = positions
    assert _write(lib, c, rope=_table(24)) == B.LOCKS_ERR_UNSUPPORTED
    for bad in (_table(130), _table(0), _table(15), _table(128, 2), _table(turns=None),
                _table(mscale=0.0), _table(mscale=float("nan"))):
        assert _write(lib, c, rope=bad) == B.LOCKS_ERR_INVALID_ARG
    assert _write(lib, c, n=(1 << 30) + 1) == B.LOCKS_ERR_UNSUPPORTED
    assert _write(lib, c, n=0) == B.LOCKS_OK


def test_read_refusals(lib):
    c = cfg()
    assert _read(lib, c, ids=None) == B.LOCKS_ERR_INVALID_ARG
    assert _read(lib, c, ko=None, vo=None) == B.LOCKS_ERR_INVALID_ARG
    assert _read(lib, c, kp=None) == B.LOCKS_ERR_INVALID_ARG
    assert _read(lib, c, vp=None) == B.LOCKS_ERR_INVALID_ARG
    assert _read(lib, c, ko=FAKE + 8) == B.LOCKS_ERR_INVALID_ARG
    assert _read(lib, c, n=-1) == B.LOCKS_ERR_INVALID_ARG
    assert _read(lib, c, n=0) == B.LOCKS_OK


def test_rope_refusals(lib):
    assert _rope(lib, None) == B.LOCKS_ERR_INVALID_ARG
    assert _rope(lib, _table(), dtype=3) == B.LOCKS_ERR_INVALID_ARG
    assert _rope(lib, _table(), dim=126) == B.LOCKS_ERR_INVALID_ARG          # rotary_dim > head_dim
    assert _rope(lib, _table(), dim=129) == B.LOCKS_ERR_INVALID_ARG
    assert _rope(lib, _table(), dim=514) == B.LOCKS_ERR_UNSUPPORTED
    assert _rope(lib, _table(), n=-1) == B.LOCKS_ERR_INVALID_ARG
    for name in ("x", "pos", "out"):
        assert _rope(lib, _table(), **{name: None}) == B.LOCKS_ERR_INVALID_ARG
    assert _rope(lib, _table(), x=FAKE + 1) == B.LOCKS_ERR_INVALID_ARG
    assert _rope(lib, _table(), dtype=2, x=FAKE + 2) == B.LOCKS_ERR_INVALID_ARG
    assert _rope(lib, _table(), n=0) == B.LOCKS_OK


SPECS = [("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
         ("llama3", dict(theta=500000.0, factor=8.0, low_freq_factor=1.0, high_freq_factor=4.0,
                         original_positions=8192.0)),
         ("yarn", dict(theta=1e6, factor=4.0, original_positions=32768.0))]
KINDS = {"none": 0, "linear": 1, "ntk": 2, "llama3": 3, "yarn": 4}


def spec_of(rot, scaling, theta=10000.0, factor=1.0, low_freq_factor=1.0, high_freq_factor=4.0,
            original_positions=8192.0, beta_fast=32.0, beta_slow=1.0):
    return B.locks_rope_spec_t(rot, KINDS[scaling], theta, factor, low_freq_factor,
                               high_freq_factor, original_positions, beta_fast, beta_slow)


@pytest.mark.parametrize("rot", [2, 4, 40, 64, 128, 512])
@pytest.mark.parametrize("scaling,kw", SPECS)
def test_frequencies(lib, rot, scaling, kw):
    if scaling == "ntk" and rot == 2:
        with pytest.raises(B.LocksError):
            B.rope_frequencies(spec_of(rot, scaling, **kw))
        return
    turns, mscale = B.rope_frequencies(spec_of(rot, scaling, **kw))
    w, m = R.frequencies(rot, scaling=scaling, **kw)
    got = np.array([t / 2.0 ** 64 for t in turns]) * 2 * np.pi
    assert len(turns) == rot // 2
    # both in double from the same formula: a few roundings of pow and of the products
    np.testing.assert_allclose(got, w, rtol=64 * 2.0 ** -53, atol=2.0 ** -60)
    assert abs(mscale - m) <= 2.0 ** -24 * m


def test_frequency_refusals(lib):
    for bad in (spec_of(0, "none"), spec_of(3, "none"), spec_of(64, "none", theta=1.0),
                spec_of(64, "none", theta=float("inf")), spec_of(64, "linear", factor=0.5),
                spec_of(64, "linear", factor=float("nan")),
                spec_of(64, "llama3", factor=8.0, high_freq_factor=1.0),
                spec_of(64, "yarn", factor=4.0, original_positions=0.0),
                spec_of(64, "yarn", factor=4.0, beta_slow=0.0)):
        with pytest.raises(B.LocksError):
            B.rope_frequencies(bad)
    bad = spec_of(64, "none")
    bad.scaling = 5
    with pytest.raises(B.LocksError):
        B.rope_frequencies(bad)
    with pytest.raises(B.LocksError) as e:
        B.rope_frequencies(spec_of(514, "none"))
    assert e.value.code == B.LOCKS_ERR_UNSUPPORTED


def test_binding_refuses_wrong_tensors(lib):
    import torch
    c = cfg()
    q = torch.zeros(2, 8, 128)
    with pytest.raises(ValueError):                    # float32 query
        B.locks_kv_decode(c, q, None, None, None, None, None, torch.zeros(1), stream=0)
    with pytest.raises(ValueError):                    # host tensor
        B.locks_kv_write(c, q[:, :2].bfloat16(), q[:, :2].bfloat16(), None, None, None, None, stream=0)
    with pytest.raises(ValueError):                    # heads do not match
        B.locks_kv_write(c, q.bfloat16(), q.bfloat16(), None, None, None, None, stream=0)
    with pytest.raises(ValueError):                    # mixed types
        B.locks_rope(None, q, None, q.bfloat16(), stream=0)


# ---- the reference itself --------------------------------------------------
@pytest.mark.parametrize("fmt", sorted(R.FORMATS.values()))
def test_reference_round_trip(fmt):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((3, 2, 16, 128)).astype(np.float32)
    x[0, 0, 3] = 0
    x[0, 0, 4, 7] = np.inf
    x[0, 0, 5, 9] = np.nan
    x[1, 0, 0] *= 1e-30
    x[1, 0, 1] *= 1e30
    code, groups, scale = R.quantise(x, fmt)
    rec = R.pack(code, groups, scale, fmt)
    c2, g2, s2 = R.unpack(rec, fmt, 16)
    assert np.array_equal(code, c2) and np.array_equal(scale, s2, equal_nan=True)
    assert groups is None or np.array_equal(groups, g2)
    y = R.read(rec, fmt, 16)
    assert np.isnan(y[0, 0, 4]).all() and np.isnan(y[0, 0, 5]).all() and (y[0, 0, 3] == 0).all()
    amax = np.abs(x).max(-1, keepdims=True)
    assert (y[1, 0, 0] == 0).all() and amax[1, 0, 0] < 2.0 ** -96     # below the smallest row kept
    ok = np.isfinite(y).all(-1)
    ok[1, 0, 0] = False
    # half a step of the code (F8: 2^-4 of the value or 2^-10 of the scale; I4: the group's
    # scale is within 2^-4 of a seventh of its largest, so clipping loses at most 2^-4 of it)
    bound = {R.F8: np.maximum(np.abs(x) * 2.0 ** -4, amax / 448 * 2.0 ** -10), R.I8: amax / 254,
             R.I4: amax * 2.0 ** -3}[fmt] * 1.001
    assert (np.abs(y - x) <= bound)[ok].all()


def test_reference_e4m3_rounding():
    import torch
    x = np.concatenate([np.linspace(-460, 460, 20011), np.linspace(-0.02, 0.02, 4001), R._POS,
                        (R._POS[1:] + R._POS[:-1]) / 2]).astype(np.float32)
    t = torch.from_numpy(np.clip(x, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.e4m3_bits(x), t)
