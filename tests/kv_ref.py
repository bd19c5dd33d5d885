"""The quantised cache in NumPy: its record layout, quantiser, rotation and
attention in 64 bits, written from the header's description.  Test
infrastructure only."""
import math

import numpy as np

F8, I8, I4 = 0, 1, 2
FORMATS = {"f8": F8, "i8": I8, "i4": I4}
D = 128
f32 = np.float32

# every e4m3 byte's value (the two NaN codes as NaN)
_b = np.arange(256)
_e, _m = (_b >> 3) & 15, _b & 7
E4M3 = np.where(_e > 0, (8 + _m) * 2.0 ** (_e - 10.0), _m * 2.0 ** -9) * np.where(_b & 128, -1.0, 1.0)
E4M3[[127, 255]] = np.nan
_POS = E4M3[:127]


def e4m3_bits(x):
    """The e4m3 byte nearest to x (ties to even, saturating)."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.searchsorted(_POS, a)                      # first value >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[np.minimum(hi, 126)] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (pick | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def row_bytes(fmt):
    return 64 if fmt == I4 else 128


def record_bytes(fmt, B):
    return B * (row_bytes(fmt) + (8 if fmt == I4 else 4))


def quantise(x, fmt):
    """Rows x [..., 128] (float32) -> (codes int [..., 128] (F8: e4m3 bytes), group bytes
    [..., 4] or None, scale float32 [...]), every step in float32."""
    x = np.asarray(x, f32)
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(-1, keepdims=True)
        bad = ~np.isfinite(x).all(-1, keepdims=True)
        dead = bad | (amax < f32(2.0 ** -96))
        top = {F8: 448.0, I8: 127.0, I4: 7.0 * 448.0}[fmt]
        scale = (amax * f32(1.0 / top)).astype(f32)
        y = np.where(dead, f32(0), x * (f32(1) / scale)).astype(f32)
        groups = None
        if fmt == F8:
            code = e4m3_bits(y).astype(np.int64)
        elif fmt == I8:
            code = np.clip(np.rint(y), -127, 127).astype(np.int64)
        else:
            yg = y.reshape(*y.shape[:-1], 4, 32)
            groups = e4m3_bits((np.abs(yg).max(-1) * f32(1.0 / 7.0)).astype(f32))
            g = E4M3[groups].astype(f32)[..., None]
            code = np.where(g > 0, np.clip(np.rint(yg * (f32(1) / g)), -7, 7), 0)
            code = code.reshape(y.shape).astype(np.int64)
        scale = np.where(bad, f32(np.nan), np.where(dead, f32(0), scale))[..., 0].astype(f32)
    return code, groups, scale


def values(code, groups, scale, fmt):
    """float64 values of codes, group bytes and scales."""
    if fmt == F8:
        v = E4M3[code]
    elif fmt == I8:
        v = code.astype(np.float64)
    else:
        v = code * np.repeat(E4M3[groups], 32, axis=-1)
    return v * scale.astype(np.float64)[..., None]


def byte_of(fmt, B):
    """Byte offset in a record of (row, dim) [B][128] (I4: of its nibble's byte)."""
    r, d = np.arange(B)[:, None], np.arange(D)[None]
    if fmt == I4:
        return r * 64 + 16 * ((d // 32) ^ ((r >> 1) & 3)) + (d % 32) // 2
    return r * 128 + 16 * ((d // 16) ^ (r & 7)) + d % 16


def pack(code, groups, scale, fmt):
    """Records uint8 [..., record_bytes] of pages of B rows [..., B, 128]."""
    B = code.shape[-2]
    rec = np.zeros((*code.shape[:-2], record_bytes(fmt, B)), np.uint8)
    at = byte_of(fmt, B)
    if fmt == I4:
        n = (code + 8).astype(np.uint8)
        rec[..., at[:, 0::2]] = n[..., 0::2] | (n[..., 1::2] << 4)
        rec[..., B * 64:B * 68] = groups.reshape(*rec.shape[:-1], 4 * B)
    else:
        rec[..., at] = code + (128 if fmt == I8 else 0)
    rec[..., -4 * B:] = np.ascontiguousarray(scale, f32).view(np.uint8)
    return rec


def unpack(rec, fmt, B):
    """(codes, group bytes or None, scales) of records [..., record_bytes]."""
    code = rec[..., byte_of(fmt, B)].astype(np.int64)
    groups = None
    if fmt == I4:
        code = ((code >> (4 * (np.arange(D) % 2))) & 15) - 8
        groups = rec[..., B * 64:B * 68].reshape(*rec.shape[:-1], B, 4)
    elif fmt == I8:
        code = code - 128
    return code, groups, np.ascontiguousarray(rec[..., -4 * B:]).view(f32)


def read(rec, fmt, B):
    """float32 values (one rounding: code * group is exact) of records."""
    code, groups, scale = unpack(rec, fmt, B)
    v = values(code, groups, np.ones_like(scale), fmt).astype(f32)
    return v * scale[..., None]


def frequencies(r, theta=10000.0, scaling="none", factor=1.0, low_freq_factor=1.0,
                high_freq_factor=4.0, original_positions=8192.0, beta_fast=32.0, beta_slow=1.0):
    """(radians per position [r / 2], factor on cos and sin)."""
    if scaling == "ntk":
        theta = theta * factor ** (r / (r - 2))
    w = np.array([theta ** (-2.0 * i / r) for i in range(r // 2)])
    if scaling == "linear":
        w = w / factor
    if scaling == "llama3":
        out = []
        for x in w:
            wave = 2 * math.pi / x
            if wave < original_positions / high_freq_factor:
                out.append(x)
            elif wave > original_positions / low_freq_factor:
                out.append(x / factor)
            else:
                z = (original_positions / wave - low_freq_factor) / (high_freq_factor - low_freq_factor)
                out.append((1 - z) * x / factor + z * x)
        w = np.array(out)
    if scaling == "yarn":
        def dim(turns):
            return r * math.log(original_positions / (turns * 2 * math.pi)) / (2 * math.log(theta))
        a, b = max(math.floor(dim(beta_fast)), 0), min(math.ceil(dim(beta_slow)), r - 1)
        z = np.clip((np.arange(r // 2) - a) / max(b - a, 1e-3), 0, 1)
        return w / factor * z + w * (1 - z), 0.1 * math.log(factor) + 1.0
    return w, 1.0


def rotate(x, pos, w, mscale, layout, inverse=False):
    """x [tokens][heads][dim] in float64."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    a = np.asarray(pos, np.float64)[:, None] * w
    c, s = (np.cos(a) * mscale)[:, None], (np.sin(a) * mscale)[:, None]
    if inverse:
        s = -s
    n = len(w)
    i = np.arange(n)
    u, v = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    y[..., u] = x[..., u] * c - x[..., v] * s
    y[..., v] = x[..., v] * c + x[..., u] * s
    return y


def attend(q, k, v):
    """One KV head: q [G][128], k, v [n][128] in float64 -> (out, lse, bounds), where bounds
    holds what the tolerances need: the sums of p|v|, and the largest sum of |q k| / sqrt(d)."""
    n = len(k)
    G = len(q)
    if n == 0:
        return np.zeros((G, D)), np.full(G, -np.inf), (np.zeros((G, D)), np.zeros(G), 0.0)
    z = q @ k.T / math.sqrt(D)
    m = z.max(-1, keepdims=True)
    p = np.exp(z - m)
    total = p.sum(-1, keepdims=True)
    size = (np.abs(q) @ np.abs(k).T / math.sqrt(D)).max(-1)
    return p @ v / total, (m + np.log(total))[:, 0], (p @ np.abs(v) / total, size, np.abs(v).max())
