"""Plain 64-bit forms of the operators of a batch that shares prefixes and lives within a budget, and
the bounds within which float32 kernels with bf16 weights and outputs have to be of them."""
import numpy as np

D = 128
HALF_BF16 = 2.0 ** -8          # half a step of bf16, relative to the value
EPS32 = 2.0 ** -24             # half a step of float32


def slots(pool, table_row, h, n):
    """The first n slots of a sequence in KV head h of a pool [blocks][heads][page]..."""
    page = pool.shape[2]
    return pool[table_row[:-(-n // page)], h].reshape(-1, *pool.shape[3:])[:n]


def limit(n, rows, r):
    """Slots that query row r of a sequence of n tokens sees."""
    return max(0, n - rows + r + 1)


def logit_error(q, k):
    """Bound of the error of q.k / sqrt(d) summed in float32 (any order), per query row."""
    return (D + 4) * EPS32 * float((np.abs(q) @ np.abs(k).T).max(initial=0.0)) / np.sqrt(D)


def attend(q, k, v):
    """(out, lse, bound of out, bound of lse) of queries [g][d] over keys and values [n][d].

    A logit z is off by e (its sum), and by a few roundings of z log2(e) in the exponent; a weight is
    rounded to bf16; the sums of weights and of products are float32.  With weights w and outputs o,
    sum w (1 + x) v / sum w (1 + x) is off by at most max|x| * sum w |v - o| (1 + max|x|)."""
    if k.shape[0] == 0:
        g = q.shape[0]
        return np.zeros((g, D)), np.full(g, -np.inf), np.zeros((g, D)), np.zeros(g)
    z = q @ k.T / np.sqrt(D)
    m = z.max(-1, keepdims=True)
    w = np.exp(z - m)
    total = w.sum(-1, keepdims=True)
    w /= total
    out, lse = w @ v, (m + np.log(total))[:, 0]
    # exponent: the logit's sum, then z * log2 e - m in one rounding each, the constant's, the
    # exponential's own 2 units, and as much again where parts are joined (twice)
    x = logit_error(q, k) + 3 * 2 * EPS32 * 1.45 * (np.abs(z).max() + 8) + 4 * 2 * EPS32
    sums = 2 * EPS32 * (64 + k.shape[0] / 64 + 700)          # chains of additions: a row's columns, stages, parts
    spread = np.einsum("gn,gnd->gd", w, np.abs(v[None] - out[:, None])) if k.shape[0] * q.shape[0] <= 1 << 16 else \
        np.stack([wi @ np.abs(v - oi) for wi, oi in zip(w, out)])
    rel = HALF_BF16 * 1.01 + x
    size = w @ np.abs(v)
    bound = rel * 1.02 * spread + 2 * sums * size + HALF_BF16 * (np.abs(out) + rel * spread + 2 * sums * size) + 2.0 ** -130
    return out, lse, bound, x + 2 * sums + 2 * EPS32 * np.abs(lse) + 2 * EPS32 * 8 + np.zeros_like(lse)


def weigh(q, lse, k, n, first, old, n_new, decay):
    """(weights, bounds) of slots first .. n - 1 that queries [rows][g][d] with lse [rows][g] give;
    old: weights [n] or None."""
    rows = q.shape[0]
    t = np.arange(first, n)
    total, bound = np.zeros(n - first), np.zeros(n - first)
    for r in range(rows):
        seen = t < limit(n, rows, r)
        z = q[r] @ k[first:].T / np.sqrt(D)
        with np.errstate(invalid="ignore", over="ignore"):
            p = np.where(np.isneginf(lse[r])[:, None], 0.0, np.exp(z - lse[r][:, None]))
        size = np.abs(z) + np.abs(np.where(np.isfinite(lse[r]), lse[r], 0.0))[:, None] + 1
        # the logit's sum, and roundings of z log2 e, of lse log2 e, of their difference, of the exponential
        e = logit_error(q[r], k[first:]) + 5 * 2 * EPS32 * 1.45 * size
        total += np.where(seen, p.sum(0), 0.0)
        bound += np.where(seen, (p * e * 1.01).sum(0), 0.0)
    bound += total * 2 * EPS32 * (rows * q.shape[1] + 4) + 2.0 ** -120
    if old is not None:
        kept = np.where(t < n - n_new, old[first:] * decay, 0.0)
        total += kept
        bound += 2 * EPS32 * (np.abs(kept) + np.abs(total))
    return total, bound


def evict(weights, positions, n, first, gone, budget, recent):
    """(holes, movers) of one head: slots [lists ascending]; weights, positions of the n slots."""
    first = min(first, n)
    if n - first <= budget:
        return np.zeros(0, int), np.zeros(0, int)
    t = np.arange(first, n)
    # order: recent ones, NaN, numbers; ties to the lower slot
    rank = np.where(np.isnan(weights), 1, 0)
    rank = np.where(positions.astype(np.int64) >= n + gone - recent, 2, rank)[first:]
    w = np.where(rank > 0, 0.0, np.nan_to_num(weights[first:], nan=0.0, posinf=np.inf, neginf=-np.inf))
    best = np.sort(t[np.lexsort((t, -w, -rank))[:budget]])
    return np.setdiff1d(np.arange(first, first + budget), best), best[best >= first + budget]
