"""The 8-bit KV cache operators in plain fp64 numpy: block format, append,
attention with its log-sum-exp, accumulated weights and eviction.

A sequence's cache is held as values: an array [slots][heads][128] that has
already been rounded the way the format rounds, with the exponent of every
block of 16 slots beside it.  Nothing here shares code with the GPU path.
"""
from __future__ import annotations

import numpy as np

SUB, HD = 16, 128
E_MIN, E_MAX = -40, 40


def e4m3_value(code: int) -> float:
    """Value of one e4m3 code (1 sign, 4 exponent bits of bias 7, 3 mantissa bits;
    the all-ones codes are NaN)."""
    ex, ma = (code >> 3) & 15, code & 7
    if code & 127 == 127:
        return float("nan")
    v = ma * 2.0 ** -9 if ex == 0 else (8 + ma) * 2.0 ** (ex - 10)
    return -v if code & 128 else v


E4M3 = np.array([e4m3_value(c) for c in range(256)])


def exponent(block) -> int:
    """Smallest e in [-40, 40] with max |x| <= 448 * 2^e over the finite entries."""
    a = np.abs(np.asarray(block, dtype=np.float64))
    a = a[np.isfinite(a)]
    top = float(a.max()) if a.size else 0.0
    e = E_MIN
    while e < E_MAX and top > 448.0 * 2.0 ** e:
        e += 1
    return e


def round_e4m3(y):
    """Nearest e4m3 value (ties to even, saturating); non-finite -> NaN."""
    y = np.asarray(y, dtype=np.float64)
    a = np.abs(y)
    with np.errstate(divide="ignore", invalid="ignore"):
        ex = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    # log2 may round across a power of two
    ex = np.where(2.0 ** ex > a, ex - 1, ex)
    ex = np.where(2.0 ** (ex + 1) <= a, ex + 1, ex)
    step = 2.0 ** (np.maximum(ex, -6) - 3)
    with np.errstate(invalid="ignore"):
        q = np.clip(np.rint(y / step) * step, -448.0, 448.0)
    return np.where(np.isfinite(y), q, np.nan)


def code_block(x):
    """Values a block [rows][128] is held as, and its exponent."""
    e = exponent(x)
    return round_e4m3(np.asarray(x, dtype=np.float64) / 2.0 ** e) * 2.0 ** e, e


def append(values, exps, start, rows):
    """Writes rows [n][heads][128] behind the first `start` slots; values and
    exps are changed in place.  values [slots][heads][128], exps [slots/16][heads]."""
    n = len(rows)
    if n == 0:
        return
    for blk in range(start // SUB, (start + n - 1) // SUB + 1):
        s0, s1 = blk * SUB, min(blk * SUB + SUB, start + n)
        for h in range(values.shape[1]):
            x = np.concatenate([values[s0:max(s0, min(start, s1)), h],
                                rows[max(s0, start) - start:s1 - start, h]])
            values[s0:s1, h], exps[blk, h] = code_block(x)


def sees(mask, k, n, r, j, anc=None):
    """Does row j of r (n slots in all) see slot k?  anc: set of ints per row."""
    if k >= n:
        return False
    i = k - (n - r)
    if mask == "none" or i < 0:
        return True
    return i <= j if mask == "causal" else i in anc[j]


def visible(mask, n, r, anc=None):
    """[r][n] bool."""
    out = np.zeros((r, max(n, 0)), dtype=bool)
    for j in range(r):
        for k in range(n):
            out[j, k] = sees(mask, k, n, r, j, anc)
    return out


def attend(q, k, v, ok):
    """q [r][H][128], k, v [n][heads][128], ok [r][n] (or [r][heads][n]) ->
    out, lse, and sum p |v| (the scale of rounding errors in p)."""
    r, H = q.shape[:2]
    heads = k.shape[1]
    out, mag = np.zeros((r, H, HD)), np.zeros((r, H, HD))
    lse = np.full((r, H), -np.inf)
    for j in range(r):
        for h in range(H):
            g = h // (H // heads)
            at = np.nonzero(ok[j] if ok.ndim == 2 else ok[j, g])[0]
            if at.size == 0:
                continue
            s = k[at, g] @ q[j, h] / np.sqrt(HD)
            m = s.max()
            lse[j, h] = m + np.log(np.exp(s - m).sum())
            p = np.exp(s - lse[j, h])
            out[j, h] = p @ v[at, g]
            mag[j, h] = p @ np.abs(v[at, g])
    return out, lse, mag


def score(q, k, ok, lse):
    """Weights received: [heads][n]."""
    r, H = q.shape[:2]
    heads = k.shape[1]
    w = np.zeros((heads, k.shape[0]))
    for j in range(r):
        for h in range(H):
            if lse[j, h] == -np.inf:
                continue
            g = h // (H // heads)
            at = np.nonzero(ok[j])[0]
            w[g, at] += np.exp(k[at, g] @ q[j, h] / np.sqrt(HD) - lse[j, h])
    return w


def evict_pick(scores, n, budget, window):
    """Kept slots of one head, ascending (scores [>= n] as stored)."""
    if n <= budget:
        return list(range(n))
    w0 = n - window
    s = [(-np.inf if np.isnan(x) else float(x)) for x in scores[:w0]]
    nan = [np.isnan(x) for x in scores[:w0]]
    best = sorted(range(w0), key=lambda i: (nan[i], -s[i], i))[:budget - window]
    return sorted(best + list(range(w0, n)))
