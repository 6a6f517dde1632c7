"""The operators over packed batches in plain fp64 numpy and Python lists: attention of
prompts over themselves, pages mapped from lengths, log probabilities.

Nothing here shares code with the GPU path.
"""
from __future__ import annotations

import math

import numpy as np

PAGE = 128


def attend(q, k, v, causal: bool):
    """q [n][H][128], k, v [n][Hkv][128] of one prompt: (out, lse, sum of p |v|)."""
    n, H, hd = q.shape
    g = H // k.shape[1]
    out, mag = np.zeros((n, H, hd)), np.zeros((n, H, hd))
    lse = np.full((n, H), -np.inf)
    for h in range(H):
        for i in range(n):
            end = i + 1 if causal else n
            s = k[:end, h // g] @ q[i, h] / math.sqrt(hd)
            m = s.max()
            p = np.exp(s - m)
            lse[i, h] = m + math.log(p.sum())
            p = p / p.sum()
            out[i, h] = p @ v[:end, h // g]
            mag[i, h] = p @ np.abs(v[:end, h // g])
    return out, lse, mag


class Pages:
    """The page state of a pool as lists; the calls return the status a caller would see."""

    def __init__(self, n_pages, n_seqs, pages_per_seq):
        self.n_pages, self.n_seqs, self.pps = n_pages, n_seqs, pages_per_seq
        self.free = list(range(n_pages - 1, -1, -1))
        self.table = [[-1] * pages_per_seq for _ in range(n_seqs)]
        self.mapped = [0] * n_seqs

    def map(self, seqs, start, counts, n_rows):
        """(offsets, lengths, rows [(seq, pos, slot)], wrong) of a call; wrong holds the kinds of
        failure met."""
        wrong, seen, need, ok = set(), set(), [], []
        offsets, full = [0], False
        for q, s, c in zip(seqs, start, counts):
            good = 0 <= q < self.n_seqs and q not in seen and s >= 0 and c >= 0
            seen.add(q)
            k = 0
            if not good:
                wrong.add("check")
            elif s + c > self.pps * PAGE:
                good = False
                wrong.add("capacity")
            else:
                k = max(0, -(-(s + c) // PAGE) - self.mapped[q])
            ok.append(good)
            need.append(k)
            offsets.append(offsets[-1] + max(c, 0))
        used, lens = 0, []
        for b, (q, s, c) in enumerate(zip(seqs, start, counts)):
            used += need[b]
            full = used > len(self.free)
            if ok[b] and (need[b] and full or offsets[b + 1] > n_rows):
                ok[b] = False
                wrong.add("capacity")
            lens.append(s + c if ok[b] else max(s, 0))
        if offsets[-1] > n_rows:
            wrong.add("capacity")
        for b, q in enumerate(seqs):
            for _ in range(need[b] if ok[b] else 0):
                self.table[q][self.mapped[q]] = self.free.pop()
                self.mapped[q] += 1
        rows = []
        for b, (q, s, c) in enumerate(zip(seqs, start, counts)):
            for j in range(min(max(c, 0), n_rows - len(rows))):
                pos = s + j
                rows.append((q, pos, self.table[q][pos // PAGE] * PAGE + pos % PAGE) if ok[b]
                            else (-1, -1, -1))
        rows = (rows + [(-1, -1, -1)] * n_rows)[:n_rows]
        return [min(o, n_rows) for o in offsets], lens, rows, wrong

    def release(self, seqs, keep):
        wrong, seen, given = set(), set(), []
        for q, k in zip(seqs, keep):
            good = 0 <= q < self.n_seqs and q not in seen and k >= 0
            seen.add(q)
            if not good:
                wrong.add("check")
                continue
            first = -(-k // PAGE)
            while self.mapped[q] > first:
                self.mapped[q] -= 1
            for i in range(first, self.pps):
                if self.table[q][i] >= 0:
                    given.append(self.table[q][i])
                    self.table[q][i] = -1
        self.free += given[::-1]
        return wrong


def logprobs(x, token, top):
    """(log probability, entropy, ids, their log probabilities) of one row.  A NaN or +inf makes
    every number NaN (the ids may be any then)."""
    x = np.asarray(x, dtype=np.float64)
    if not (x < np.inf).all():
        return np.nan, np.nan, [-1] * top, [np.nan] * top
    alive = np.flatnonzero(x > -np.inf)
    if alive.size == 0:
        return -np.inf, 0.0, [-1] * top, [-np.inf] * top
    m = x[alive].max()
    log_s = math.log(np.exp(x[alive] - m).sum())
    lp = (x[alive] - m) - log_s  # (m + log_s would round log_s away beside a huge m)
    entropy = float(-(np.exp(lp) * lp).sum())
    order = alive[np.lexsort((alive, -x[alive]))][:top]
    ids = [int(i) for i in order] + [-1] * (top - order.size)
    vals = [float((x[i] - m) - log_s) for i in order] + [-np.inf] * (top - order.size)
    mine = (x[token] - m) - log_s if 0 <= token < x.size else -np.inf
    return mine, entropy, ids, vals
