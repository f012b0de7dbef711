"""Attention over packed prompts and over a paged cache, and the cache's pages, in plain fp64 numpy.

Independent of the library: written from the definitions.  ``attend`` also gives
what an error bound needs: the absolute attention sum_j p_j |v_j| and the largest
sum_d |q_d k_d| of each query.
"""

from __future__ import annotations

import numpy as np


def attend(q, k, v, scale, lo, hi):
    """q [i, D], k, v [j, D] (one head); query i sees lo[i] <= j < hi[i].

    Returns o [i, D], lse [i], absolute attention [i, D], largest absolute score sum [i].
    Keys that no query sees are never touched, so they may hold anything.
    """
    q = np.asarray(q, np.float64)
    n, D = q.shape
    o, a = np.zeros((n, D)), np.zeros((n, D))
    lse, big = np.full(n, -np.inf), np.zeros(n)
    for i in range(n):
        kk, vv = np.asarray(k[lo[i]:hi[i]], np.float64), np.asarray(v[lo[i]:hi[i]], np.float64)
        if kk.shape[0] == 0:
            continue
        s = kk @ q[i] * scale
        m = s.max()
        p = np.exp(s - m)
        lse[i] = m + np.log(p.sum())
        p /= p.sum()
        o[i], a[i] = p @ vv, p @ np.abs(vv)
        big[i] = (np.abs(kk) @ np.abs(q[i])).max() * scale
    return o, lse, a, big


def visible(q_len, k_len, causal, window):
    """First and one-past-last key that each query of a sequence sees."""
    lo, hi = [], []
    for i in range(q_len):
        p = k_len - q_len + i
        b = min(k_len, p + 1) if causal else k_len
        a = max(0, p + 1 - window) if window else 0
        lo.append(a)
        hi.append(max(a, b))
    return np.array(lo, int), np.array(hi, int)


def prefill(q, k, v, q_lens, k_lens, scale, causal=True, window=0):
    """q [Tq, H, D], k, v [Tk, Hk, D]; sequences one after the other."""
    H, g = q.shape[1], q.shape[1] // k.shape[1]
    o, a = np.zeros(q.shape), np.zeros(q.shape)
    lse, big = np.full(q.shape[:2], -np.inf), np.zeros(q.shape[:2])
    x = y = 0
    for nq, nk in zip(q_lens, k_lens):
        lo, hi = visible(nq, nk, causal, window)
        for h in range(H):
            r = attend(q[x:x + nq, h], k[y:y + nk, h // g], v[y:y + nk, h // g], scale, lo, hi)
            o[x:x + nq, h], lse[x:x + nq, h], a[x:x + nq, h], big[x:x + nq, h] = r
        x, y = x + nq, y + nk
    return o, lse, a, big


def tolerance(o, a, big, n_keys, head_dim, unit, v_max):
    """Largest error of an output of unit roundoff ``unit`` (2^-8 bf16, 2^-11 fp16) from the steps that round.

    Weights are rounded to the output's type once (unit * a), the result once (unit * |o|).  A score is
    an fp32 dot product: at most (head_dim + 4) roundings of 2^-24 on sum |q k| scale = big; a relative
    error e of every weight moves o by 2 e a.  The sums over n_keys add (n_keys + 8) 2^-24 a each.  Weights
    below the smallest fp16 are lost: n_keys 2^-25 v_max.
    """
    e = (big * (head_dim + 4) * 2.0 ** -24)[..., None]
    e = e + 2.0 ** -20            # the exponential and its argument
    return (unit * np.abs(o) + (unit + 2 * e + 2 * (n_keys + 8) * 2.0 ** -24) * a * (1 + unit)
            + (n_keys * 2.0 ** -25 * v_max if unit < 2.0 ** -10 else 0.0) + 2.0 ** -25)


def lse_tolerance(lse, big, n_keys, head_dim):
    return big * (head_dim + 4) * 2.0 ** -24 + (n_keys + 8) * 2.0 ** -24 + (np.abs(lse) + 8) * 2.0 ** -22


def e4m3_round(x):
    """x to the nearest E4M3 value (ties to even), clamped to +-448; NaN stays."""
    x = np.clip(np.asarray(x, np.float64), -448.0, 448.0)
    m = np.abs(x)
    e = np.maximum(np.floor(np.log2(np.where(m > 0, m, 1.0))), -6)
    step = np.exp2(e - 3)
    return np.round(x / step) * step


class Pages:
    """The page bookkeeping, one request after the other; page contents as one number per page."""

    def __init__(self, n_pages, page_size, max_seqs, max_pages):
        self.ps, self.n_pages, self.max_pages = page_size, n_pages, max_pages
        self.table = np.full((max_seqs, max_pages), -1, np.int32)
        self.length = np.zeros(max_seqs, np.int32)
        self.ref = np.zeros(n_pages, np.int32)
        self.content = np.arange(n_pages, dtype=np.int64)

    def _held(self, s):
        return -(-int(self.length[s]) // self.ps)

    def free(self, seqs):
        for s in seqs:
            for c in range(self._held(s)):
                self.ref[self.table[s, c]] -= 1
                self.table[s, c] = -1
            self.length[s] = 0

    def reserve(self, seqs, n_new):
        """Returns the requests that were not served."""
        failed, free, blocked = [], [int(p) for p in np.flatnonzero(self.ref == 0)], False
        for i, (s, new) in enumerate(zip(seqs, n_new)):
            have, to = self._held(s), -(-(int(self.length[s]) + int(new)) // self.ps)
            if to > self.max_pages:
                failed.append(i)
                continue
            if to > have and (blocked or to - have > len(free)):
                blocked = True
                failed.append(i)
                continue
            for c in range(have, to):
                p = free.pop(0)
                self.table[s, c], self.ref[p] = p, 1
            self.length[s] += new
        return failed

    def fork(self, src, dst):
        failed, free = [], [int(p) for p in np.flatnonzero(self.ref == 0)]
        for i, (s, d) in enumerate(zip(src, dst)):
            L = int(self.length[s])
            if L % self.ps and not free:
                failed.append(i)
                continue
            for c in range(L // self.ps):
                self.table[d, c] = self.table[s, c]
                self.ref[self.table[s, c]] += 1
            if L % self.ps:
                p = free.pop(0)
                self.content[p] = self.content[self.table[s, L // self.ps]]
                self.table[d, L // self.ps], self.ref[p] = p, 1
            self.length[d] = L
        return failed

    def compact(self):
        live = int((self.ref > 0).sum())
        holes = [p for p in range(live) if self.ref[p] == 0]
        movers = [p for p in range(live, self.n_pages) if self.ref[p] > 0]
        for a, b in zip(movers, holes):
            self.table[self.table == a] = b
            self.ref[b], self.ref[a] = self.ref[a], 0
            self.content[b] = self.content[a]
        return live
