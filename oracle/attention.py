"""64-bit definitions of the attention and key-value cache operators (include/bitnet.h), one row and one page at a
time, with the error bounds that the tests hold the kernels to."""
from __future__ import annotations

import numpy as np

U_BF16 = 2.0 ** -8      # half a step of bf16, relative
U_SUM = 2.0 ** -23      # one addition in fp32 that may truncate


def row(q, keys, vals, scale):
    """One query row [D] over its visible keys [n, D] and values [n, D] (float64).  Returns (y, lse, tol_y, tol_lse).

    The bounds follow the kernels' arithmetic: products of bf16 values are exact in fp32; a score is a sum of D of them
    (D additions) scaled once, so it is off by at most ds = (D + 4) U_SUM scale sum|q k|; a weight exp(s - m) carries
    that, 2^-22 of the exponential and, in the product with the values, half a bf16 step; sums over n keys add n U_SUM;
    numerator and denominator both carry it.  The output is rounded to bf16 once."""
    n, D = keys.shape
    if n == 0:
        return np.zeros(D), -np.inf, np.zeros(D), 0.0
    with np.errstate(invalid="ignore", over="ignore"):
        s = keys @ q * scale
        top = np.max(s)
        if top == -np.inf:
            return np.zeros(D), -np.inf, np.zeros(D), 0.0
        p = np.exp(s - top)
        total = p.sum()
        y = (p[:, None] * vals).sum(0) / total
        lse = top + np.log(total)
        fin = np.isfinite(s)
        mag = (np.abs(keys[fin]) @ np.abs(q)).max(initial=0.0) * scale
        ds = (D + 4) * U_SUM * mag
        spread = (p[:, None] * np.abs(vals)).sum(0) / total
        rel = ds + 2.0 ** -22 + (n + 8) * U_SUM
        tol_y = spread * (U_BF16 + 2.0 * rel) * 1.01 + np.abs(y) * U_BF16 + 2.0 ** -126
        tol_lse = ds + (n + 16) * U_SUM + np.abs(lse) * 2.0 ** -22
    return y, lse, tol_y, tol_lse


def prompt(q, k, v, cu_q, cu_k, scale, rows=None):
    """Packed causal attention.  q [Tq,Hq,D], k and v [Tk,Hkv,D] float64; `rows` limits the rows of each sequence that
    are computed (a set).  Yields (token, head, y, lse, tol_y, tol_lse)."""
    group = q.shape[1] // k.shape[1]
    for i in range(len(cu_q) - 1):
        ql, kl = cu_q[i + 1] - cu_q[i], cu_k[i + 1] - cu_k[i]
        for r in range(ql):
            if rows is not None and r not in rows and r - ql not in rows:
                continue
            n = max(0, min(kl, r + kl - ql + 1))
            for h in range(q.shape[1]):
                yield (cu_q[i] + r, h) + row(q[cu_q[i] + r, h], k[cu_k[i]:cu_k[i] + n, h // group],
                                             v[cu_k[i]:cu_k[i] + n, h // group], scale)


class Pool:
    """The page tables on the host, entry by entry."""

    def __init__(self, n_slots, max_pages, n_pages, page_size):
        self.table = np.full((n_slots, max_pages), -1, np.int32)
        self.lens = np.zeros(n_slots, np.int32)
        self.refs = np.zeros(n_pages, np.int32)
        self.page_size = page_size

    def _free(self):
        return [p for p in range(len(self.refs)) if self.refs[p] == 0]

    def _pages(self, tokens):
        return -(-tokens // self.page_size)

    def extend(self, add, slots=None):
        """0, the number of lacking pages, or -1; nothing changes unless 0."""
        slots = list(range(len(add))) if slots is None else list(slots)
        limit = self.table.shape[1] * self.page_size
        if len(set(slots)) < len(slots) or any(s < 0 or s >= len(self.lens) for s in slots):
            return -1
        if any(a < 0 or self.lens[s] + a > limit for s, a in zip(slots, add)):
            return -1
        want = [(s, e) for s, a in zip(slots, add)
                for e in range(self._pages(self.lens[s]), self._pages(self.lens[s] + a)) if self.table[s, e] < 0]
        free = self._free()
        if len(free) < len(want):
            return len(want) - len(free)
        for (s, e), p in zip(want, free):
            self.table[s, e] = p
            self.refs[p] = 1
        for s, a in zip(slots, add):
            self.lens[s] += a
        return 0

    def fork(self, parents, children):
        """(status as extend, copies)"""
        ok = lambda s: 0 <= s < len(self.lens)  # noqa: E731
        if not all(map(ok, parents)) or not all(map(ok, children)):
            return -1, []
        if len(set(children)) < len(children) or set(children) & set(parents) or any(self.lens[c] for c in children):
            return -1, []
        held = [self.table[p, :self._pages(self.lens[p])] for p in parents]
        if any(((t < 0) | (t >= len(self.refs))).any() for t in held):
            return -1, []
        need = [p for p in parents if self.lens[p] % self.page_size]
        free = self._free()
        if len(free) < len(need):
            return len(need) - len(free), []
        pairs = []
        for p, c in zip(parents, children):
            full = self.lens[p] // self.page_size
            self.table[c] = -1
            self.table[c, :full] = self.table[p, :full]
            for page in self.table[p, :full]:
                self.refs[page] += 1
            if self.lens[p] % self.page_size:
                page = free.pop(0)
                self.refs[page] = 1
                self.table[c, full] = page
                pairs.append((int(self.table[p, full]), page))
            self.lens[c] = self.lens[p]
        return 0, pairs

    def free(self, slots):
        for s in slots:
            for e in range(self.table.shape[1]):
                if self.table[s, e] >= 0:
                    self.refs[self.table[s, e]] -= 1
                    self.table[s, e] = -1
            self.lens[s] = 0

    def compact(self):
        """(pages in use, copies)"""
        live = int((self.refs > 0).sum())
        pairs = []
        for p in range(live, len(self.refs)):
            if self.refs[p] > 0:
                dst = self._free()[0]
                pairs.append((p, dst))
                self.table[self.table == p] = dst
                self.refs[dst], self.refs[p] = self.refs[p], 0
        return live, pairs
