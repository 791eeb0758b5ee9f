"""Shared helpers of the paged-cache tests: a plain model of the bookkeeping (Python
lists and numpy, written from the rules in include/eta.h) and attention outputs in 64
bits with the error bounds that the tests hold the kernels to."""
from __future__ import annotations

import math

import numpy as np

from oracle import eta_oracle as O

NO_PAGE, BAD_ROW, BAD_LENGTH, BAD_BLOCK = 0x20, 0x40, 0x8, 0x4


class PageModel:
    """The bookkeeping of a paged cache, one call at a time; `status` collects the bits."""

    def __init__(self, B, blk, max_pages, n_pages):
        self.B, self.blk, self.max_pages, self.n_pages = B, blk, max_pages, n_pages
        self.len = [0] * B
        self.pages = [[] for _ in range(B)]
        self.ref = [0] * n_pages
        self.free_stack = list(range(n_pages - 1, -1, -1))
        self.stale = list(self.free_stack)     # what lies behind the top of the stack
        self.status = 0
        self.moves = []                        # (from page, to page, tokens) of the last call
        self.tokens = {}                       # (page, slot) -> token number of an append

    def _nb(self, n):
        return -(-n // self.blk)

    def _pop(self):
        p = self.free_stack.pop()
        self.ref[p] = 1
        return p

    def _push(self, p):
        self.free_stack.append(p)
        self.stale[len(self.free_stack) - 1] = p

    def append(self, cu, n_new):
        if any(not 0 <= a <= b <= n_new for a, b in zip(cu, cu[1:])):
            self.status |= BAD_LENGTH
            return
        taken = 0
        n_free = len(self.free_stack)
        plan = []
        for b in range(self.B):
            c0, c1 = cu[b], cu[b + 1]
            n = c1 - c0
            if self.len[b] + n > self.max_pages * self.blk:
                self.status |= BAD_LENGTH
                continue
            if n == 0:
                continue
            if self.len[b] % self.blk and self.ref[self.pages[b][-1]] != 1:
                self.status |= BAD_ROW
                continue
            need = self._nb(self.len[b] + n) - self._nb(self.len[b])
            taken += need
            if need and taken > n_free:
                self.status |= NO_PAGE
                continue
            plan.append((b, c0, n, need))
        for b, c0, n, need in plan:
            self.pages[b] += [self._pop() for _ in range(need)]
            for i in range(n):
                pos = self.len[b] + i
                self.tokens[self.pages[b][pos // self.blk], pos % self.blk] = c0 + i
            self.len[b] += n

    def fork(self, src, dst):
        self.moves = []
        len0, pages0 = list(self.len), [list(p) for p in self.pages]
        seen, taken, n_free = set(), 0, len(self.free_stack)
        for f, t in zip(src, dst):
            if not (0 <= f < self.B and 0 <= t < self.B) or t in seen or len0[t] != 0:
                self.status |= BAD_ROW
                if 0 <= t < self.B:
                    seen.add(t)
                continue
            seen.add(t)
            full, part = divmod(len0[f], self.blk)
            taken += part > 0
            if part and taken > n_free:
                self.status |= NO_PAGE
                continue
            self.pages[t] = pages0[f][:full]
            for p in self.pages[t]:
                self.ref[p] += 1
            if part:
                new = self._pop()
                self.moves.append((pages0[f][full], new, part))
                self.pages[t] = self.pages[t] + [new]
            self.len[t] = len0[f]

    def free(self, rows):
        gone = []
        for b in rows:
            if not 0 <= b < self.B:
                self.status |= BAD_ROW
                continue
            for p in self.pages[b]:
                self.ref[p] -= 1
                if self.ref[p] == 0:
                    gone.append(p)
            self.pages[b], self.len[b] = [], 0
        for p in sorted(gone, reverse=True):
            self._push(p)

    def compact(self):
        n_live = self.n_pages - len(self.free_stack)
        holes = [p for p in range(n_live) if self.ref[p] == 0]
        movers = [p for p in range(n_live, self.n_pages) if self.ref[p] > 0]
        to = dict(zip(movers, holes))
        self.moves = [(f, t, self.blk) for f, t in to.items()]
        for f, t in to.items():
            self.ref[t], self.ref[f] = self.ref[f], 0
        self.pages = [[to.get(p, p) for p in row] for row in self.pages]
        n = len(self.free_stack)
        self.free_stack = [self.n_pages - 1 - k for k in range(n)]
        self.stale[:n] = self.free_stack

    def check(self, cache):
        """The device's bookkeeping, all of it."""
        assert cache.lengths.tolist() == self.len
        table = np.full((self.B, self.max_pages), -1)
        for b, row in enumerate(self.pages):
            table[b, :len(row)] = row
        np.testing.assert_array_equal(cache.table.cpu().numpy(), table)
        assert cache.ref.tolist() == self.ref
        assert int(cache.n_free) == len(self.free_stack)
        assert cache.free_list.tolist() == self.stale
        assert self.stale[:len(self.free_stack)] == self.free_stack
        assert sorted(self.free_stack) == [p for p in range(self.n_pages) if self.ref[p] == 0]


def rows_of(K, table, lengths, blk):
    """Pools [n_pages, Hkv, blk, d] -> every row's own tokens, a list of [len, Hkv, d]."""
    out = []
    for b, n in enumerate(lengths):
        pages = table[b, :-(-n // blk)]
        out.append(K[pages].transpose(0, 2, 1, 3).reshape(-1, K.shape[1], K.shape[3])[:n])
    return out


def attention(q, k, v, keep, tau, T, scale, p_eps, out_eps, gate_eps=2.0 ** -20):
    """One query head in 64 bits over the tokens `keep` (index array) of one row, and how
    far a kernel may be from it: (o, lse, bound of |o|'s error [d], bound of lse's error).
    tau None: no gate.

    q.k is an fp32 sum of d exact products: off by at most d * 2^-24 * sum |q_i k_i|, and
    the scale and the base-2 argument of the exponential round twice more: with
    A = max scale * sum |q_i k_i|, |ds| <= (d + 4) 2^-24 A; a soft gate multiplies that by
    at most its slope, 1 + 0.28 |s| / T, and its sigmoid is off by gate_eps: 2^-20 from an
    exponential and a division, 2^-10 from the approximate tanh.  A weight is then off by
    e_w = |ds'| + 2^-21 (approximate exponentials, two of them through a rescaled maximum),
    its rounding adds p_eps, and sums of n terms in tiles of 128 add (128 + n / 128) 2^-24.  Numerator and denominator err together:
    |do| <= 2 (e_w + p_eps + e_sum) * sum p |v| / sum p, plus the output's own rounding;
    |dlse| <= e_w + e_sum + 2^-23 |lse|.
    """
    d = q.shape[0]
    if keep.size == 0:
        return np.zeros(d), -math.inf, np.zeros(d), 0.0, False
    K, V = k[keep], v[keep]
    s = scale * (K @ q)
    A = float((scale * (np.abs(K) @ np.abs(q))).max())
    ds = (d + 4) * 2.0 ** -24 * A
    tie = False
    if tau is None:
        x = s
    else:
        x = O.gate(s, tau, T)
        if T == 0.0:
            tie = bool(np.any(np.abs(s - tau) <= 2 * ds + 2.0 ** -22 * abs(tau)))
        else:
            ds = ds * (1 + 0.28 * float(np.abs(s).max()) / T) + gate_eps * float(
                np.abs(s).max())
    m = x.max()
    p = np.exp(x - m)
    L = p.sum()
    o = p @ V / L
    lse = m + math.log(L)
    e_w = ds + 2.0 ** -21
    e_sum = (128 + keep.size / 128) * 2.0 ** -24
    mean_abs = p @ np.abs(V) / L
    tol_o = 2 * (e_w + p_eps + e_sum) * mean_abs + out_eps * np.abs(o) + 1e-30
    return o, lse, tol_o, e_w + e_sum + 2.0 ** -23 * abs(lse), tie
