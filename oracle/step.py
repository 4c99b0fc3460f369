"""Plain forms of what a step takes beside the linears, the norm, the cache and
sampling: the embedding lookup, the norm and rotation of queries and keys, a
linear's epilogue, and the pages under the cache.  numpy and Python lists, one
row, head or page at a time; no code shared with the library.
"""
import numpy as np

from . import exp32, linear, swiglu

F = np.float32


def embed(W, s_row, ids, scale):
    """M x K fp32 rows of the int8 table, zeros for ids outside it."""
    out = np.zeros((len(ids), W.shape[1]), F)
    for m, i in enumerate(ids):
        if 0 <= i < len(W):
            out[m] = (W[i].astype(F) * F(s_row[i])) * F(scale)
    return out


def norm_rope(x, gain, eps, p, inv_freq, magnitude):
    """One head's row in fp64: (y, the size of what each element is summed from)."""
    n = x.astype(np.float64)
    if gain is not None:
        n = n * gain.astype(np.float64) / np.sqrt((n * n).mean() + float(F(eps)))
    y, size = n.copy(), np.abs(n)
    h = len(inv_freq)
    a = np.float64(p) * inv_freq.astype(np.float64)
    c, s, m = np.cos(a), np.sin(a), float(F(magnitude))
    y[:h] = m * (n[:h] * c - n[h: 2 * h] * s)
    y[h: 2 * h] = m * (n[h: 2 * h] * c + n[:h] * s)
    size[:h] = size[h: 2 * h] = abs(m) * (np.abs(n[:h]) + np.abs(n[h: 2 * h]))
    return y, size


def positions(start, length, rows, max_new):
    """Each row's position, None where it has no place."""
    out = [None] * rows
    for s in reversed(range(len(length))):
        r0, r1 = int(start[s]), int(start[s + 1])
        if not 0 <= r0 <= r1 <= rows:
            continue
        for r in range(r0, r1):
            p = max(int(length[s]), 0) - (r1 - r0) + r - r0
            out[r] = p if p >= 0 and r - r0 < max_new else None
    return out


def gelu(x):
    """x / (1 + e^(-2 sqrt(2 / pi) (x + 0.044715 x^3))) in fp32 steps."""
    cube = (x * x) * x
    t = F(-2 * np.sqrt(2 / np.pi)) * (x + F(0.044715) * cube)
    return x / (F(1) + exp32(np.clip(t, F(-87), F(100))))


def linear_epilogue(w, up, K, q, s_act, z, act, res):
    """y of a linear (packed, s_row, rowsum, bias) with its epilogue, fp32 step
    by step; act is None, 'silu' or 'gelu'."""
    def product(packed, s_row, rowsum, bias):
        y = linear(packed, s_row, rowsum, K, q, s_act, z)[1]
        return y if bias is None else y + bias
    v = product(*w)
    u = np.ones_like(v) if up is None else product(*up)
    if act == "silu":
        v = swiglu(v, u)
    else:
        v = (gelu(v) if act == "gelu" else v) * u
    return v if res is None else res + v


class Pool:
    """Pages and who holds them."""

    def __init__(self, pages, S, columns, P, rng=None):
        self.refs, self.P = [0] * pages, P
        # (what stands in entries that hold nothing must not matter)
        self.table = [[-1 if rng is None else int(rng.integers(-9, pages + 9)) for _ in range(columns)] for _ in range(S)]

    def count(self, tokens):
        return -(-max(int(tokens), 0) // self.P)

    def page(self, s, j):
        p = self.table[s][j]
        return p if 0 <= p < len(self.refs) else None

    def fork(self, length, src, dst):
        for i, (a, b) in enumerate(zip(src, dst)):
            if not (0 <= a < len(self.table) and 0 <= b < len(self.table)) or b in src or b in dst[i + 1:]:
                continue
            for j in range(min(self.count(length[a]), len(self.table[a]))):
                p = self.page(a, j)
                self.table[b][j] = -1 if p is None else p
                if p is not None:
                    self.refs[p] += 1

    def truncate(self, length, keep):
        for s, row in enumerate(self.table):
            for j in range(self.count(keep[s]), min(self.count(length[s]), len(row))):
                p = self.page(s, j)
                if p is not None:
                    self.refs[p] = max(self.refs[p] - 1, 0)
                row[j] = -1

    def reserve(self, length, want):
        """(granted, from, to) lists."""
        S, columns = len(self.table), len(self.table[0])
        free = [p for p, n in enumerate(self.refs) if n <= 0]
        refs, used = list(self.refs), 0

        def written(s):
            n = max(int(length[s]), 0)
            if want[s] <= n or n % self.P == 0 or self.count(want[s]) > columns:
                return None
            return self.page(s, n // self.P)
        writes = [written(s) for s in range(S)]
        granted, src, dst = [0] * S, [-1] * S, [-1] * S
        for s in range(S):
            have, need = self.count(length[s]), self.count(want[s])
            if want[s] <= max(int(length[s]), 0):
                granted[s] = 1
                continue
            if need > columns:
                continue
            w = writes[s]
            shared = w is not None and refs[w] > 1
            sole = shared and sum(x == w for x in writes) >= refs[w] and w not in writes[s + 1:]
            n = need - have + (shared and not sole)
            used += n
            if not (used <= len(free) or (n == 0 and not sole)):
                continue
            granted[s] = 1
            ids = free[used - n: used]
            for p in ids:
                self.refs[p] = 1
            if shared and not sole:
                src[s], dst[s] = w, ids.pop(0)
                self.refs[w] -= 1
                self.table[s][have - 1] = dst[s]
            self.table[s][have: need] = ids
        return granted, src, dst

    def compact(self, length, moves):
        """(from, to, pages in use)."""
        live = sum(n > 0 for n in self.refs)
        holes = [p for p in range(live) if self.refs[p] <= 0]
        movers = [p for p in reversed(range(live, len(self.refs))) if self.refs[p] > 0]
        goes = dict(list(zip(movers, holes))[:moves])
        for a, b in goes.items():
            self.refs[a], self.refs[b] = 0, self.refs[a]
        for s, row in enumerate(self.table):
            for j in range(min(self.count(length[s]), len(row))):
                row[j] = goes.get(row[j], row[j])
        pad = [-1] * (moves - len(goes))
        return list(goes) + pad, list(goes.values()) + pad, live
