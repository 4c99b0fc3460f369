"""Plain forms of the decode step's operators between the linears: the norm
with its int8 output, the append to the paged int8 cache, the attention over
it, and sampling.  numpy, in 64 bits except for the roundings to fp32 and to
codes that the formats are defined by; one row, page or token at a time, no
code shared with the library.
"""
import numpy as np

from . import quantize_act

F = np.float32


def rmsnorm_quantize(x, res, gain, eps):
    """(h, q, s_act, z) of M x K fp32 rows; res may be None."""
    h = x.astype(F) if res is None else (x.astype(F) + res.astype(F))
    d = h.astype(np.float64)
    y = d * gain.astype(np.float64) / np.sqrt((d * d).mean(1, keepdims=True) + float(F(eps)))
    return (h,) + tuple(quantize_act(y.astype(F)))


class Cache:
    """A paged cache on the host: k (pages, heads, P, D), v (pages, heads, D,
    P), scales (pages, heads)."""

    def __init__(self, k, v, k_scale, v_scale):
        self.k, self.v, self.k_scale, self.v_scale = k.copy(), v.copy(), k_scale.copy(), v_scale.copy()
        self.pages, self.heads, self.P, self.D = k.shape

    def page(self, table, s, j):
        """The page of positions j * P ..., or None."""
        if j < 0 or j >= table.shape[1]:
            return None
        p = int(table[s, j])
        return p if 0 <= p < self.pages else None

    def values(self, table, s, n, h):
        """(present, k, v) of positions 0 .. n - 1 of one KV head, fp64."""
        present = np.zeros(n, bool)
        k, v = np.zeros((n, self.D)), np.zeros((n, self.D))
        for j in range(-(-n // self.P)):
            p = self.page(table, s, j)
            m = min(self.P, n - j * self.P)
            if p is None:
                continue
            at = slice(j * self.P, j * self.P + m)
            present[at] = True
            k[at] = self.k[p, h, :m].astype(np.float64) * float(self.k_scale[p, h])
            v[at] = self.v[p, h, :, :m].T.astype(np.float64) * float(self.v_scale[p, h])
        return present, k, v


def sequences(start, length, rows, P, columns):
    """(first row, new rows, first new position, positions held) of each
    sequence, as the calls define them."""
    out = []
    for s in range(len(length)):
        r0, r1 = int(start[s]), int(start[s + 1])
        if not (0 <= r0 <= r1 <= rows):
            r0 = r1 = 0
        n, ln = r1 - r0, max(0, int(length[s]))
        out.append((r0, n, ln - n, min(ln, columns * P)))
    return out


def kv_append(cache, table, start, length, k_new, v_new, max_new):
    """Appends in place; k_new and v_new are rows x heads x D fp32."""
    P = cache.P
    for s, (r0, n, pos0, held) in enumerate(sequences(start, length, len(k_new), P, table.shape[1])):
        first, last = max(pos0, 0), min(held, pos0 + min(n, max_new))
        j = first // P
        while first < last:
            hi = min(last, (j + 1) * P)
            p = cache.page(table, s, j)
            rows = slice(r0 + first - pos0, r0 + hi - pos0)
            lo, m = first - j * P, hi - j * P
            first, j = hi, j + 1
            if p is None:
                continue
            for h in range(cache.heads):
                for x, scale, codes in ((k_new[rows, h], cache.k_scale, cache.k[p, h]),
                                        (v_new[rows, h], cache.v_scale, cache.v[p, h].T)):
                    was = F(scale[p, h]) if lo else F(0)
                    now = max(was, F(np.abs(x).max()) / F(127))
                    if now > was and lo:
                        ratio = was / now
                        codes[:lo] = np.rint(codes[:lo].astype(F) * ratio).astype(np.int8)
                    q = np.zeros_like(x) if now == 0 else np.rint(x / now)
                    codes[lo:m] = np.clip(q, -127, 127).astype(np.int8)
                    scale[p, h] = now


def attention(cache, table, start, length, q, scale, max_new, y):
    """Fills the rows of y (rows x q_heads x D, fp64) that belong to a
    sequence; returns for each of those rows and heads (sum of |q k| * |scale|
    at its largest, largest |v|), the measures of the rounding errors."""
    heads = q.shape[1]
    G = heads // cache.heads
    size = np.zeros(y.shape[:2] + (2,))
    for s, (r0, n, pos0, held) in enumerate(sequences(start, length, len(q), cache.P, table.shape[1])):
        for h in range(cache.heads):
            present, k, v = cache.values(table, s, held, h)
            for i in range(min(n, max_new)):
                m = max(0, min(held, pos0 + i + 1))
                see = present[:m]
                for g in range(h * G, (h + 1) * G):
                    y[r0 + i, g] = 0
                    if not see.any():
                        continue
                    qd = q[r0 + i, g].astype(np.float64)
                    a = (k[:m][see] @ qd) * scale
                    w = np.exp(a - a.max())
                    y[r0 + i, g] = (w / w.sum()) @ v[:m][see]
                    size[r0 + i, g] = (np.abs(k[:m][see]) @ np.abs(qd)).max() * abs(scale), np.abs(v[:m][see]).max()
    return size


def sample(x, temperature, u, top_k=None, top_p=None, min_p=None):
    """(token, prob, kept) of one row of logits."""
    x = np.asarray(x, np.float64)
    live = np.flatnonzero(x > -np.inf)  # (NaN compares false)
    if not len(live):
        return -1, 0.0, 0
    order = live[np.argsort(-x[live], kind="stable")]
    if not temperature > 0:
        return int(order[0]), 1.0, 1
    v = x[order]
    with np.errstate(all="ignore"):
        w = np.where(v == v[0], 1.0, np.exp((v - v[0]) / float(temperature)))
    n = len(order)
    if top_k is not None and top_k > 0:
        n = min(n, int(top_k))
    if top_p is not None and top_p < 1:
        before = np.cumsum(w[:n]) - w[:n]
        n = max(1, int((before < max(float(top_p), 0.0) * w[:n].sum()).sum()))
    if min_p is not None and min_p > 0:
        n = max(1, min(n, int((w >= min(float(min_p), 1.0)).sum())))
    kept = np.argsort(order[:n])
    run = np.cumsum(w[kept])
    i = min(int((run <= min(max(float(u), 0.0), 1.0) * run[-1]).sum()), n - 1)
    return int(order[kept[i]]), float(w[kept[i]] / run[-1]), n
