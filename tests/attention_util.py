"""Attention's error against 64 bits, measured by the weighted values that make
a row up, dim by dim, and not by the largest value in sight.

Per row, head and dim d, with weights w_j = e^(a_j - max a), W their sum, A_j =
|scale| sum_d |q_d k_jd| and s_j = a_j / ln 2:
  - a score is off by at most A_j * (2^-23 + 24 * 2^-24): q enters as two fp16
    numbers rounded to nearest, eight matrix instructions add to an fp32
    accumulator twice each, and a few products follow;
  - its exponent is rounded three times, at magnitudes up to S + Z + 12 each and
    once more up to 2 S (S the largest |s|, Z the octaves between the V scales
    seen): ln 2 * 2^-24 * (5 S + 3 Z + 36);
  - the exponential, the two fp16 numbers, the V scale's logarithm and reciprocal
    and the product with it: 2^-23 each, 6 of them;
  - sums of weights and of weighted values: one rounding per 16 positions and
    lane and per joining step, at most (n / 64 + 32) * 4 roundings of 2^-24;
  - a weight far below a row's largest is off by up to 2^-25 in units in which the
    row's largest sum is 2^8 or more, that is by 2^-33 of sum_j w_j max_d |v_jd|, with a
    standard deviation of 2^-25.8; many of them add as independent errors (six
    deviations are allowed), and weights 2^-60 of the largest may be missing.
Numerator and denominator carry these."""
import numpy as np
import torch

from oracle import decode
from packed_bit_gemv_tern_amd import tern
from gpu_util import DEV, to_dev


def reference(pg, q, scale):
    """(y, allowed error) of every row, head and dim, in 64 bits (0 and 0 for rows that see nothing)."""
    y, tol = np.zeros((2,) + q.shape)
    G, P = q.shape[1] // pg.heads, pg.P
    for s, (r0, n, pos0, held) in enumerate(decode.sequences(pg.start, pg.length, len(q), P, pg.table.shape[1])):
        for h in range(pg.heads):
            present, k, v = pg.host.values(pg.table, s, held, h)
            vs = np.zeros(held)
            for j in range(-(-held // P)):
                p = pg.host.page(pg.table, s, j)
                vs[j * P: (j + 1) * P] = 0 if p is None else pg.host.v_scale[p, h]
            for i in range(n):
                m = max(0, min(held, pos0 + i + 1))
                see = np.flatnonzero(present[:m])
                if not len(see):
                    continue
                x, kk, vv, z = q[r0 + i, h * G: (h + 1) * G].astype(np.float64), k[see], v[see], vs[see]
                a = x @ kk.T * scale  # G x positions
                A = np.abs(x) @ np.abs(kk).T * abs(scale)
                w = np.exp(a - a.max(1, keepdims=True))
                W = w.sum(1, keepdims=True)
                S = np.abs(a).max(1, keepdims=True) / np.log(2)
                Z = np.ptp(np.log2(z[z > 0])) if (z > 0).any() else 0
                delta = A * 26 * 2 ** -24 + np.log(2) * 2 ** -24 * (5 * S + 3 * Z + 36) + 6 * 2 ** -23
                c = (m / 64 + 32) * 4 * 2 ** -24
                size, num = w @ np.abs(vv) / W, w @ vv / W
                wz = w * z
                codes = np.abs(vv) / np.where(z > 0, z, 1)[:, None]
                rows = slice(h * G, (h + 1) * G)
                floor = (6 * 2 ** -33.8 * np.sqrt((codes ** 2).sum(0)) * (w @ np.abs(vv).max(1))[:, None]
                         + 2 ** -60 * wz.max(1, keepdims=True) * codes.sum(0)) / W
                y[r0 + i, rows] = num
                tol[r0 + i, rows] = ((w * delta) @ np.abs(vv) / W + np.abs(num) * ((w * delta).sum(1, keepdims=True) / W)
                                     + c * (size + np.abs(num)) + floor)
    return y, tol


def attend(pg, new, length, q, scale=None, **kw):
    b = pg.batch(new, length, **kw)
    rows, heads, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    qd, y = to_dev(q.reshape(rows, -1)), torch.full((rows, heads * D), 77.0, device=DEV)
    ws = torch.full((tern.tern_attention_workspace_bytes(pg.cache, b, heads),), 255, dtype=torch.uint8, device=DEV)
    tern.tern_attention(pg.cache, b, qd, heads * D, heads, scale, y, heads * D, ws)
    torch.cuda.synchronize()
    got = y.cpu().numpy().reshape(q.shape)
    ref, tol = reference(pg, q, scale)
    assert np.isfinite(got).all()
    err = np.abs(got - ref)
    worst = np.unravel_index(np.argmax(err / np.maximum(tol, 1e-300)), err.shape)
    assert (err <= tol).all(), "%s: %g, not %g (off by %.3g, %.3g allowed)" % (
        worst, got[worst], ref[worst], err[worst], tol[worst])
    return got


def pad_table(pg, positions):
    columns = -(-positions // pg.P)
    pg.table = np.pad(pg.table, ((0, 0), (0, columns - pg.table.shape[1])), constant_values=-1)


# rows of a sequence and KV head (new tokens, query heads) and the table's positions: tiles of 8, 16, 32 and of 128 in pieces
TILES = [(1, 4, 0), (3, 4, 0), (6, 4, 0), (40, 4, 0), (40, 4, 20000)]
