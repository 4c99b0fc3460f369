"""Scores whose terms are far apart: key channels far larger than the others
with queries that do not average to 0, query elements far apart, and queries
near the largest fp32 numbers.  The error of each row against 64 bits is
measured by the sums of |q k| position by position, through every tile."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from packed_bit_gemv_tern_amd import tern  # noqa: E402
from attention_util import TILES, attend, pad_table  # noqa: E402
from gpu_util import DEV, to_dev  # noqa: E402
from kv_util import Paged  # noqa: E402


def pages(new, columns, n, D, seed):
    pg = Paged(2, -(-n // 16), 1, D, 16, seed=seed, scales=lambda rng, shape: rng.uniform(0.005, 0.03, shape))
    if columns:
        pad_table(pg, columns)
    return pg


@pytest.mark.parametrize("n", [50, 300])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,group,columns", TILES)
def test_key_channel_far_above_the_others(new, group, columns, D, n):
    """A page's scale belongs to its largest channel: the others' codes are
    small; queries are all positive."""
    pg = pages(new, columns, n, D, 1)
    k = np.where(pg.rng.random(pg.host.k.shape) < 0.3, pg.rng.choice([-1, 1], pg.host.k.shape), 0)
    k[..., 7] = pg.rng.choice([-127, 126, 127], k.shape[:-1])
    pg.host.k[:] = k
    q = (3 + 0.3 * pg.rng.normal(0, 1, (2 * new, group, D))).astype(np.float32)
    attend(pg.upload(), [new, new], [n, n - 7], q, scale=1.0)


@pytest.mark.parametrize("new,group,columns", TILES)
@pytest.mark.parametrize("q_size,scale", [(1e37, 1e-10), (1e-30, 1e25)])
def test_queries_of_extreme_size(new, group, columns, q_size, scale):
    """Queries near the ends of fp32, with scales that bring the scores back to
    ordinary ones."""
    pg = pages(new, columns, 100, 64, 2)
    pg.host.k_scale *= np.float32(2e-28 if q_size > 1 else 20)
    q = (q_size * pg.rng.normal(0, 3, (2 * new, group, 64))).astype(np.float32)
    attend(pg.upload(), [new, new], [100, 93], q, scale=scale)


@pytest.mark.parametrize("new,group,columns", TILES)
def test_query_element_far_above_the_others(new, group, columns):
    """One element of q 2^12 times the others, in a channel where the codes
    are 0: the scores are the others'."""
    pg = pages(new, columns, 200, 128, 3)
    pg.host.k[..., 5] = 0
    q = pg.rng.normal(0, 3, (2 * new, group, 128)).astype(np.float32)
    q[..., 5] *= 4096
    attend(pg.upload(), [new, new], [200, 150], q)


@pytest.mark.parametrize("new,group,columns", TILES)
@pytest.mark.parametrize("size", [1e4, 1e7, 1e8, 1e10, 1e30])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_finite_size(new, group, columns, size, sign):
    """One key, held at several positions of pages with different V scales,
    scores above all others by a hundredth of scores of `size`, which are all
    positive or all negative; every third row has ordinary queries.  The rows of
    such scores are the mean of its values: each weight is off by 2^-20 at most
    (equal scores, the exponential, the split), sums by the roundings of
    attention_util.  Scores s / ln 2 below 2^20 share their exponent's digits with the V
    scale's logarithm: its rounding is ln 2 * 2^-24 * 5 |s| at most, as there."""
    n = 900
    pg = pages(new, columns, n, 64, 4)
    way = pg.rng.choice(np.array([-1.0, 1.0]), 64)
    pg.host.k[:] = (sign * 60 * way + pg.rng.integers(-3, 4, pg.host.k.shape)).astype(np.int8)
    pg.host.k_scale[:] = np.float32(1 / 127)
    top = [5, 16, 70, 71, 300, 640, 820]
    for s in range(2):
        for j in top:
            pg.host.k[pg.table[s, j // 16], 0, j % 16] = (sign * 60 + 6) * way
    length = [n, n - 70]
    q = np.empty((2 * new, group, 64), np.float32)
    q[:] = size * way / 30
    ordinary = np.arange(2 * new) % 3 == 2
    q[ordinary] = pg.rng.normal(0, 1, q[ordinary].shape)
    got = attend(pg.upload(), [new, new], length, q, scale=1.0)
    for r in np.flatnonzero(~ordinary):
        s = r // new
        v = np.array([pg.host.v[pg.table[s, j // 16], 0, :, j % 16] * float(pg.host.v_scale[pg.table[s, j // 16], 0])
                      for j in top if j < length[s] - new + 1 + r % new])
        S = np.abs(q[r, 0] * 66 / 127).sum() / np.log(2)
        exponent = np.log(2) * 2 ** -24 * 5 * S if S < 2 ** 20 else 0
        tol = (2 ** -19 + exponent + (n / 64 + 32) * 8 * 2 ** -24) * np.abs(v).mean(0)
        assert (np.abs(got[r] - v.mean(0)) <= tol).all(), r


@pytest.mark.parametrize("new,group", [(1, 4), (3, 4), (6, 4), (40, 4)])
def test_scores_that_pass_the_border_in_small_steps(new, group):
    """Two keys whose scores lie just under and just over 2^20 (times ln 2), two
    octaves apart, in steps of one wave, beside rows of far larger scores: both
    count, as 1 to 4.  A score there is rounded to 2^-4 some five times (two
    products' sums, three factors), which moves a weight of 1/5 by less than 0.06."""
    n = 400
    pg = pages(new, 0, n, 64, 5)
    pad_table(pg, 100000)
    way = pg.rng.choice(np.array([-1.0, 1.0]), 64)
    pg.host.k[:] = -60 * way
    pg.host.k_scale[:] = np.float32(1 / 64)
    a, b = 3, 266  # the same wave's, whichever tile
    for s in range(2):
        for j, c in ((a, -60), (b, 60)):
            page = pg.table[s, j // 16]
            pg.host.k[page, 0, j % 16] = 64 * way
            pg.host.k[page, 0, j % 16, 0] = c
    q = np.empty((2 * new, group, 64), np.float32)
    q[:] = 2 ** 20 * np.log(2) / 63 * way  # 63 channels of one: a score of 2^20
    q[..., 0] = 2 * np.log(2) / (120 / 64)
    far = np.arange(2 * new * group).reshape(2 * new, group) % 2 == 1
    q[far] *= 1000
    length = [n, n - 20]
    bt = pg.upload().batch([new, new], length)
    y = torch.empty((2 * new, group * 64), device=DEV)
    ws = torch.empty(tern.tern_attention_workspace_bytes(pg.cache, bt, group), dtype=torch.uint8, device=DEV)
    tern.tern_attention(pg.cache, bt, to_dev(q.reshape(2 * new, -1)), group * 64, group, 1.0, y, group * 64, ws)
    got = y.cpu().numpy().reshape(q.shape)
    for r in range(2 * new):
        s = r // new
        v = [pg.host.v[pg.table[s, j // 16], 0, :, j % 16] * float(pg.host.v_scale[pg.table[s, j // 16], 0]) for j in (a, b)]
        near = ~far[r]
        assert (np.abs(got[r, near] - (0.2 * v[0] + 0.8 * v[1])) <= 0.06 * np.abs(v[0] - v[1]) + 1e-5).all(), r
        assert (np.abs(got[r, far[r]] - v[1]) <= 1e-5).all(), r


@pytest.mark.parametrize("new,group", [(1, 4), (3, 4), (6, 4), (40, 4)])
@pytest.mark.parametrize("first,then", [(1e8, 3.3e8), (1e10, 7.7e10), (3e6, 1e9), (2 ** 20, 2 ** 21), (1e30, 2.9e30)])
def test_far_scores_that_grow(new, group, first, then):
    """A row's largest score is met first in one step of a wave, one some times as
    large in a later step of it, and the same key twice more after that: the row is
    the mean of the values of those three (each weight to 2^-20, see above)."""
    n = 1800
    pg = pages(new, 0, n, 64, 6)
    pad_table(pg, 100000)
    way = pg.rng.choice(np.array([-1.0, 1.0]), 64)
    pg.host.k[:] = -60 * way
    pg.host.k_scale[:] = np.float32(1 / 127)
    top = [266, 520, 780]
    for s in range(2):
        for j in [3] + top:
            page = pg.table[s, j // 16]
            pg.host.k[page, 0, j % 16] = (127 if j in top else max(1, round(127 * first / then))) * way
    q = np.empty((2 * new, group, 64), np.float32)
    q[:] = then / 64 * way * pg.rng.uniform(0.9, 1.1, (2 * new, group, 1))
    length = [n, n - 20]
    bt = pg.upload().batch([new, new], length)
    y = torch.empty((2 * new, group * 64), device=DEV)
    ws = torch.empty(tern.tern_attention_workspace_bytes(pg.cache, bt, group), dtype=torch.uint8, device=DEV)
    tern.tern_attention(pg.cache, bt, to_dev(q.reshape(2 * new, -1)), group * 64, group, 1.0, y, group * 64, ws)
    got = y.cpu().numpy().reshape(q.shape)
    for r in range(2 * new):
        s = r // new
        v = np.array([pg.host.v[pg.table[s, j // 16], 0, :, j % 16] * float(pg.host.v_scale[pg.table[s, j // 16], 0])
                      for j in top])
        tol = (2 ** -19 + (n / 64 + 32) * 8 * 2 ** -24) * np.abs(v).mean(0)
        assert (np.abs(got[r] - v.mean(0)) <= tol).all(), r


@pytest.mark.parametrize("new,group,columns", TILES)
@pytest.mark.parametrize("size", [1e4, 1e6, 1e7, 3e7, 1e8, 1e9, 1e20])
def test_far_scores_on_values_of_0(new, group, columns, size):
    """The keys of the largest scores lie on pages whose V scale is 0, and the others
    far below them: those rows are 0, ordinary ones beside them as ever."""
    n = 700
    pg = pages(new, columns, n, 64, 7)
    way = pg.rng.choice(np.array([-1.0, 1.0]), 64)
    pg.host.k[:] = (-60 * way + pg.rng.integers(-30, 30, pg.host.k.shape)).astype(np.int8)
    pg.host.k_scale[:] = np.float32(1 / 127)
    for s in range(2):
        for j in (5, 70, 300, 301, 600):
            pg.host.k[pg.table[s, j // 16], 0, j % 16] = 127 * way
            pg.host.v_scale[pg.table[s, j // 16]] = 0
    q = np.empty((2 * new, group, 64), np.float32)
    q[:] = size * way / 30 * pg.rng.uniform(0.5, 1.5, (2 * new, group, 1))
    ordinary = np.arange(2 * new) % 3 == 2
    q[ordinary] = pg.rng.normal(0, 1, q[ordinary].shape)
    got = attend(pg.upload(), [new, new], [n, n - 70], q, scale=1.0)
    assert (got[~ordinary] == 0).all()


@pytest.mark.parametrize("new,group,columns", TILES)
@pytest.mark.parametrize("size", [1e6, 1e7, 3e7, 6e7, 1e8, 3e8, 1e9])
@pytest.mark.parametrize("seed", [8, 9])
def test_equal_far_scores_below_values_of_0(new, group, columns, size, seed):
    """The same as above where the others' scores are equal and their V scales
    octaves apart: their weights' ratios are ordinary, 10^6 octaves and more below
    the base."""
    n = 700
    pg = pages(new, columns, n, 64, seed)
    way = pg.rng.choice(np.array([-1.0, 1.0]), 64)
    pg.host.k[:] = -60 * way
    pg.host.k_scale[:] = np.float32(1 / 127)
    pg.host.v_scale[:] = 2.0 ** pg.rng.uniform(-12, 12, pg.host.v_scale.shape)
    for s in range(2):
        for j in (5, 70, 300, 301, 600):
            pg.host.k[pg.table[s, j // 16], 0, j % 16] = 127 * way
            pg.host.v_scale[pg.table[s, j // 16]] = 0
    q = np.empty((2 * new, group, 64), np.float32)
    q[:] = size * way / 30 * pg.rng.uniform(0.5, 1.5, (2 * new, group, 1))
    got = attend(pg.upload(), [new, new], [n, n - 70], q, scale=1.0)
    assert (got == 0).all()
