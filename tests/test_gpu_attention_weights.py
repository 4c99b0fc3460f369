"""Attention where most of a row's softmax weight lies on values near 0, or on
pages whose V scale is far below that of others: held to the accuracy of the
weighted values that make each row up (attention_util)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
pytest.importorskip("torch")
from attention_util import TILES, attend, pad_table  # noqa: E402
from kv_util import Paged  # noqa: E402


def setup(new, group, columns, n, D=128, P=16, seed=0, scales=None, spread=1.0, heads=1):
    """Contexts of n and n - 20 positions and queries near one direction (the
    returned one), so that a key can be made to score high for every row."""
    pg = Paged(2, -(-n // P), heads, D, P, seed=seed, scales=scales)
    way = pg.rng.choice(np.array([-1.0, 1.0]), D)
    q = way + 0.3 * pg.rng.normal(0, spread, (2 * new, heads * group, D))
    if columns:
        pad_table(pg, columns)
    return pg, way, q.astype(np.float32)


def key_towards(pg, s, j, way, by=127):
    """Key codes of position j of sequence s: `by` along the given signs."""
    pg.host.k[pg.table[s, j // pg.P], :, j % pg.P] = by * way


@pytest.mark.parametrize("gap", [8, 12, 16, 20])
@pytest.mark.parametrize("n", [60, 700, 2500])
@pytest.mark.parametrize("new,group,columns", TILES)
def test_one_position_takes_the_weight_and_holds_nothing(new, group, columns, n, gap):
    """The first position scores `gap` above all others; its value is 0."""
    def scales(rng, shape):
        s = rng.uniform(0.005, 0.03, shape)
        s[0] = 1.0 / 127
        return s
    pg, way, q = setup(new, group, columns, n, seed=gap, scales=scales)
    for s in range(2):
        key_towards(pg, s, 0, way)
        pg.host.v[pg.table[s, 0], :, :, 0] = 0
    attend(pg.upload(), [new, new], [n, n - 20], q, scale=gap / 128)


@pytest.mark.parametrize("octaves", [6, 14, 20, 26, 34, 60, 90])
@pytest.mark.parametrize("new,group,columns", TILES)
def test_weight_on_pages_of_small_values(new, group, columns, octaves):
    """Every row's weight lies on the first page and one far on, whose V scales
    are far below those of all others; the others' scores are lower by more."""
    n = 300
    def scales(rng, shape):
        s = rng.uniform(0.005, 0.03, shape)
        s[0] = 1.0 / 127
        s[1] = rng.uniform(0.5, 1.0, shape[1:])
        return s
    pg, way, q = setup(new, group, columns, n, seed=octaves, scales=scales)
    pg.host.k //= 4
    for s in range(2):
        for j in list(range(0, 16)) + list(range(160, 176)):
            key_towards(pg, s, j, way)
            pg.host.k[pg.table[s, j // 16], :, j % 16] -= pg.rng.integers(0, 12, 128) * way.astype(int)
        for p in (0, 10):
            pg.host.v_scale[pg.table[s, p]] *= np.float32(2.0 ** -octaves)
    gap = octaves * np.log(2) + 8
    attend(pg.upload(), [new, new], [n, n - 20], q, scale=gap / 128)


@pytest.mark.parametrize("P", [16, 32])
@pytest.mark.parametrize("n,new,group,columns", [(20, 8, 1, 0), (36, 8, 1, 0), (40, 16, 1, 0), (60, 32, 1, 0),
                                                 (64, 64, 1, 0), (64, 64, 4, 20000), (150, 150, 1, 20000)])
def test_later_pages_that_a_row_does_not_see(n, new, group, columns, P):
    """Early rows see the first page alone, whose V scale is 2^-30 of the
    next one's, within one step of 64 positions and beyond."""
    def scales(rng, shape):
        s = rng.uniform(0.005, 0.03, shape)
        return s
    pg, way, q = setup(new, group, columns, n + 20, P=P, seed=n, scales=scales)
    for s in range(2):
        pg.host.v_scale[pg.table[s, 0]] *= np.float32(2.0 ** -30)
    attend(pg.upload(), [new, new], [n, n - 1], q)


@pytest.mark.parametrize("new,group,columns", TILES)
@pytest.mark.parametrize("lo,hi,zeros", [(-6, 3, 0.2), (-3, 0, 0.5), (-30, 30, 0.1)])
def test_scales_far_apart(new, group, columns, lo, hi, zeros):
    """V scales over many powers of ten, some 0 (with codes that are not), in
    every order, and tokens without a page."""
    def scales(rng, shape):
        s = 10.0 ** rng.uniform(lo, hi, shape)
        s[0] = rng.uniform(0.005, 0.03, shape[1:])
        s[1][rng.random(shape[1:]) < zeros] = 0
        return s
    pg, way, q = setup(new, group, columns, 700, D=64, seed=3, scales=scales, spread=10.0, heads=2)
    pg.table[0, [2, 9, 10, 11, 12, 13]] = -1
    attend(pg.upload(), [new, new], [700, 411], q)


@pytest.mark.parametrize("new,group,columns", TILES)
def test_zeros_take_the_weight(new, group, columns):
    """A page whose V scale is 0 (its codes are not) takes nearly all of the
    weight: it counts in the sum of weights, and adds nothing."""
    n = 300
    pg, way, q = setup(new, group, columns, n, seed=5, scales=lambda rng, shape: rng.uniform(0.005, 0.03, shape))
    for s in range(2):
        for j in range(64, 80):
            key_towards(pg, s, j, way)
        pg.host.k_scale[pg.table[s]] = 1.0 / 127
        pg.host.v_scale[pg.table[s, 4]] = 0
    attend(pg.upload(), [new, new], [n, n - 20], q, scale=14 / 128)


@pytest.mark.parametrize("D", [64, 128])
def test_whole_contexts_in_tiles_of_128(D):
    """Enough workgroups for tiles of 128 rows without pieces: a position that
    takes the weight and holds nothing, pages missing inside the context, pages
    of zeros and scales far apart."""
    pg = Paged(2, 20, 2, D, 16, seed=6)
    way = pg.rng.choice(np.array([-1.0, 1.0]), D)
    q = (way + 0.3 * pg.rng.normal(0, 1, (140 + 254 + 66, 8, D))).astype(np.float32)
    idle = np.full((254, 20), -1, np.int32)
    for p in pg.table[0]:
        pg.host.k_scale[p] = 1.0 / 127
    key_towards(pg, 0, 5, way)
    pg.host.v[pg.table[0, 0], :, :, 5] = 0
    pg.host.v_scale[pg.table[1]] = 10.0 ** pg.rng.uniform(-6, 3, (20, 2))
    pg.host.v_scale[pg.table[1, [4, 9]]] = 0
    pg.table[1, [3, 7, 8, 12]] = -1
    pg.table = np.concatenate([pg.table[:1], idle, pg.table[1:]])
    got = attend(pg.upload(), [140] + [1] * 254 + [66], [310] + [0] * 254 + [300], q, scale=14 / 128, max_len=320)
    assert (got[140: 394] == 0).all()


@pytest.mark.parametrize("gap", [5, 11, 14, 16])
@pytest.mark.parametrize("scale", [1e30, 1e-30])
@pytest.mark.parametrize("new,group,columns", TILES)
def test_scores_that_grow_beside_extreme_scales(new, group, columns, scale, gap):
    """V scales at either end of the range, the first 64 positions' scores
    below the others' by `gap`."""
    n = 900
    pg, way, q = setup(new, group, columns, n, seed=gap, scales=lambda rng, shape: rng.uniform(0.5, 1.0, shape))
    pg.host.v_scale *= np.float32(scale)
    pg.host.k_scale[:] = 1.0 / 127
    pg.host.k //= 8
    for s in range(2):
        for j in range(64, n - 20 * s):
            pg.host.k[pg.table[s, j // 16], :, j % 16] = 100 * way + pg.rng.integers(-20, 20, 128)
    attend(pg.upload(), [new, new], [n, n - 20], q, scale=gap / 100)
