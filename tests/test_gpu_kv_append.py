"""The append to the paged int8 cache against the oracle: the whole cache
(codes and scales, untouched pages and slots included) bit for bit."""
import numpy as np
import pytest

from oracle import decode

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from packed_bit_gemv_tern_amd import tern  # noqa: E402
from gpu_util import DEV, to_dev  # noqa: E402
from kv_util import Paged  # noqa: E402


def values(rng, rows, heads, D, size=1.0):
    x = rng.normal(0, size, (rows, heads, D))
    x[:, :, ::13] *= 5
    return x.astype(np.float32)


def append(pg, new, length, k, v, extra=0, **kw):
    b = pg.batch(new, length, **kw)
    width = pg.heads * pg.D
    out = []
    for a in (k, v):
        t = torch.full((max(1, pg.rows), width + extra), float("nan"), device=DEV)
        t[:, :width] = to_dev(a.reshape(len(a), width))
        out.append(t)
    tern.tern_kv_append(pg.cache, b, out[0], width + extra, out[1], width + extra)
    decode.kv_append(pg.host, pg.table, pg.start, pg.length, k, v, pg.max_new)
    pg.check()


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [1, 3, 8])
def test_append_prompt_then_tokens(P, D, heads):
    """A ragged prompt, then single tokens whose values grow: pages fill,
    their scales grow and held codes move."""
    pg = Paged(3, 5, heads, D, P).upload()
    length = [2 * P + 5, 1, P]
    append(pg, length, length, *(values(pg.rng, sum(length), heads, D) for _ in "kv"))
    for step in range(4):
        length = [n + 1 for n in length]
        size = [1.0, 2.5, 0.3, 6.0][step]
        append(pg, [1, 1, 1], length, *(values(pg.rng, 3, heads, D, size) for _ in "kv"))


@pytest.mark.parametrize("new,length", [([5, 1, 9], [40, 1, 9]), ([33], [64]), ([17, 17], [33, 160]), ([16], [32]),
                                        ([1, 40, 2], [48, 64, 17])])
@pytest.mark.parametrize("P", [16, 64])
def test_append_drafted(new, length, P):
    pg = Paged(len(new), -(-160 // P), 2, 128, P, seed=1).upload()
    append(pg, new, length, *(values(pg.rng, sum(new), 2, 128) for _ in "kv"), extra=3)


def test_append_zero_tokens_and_values():
    """All-zero keys in a fresh page give scale 0 and codes 0; zero tokens
    after others keep the scale; a sequence with no new rows is untouched."""
    pg = Paged(3, 2, 2, 64, 16, seed=2).upload()
    zero = np.zeros((6, 2, 64), np.float32)
    append(pg, [3, 0, 3], [3, 20, 12], zero, zero)
    assert (pg.host.k_scale[pg.table[0, 0]] == 0).all()
    append(pg, [1, 0, 2], [4, 20, 14], *(values(pg.rng, 3, 2, 64) for _ in "kv"))


def test_append_tiny_and_ties():
    """Values on and between the steps (ties to even), and values whose scale
    is subnormal."""
    pg = Paged(2, 2, 1, 64, 32, seed=3).upload()
    x = (pg.rng.integers(-254, 255, (8, 1, 64)) / 2.0).astype(np.float32)
    x[0, 0, 0] = 127.0
    append(pg, [8, 0], [8, 0], x, x * np.float32(0.25))
    y = x * np.float32(1e-40)
    append(pg, [0, 8], [8, 8], y, y)


def test_append_bad_pages_and_bounds():
    """Ids outside the cache, lengths past the table, negative positions, rows
    outside the buffers and rows past max_new: passed over, all else as
    defined."""
    pg = Paged(6, 3, 2, 64, 16, seed=4).upload()
    pg.table[0, 1] = -1
    pg.table[1, 0] = pg.host.pages
    pg.table[1, 1] = 2 ** 31 - 1
    new, length = [20, 30, 5, 1, 4, 9], [40, 35, 60, 0, 2, 30]
    append(pg, new, length, *(values(pg.rng, sum(new), 2, 64) for _ in "kv"))
    append(pg, new, length, *(values(pg.rng, sum(new), 2, 64) for _ in "kv"), max_new=8)
    # offsets that do not lie in the buffers, or fall
    k, v = (values(pg.rng, 30, 2, 64) for _ in "kv")
    append(pg, [1] * 6, [10, 20, 30, 12, 8, 9], k, v, rows=30, max_new=16, start=[0, 4, 40, -3, 2, 1, 30])


def test_append_rows_of_a_padded_batch():
    """Rows past the last sequence's are not read (here: NaN)."""
    pg = Paged(2, 2, 2, 64, 16, seed=5).upload()
    k, v = (values(pg.rng, 8, 2, 64) for _ in "kv")
    k[5:], v[5:] = np.nan, np.nan
    append(pg, [3, 2], [9, 2], k, v, rows=8)
