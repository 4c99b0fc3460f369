"""Attention over the paged int8 cache against the oracle in fp64.

The tolerance counts the roundings of the definition's fp32 evaluation, per
row and head, with A the largest sum of |scale q_d k_jd| over d, V the largest
|v|, n the positions seen:
  - a score is off by at most A * (2^-21 + 24 * 2^-24): q enters as two fp16
    numbers (22 bits of the row's largest element), eight matrix instructions
    add to an fp32 accumulator twice each, and a few products follow;
  - a weight e^x is then off by that, plus 2^-22 for the exponential and 2^-21
    for its two fp16 numbers;
  - sums of weights and of weighted values: one rounding per 16 positions and
    lane and per joining step, at most (n / 64 + 32) * 4 roundings of 2^-24.
Numerator and denominator each carry the error, so y is off by at most twice
its sum times V."""
import numpy as np
import pytest

from oracle import decode

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from packed_bit_gemv_tern_amd import tern  # noqa: E402
from gpu_util import DEV, to_dev  # noqa: E402
from kv_util import Paged  # noqa: E402


def attend(pg, new, length, q_heads, extra=0, q_size=2.0, scale=None, q=None, **kw):
    b = pg.batch(new, length, **kw)
    D, width = pg.D, q_heads * pg.D
    scale = D ** -0.5 if scale is None else scale
    q = pg.rng.normal(0, q_size, (pg.rows, q_heads, D)).astype(np.float32) if q is None else q
    qd = torch.full((pg.rows, width + extra), float("nan"), device=DEV)
    qd[:, :width] = to_dev(q.reshape(pg.rows, width))
    y = torch.full((pg.rows, width + extra), 77.0, device=DEV)
    n = tern.tern_attention_workspace_bytes(pg.cache, b, q_heads)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)  # (NaN where read before it is written)
    tern.tern_attention(pg.cache, b, qd, width + extra, q_heads, scale, y, width + extra, ws)
    torch.cuda.synchronize()
    got = y.cpu().numpy()
    assert (got[:, width:] == 77).all()
    got = got[:, :width].reshape(pg.rows, q_heads, D)
    ref = np.full((pg.rows, q_heads, D), 77.0)
    size = decode.attention(pg.host, pg.table, pg.start, pg.length, q, scale, pg.max_new, ref)
    A, V = size[..., 0:1], size[..., 1:2]
    n = max(1, int(max(length)))
    tol = 2 * V * (A * (2 ** -21 + 24 * 2 ** -24) + 2 ** -22 + 2 ** -21 + (n / 64 + 32) * 4 * 2 ** -24)
    err = np.abs(got - ref)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), "off by %.3g, %.3g allowed, at %s" % (
        err.max(), tol.flat[np.argmax(err - tol)], np.unravel_index(np.argmax(err - tol), err.shape))
    return got


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 255, 256, 257, 1000])
@pytest.mark.parametrize("P,D", [(16, 128), (64, 128), (32, 64), (128, 64)])
def test_one_token(length, P, D):
    pg = Paged(2, -(-1000 // P), 2, D, P).upload()
    attend(pg, [1, 1], [length, max(1, length // 2)], 8)


@pytest.mark.parametrize("heads,group", [(1, 1), (8, 4), (3, 5), (2, 8), (1, 17), (2, 40)])
def test_head_layouts(heads, group):
    pg = Paged(2, 5, heads, 128, 64, seed=1).upload()
    attend(pg, [1, 1], [300, 77], heads * group)
    attend(pg, [3, 5], [300, 5], heads * group)


@pytest.mark.parametrize("new", [2, 4, 5, 8, 9, 16, 31, 64, 100])
@pytest.mark.parametrize("P", [16, 64])
def test_drafted_tokens_and_prompts(new, P):
    """Causal among the new rows: context before them, and none."""
    pg = Paged(3, -(-700 // P), 2, 128, P, seed=2).upload()
    attend(pg, [new, max(1, new // 2), new], [700, max(1, new // 2), new + 1], 8)


@pytest.mark.parametrize("max_len", [0, 1, 5000, 10 ** 6])
def test_long_context_and_hint(max_len):
    """The hint sets the pieces, not the result: too small, right, too large."""
    pg = Paged(2, -(-5000 // 32), 1, 128, 32, seed=3).upload()
    attend(pg, [1, 1], [5000, 1300], 4, max_len=max_len)
    attend(pg, [6, 6], [4999, 64], 4, max_len=max_len)


def test_ragged_batch_with_idle_slots():
    """Idle slots (one row, length 0) give 0; rows of no sequence are left as
    they were, and sequences without rows cost nothing."""
    pg = Paged(9, 8, 2, 64, 16, seed=4).upload()
    got = attend(pg, [1, 1, 0, 3, 1, 1, 1, 0, 2], [100, 0, 50, 3, 128, 17, 0, 0, 1], 4, rows=14)
    assert (got[1] == 0).all() and (got[7] == 0).all()
    assert (got[8] == 0).all()   # the first of two new rows where one position is held
    assert (got[10:] == 77).all()


def test_bad_pages():
    """A page outside the cache holds nothing; a row that sees only such pages
    is 0; lengths past the table end at it."""
    pg = Paged(4, 4, 2, 128, 64, seed=5).upload()
    pg.table[0, 1], pg.table[1, :], pg.table[2, 3] = -5, pg.host.pages, 2 ** 31 - 1
    got = attend(pg, [1, 2, 3, 1], [256, 200, 250, 10 ** 9], 8)
    assert (got[1:3] == 0).all()


def test_pages_never_written():
    """Slots past the length, and pages the table names past it, hold
    anything, scales of NaN and infinity among it."""
    pg = Paged(2, 6, 2, 64, 16, seed=6)
    for p in pg.table[:, 3:].flat:
        pg.host.k_scale[p], pg.host.v_scale[p] = np.nan, np.inf
    pg.upload()
    attend(pg, [1, 3], [48, 33], 4)
    pg.table[:, 3:] = -1
    attend(pg, [1, 3], [48, 33], 4)


@pytest.mark.parametrize("lo,hi", [(-6, 3), (-20, -15), (8, 12)])
def test_value_scales_apart(lo, hi):
    """Value scales over many powers of ten in one context, and pages of
    zeros."""
    def scales(rng, shape):
        s = 10.0 ** rng.uniform(lo, hi, shape)
        s[0] = rng.uniform(0.005, 0.02, shape[1:])
        s[1][rng.random(shape[1:]) < 0.2] = 0
        return s
    pg = Paged(2, 20, 2, 128, 16, seed=7, scales=scales).upload()
    attend(pg, [1, 4], [320, 211], 8)


@pytest.mark.parametrize("q_size", [0.0, 1e-12, 1e-3, 10.0, 1e6])
def test_query_sizes(q_size):
    """From scores of nothing (the mean of the values) to one position taking
    it all."""
    pg = Paged(2, 5, 2, 64, 64, seed=8).upload()
    attend(pg, [1, 2], [300, 40], 8, q_size=q_size)


def test_negative_and_zero_scale():
    pg = Paged(2, 5, 2, 64, 64, seed=9).upload()
    attend(pg, [1, 2], [300, 40], 8, scale=-0.2)
    attend(pg, [1, 2], [300, 40], 8, scale=0.0)


def test_strides():
    pg = Paged(2, 5, 2, 128, 32, seed=10).upload()
    attend(pg, [2, 1], [130, 40], 8, extra=1)
    attend(pg, [2, 1], [130, 40], 8, extra=4)


def test_shared_pages():
    """Two sequences reading the same pages, and one page twice in a table."""
    pg = Paged(2, 5, 2, 128, 32, seed=11).upload()
    pg.table[1, :3] = pg.table[0, :3]
    pg.table[1, 4] = pg.table[1, 3]
    attend(pg, [1, 1], [160, 155], 8)


def test_rows_past_max_new():
    pg = Paged(2, 5, 2, 128, 32, seed=12).upload()
    got = attend(pg, [6, 2], [130, 40], 8, max_new=4)
    assert (got[4:6] == 77).all()


# prompts: row tiles of 128 that end inside a token's heads, inside a wave and inside a step, windows of pages, splits
@pytest.mark.parametrize("new,length,heads,group,P,D", [
    ([130, 1, 77], [130, 40, 300], 2, 4, 16, 128), ([33, 64], [700, 64], 1, 3, 64, 64),
    ([200], [4500], 1, 2, 32, 128), ([65, 128], [5000, 4097], 1, 1, 128, 128), ([17, 40], [17, 1000], 2, 8, 64, 64),
    ([300], [300], 1, 5, 16, 64)])
def test_prompts(new, length, heads, group, P, D):
    pg = Paged(len(new), -(-max(length) // P), heads, D, P, seed=13).upload()
    attend(pg, new, length, heads * group, max_len=max(length))
    attend(pg, new, length, heads * group, max_len=64, extra=3)


def test_prompt_with_bad_pages_and_scales():
    def scales(rng, shape):
        s = 10.0 ** rng.uniform(-6, 3, shape)
        s[0] = rng.uniform(0.005, 0.02, shape[1:])
        s[1][rng.random(shape[1:]) < 0.2] = 0
        return s
    pg = Paged(3, 20, 2, 128, 16, seed=14, scales=scales).upload()
    pg.table[0, [0, 3, 7]], pg.table[1, :] = -1, pg.host.pages
    got = attend(pg, [40, 70, 90], [300, 200, 90], 8, rows=230)
    assert (got[40:110] == 0).all() and (got[200:] == 77).all()


def pad_table(pg, positions):
    """More columns than the sequences need: what the split is chosen by where
    no longest length is given."""
    columns = -(-positions // pg.P)
    pg.table = np.pad(pg.table, ((0, 0), (0, columns - pg.table.shape[1])), constant_values=-1)


@pytest.mark.parametrize("new,length,heads,group,P,D", [
    ([130, 1, 77], [130, 40, 300], 2, 4, 16, 128), ([33, 64], [700, 64], 1, 4, 64, 64),
    ([200], [4500], 1, 2, 32, 128), ([65, 128], [5000, 4097], 1, 2, 128, 128), ([17, 40], [17, 1000], 2, 8, 64, 64),
    ([300], [300], 1, 5, 16, 64)])
def test_prompts_in_long_tables(new, length, heads, group, P, D):
    """Tables of 20,000 positions and more: tiles of 128 rows, in pieces, most
    of them empty."""
    pg = Paged(len(new), -(-max(length) // P), heads, D, P, seed=15).upload()
    pad_table(pg, 20000)
    attend(pg, new, length, heads * group)
    pad_table(pg, 100000)
    attend(pg, new, length, heads * group, extra=3)


@pytest.mark.parametrize("D", [64, 128])
def test_prompts_among_idle_slots(D):
    """Enough workgroups for tiles of 128 rows over whole contexts: windows of
    pages, a last tile of two rows, idle slots."""
    pg = Paged(520, 2, 1, D, 64, seed=16).upload()
    pg.table = np.pad(pg.table, ((0, 0), (0, 78)), constant_values=-1)
    pg.table[0] = pg.table[: 80, 0]
    pg.table[519] = pg.table[100: 180, 1]
    got = attend(pg, [130] + [1] * 517 + [2, 65], [5101] + [0] * 517 + [2, 4096], 2)
    assert (got[130: 647] == 0).all()


def test_many_short_prompts():
    pg = Paged(16, 5, 8, 64, 32, seed=17).upload()
    attend(pg, [17, 33] * 8, [150, 33] * 8, 32)


@pytest.mark.parametrize("new,columns", [(1, 5), (1, 40), (3, 40), (6, 40), (20, 40), (50, 40), (50, 320)])
def test_queries_that_are_not_finite(new, columns):
    """NaN and infinity in a row of q stay in its row and head, whatever the
    tile and the split."""
    pg = Paged(2, 5, 1, 64, 64, seed=18).upload()
    pad_table(pg, 64 * columns)
    q = pg.rng.normal(0, 2, (2 * new, 4, 64)).astype(np.float32)
    length = [300, 200]
    good = attend(pg, [new, new], length, 4, q=q)
    b = pg.batch([new, new], length)
    q[0, 1, 5], q[2 * new - 1, 2, 63] = np.nan, np.inf
    qd, y = to_dev(q), torch.full((2 * new, 256), 77.0, device=DEV)
    ws = torch.empty(tern.tern_attention_workspace_bytes(pg.cache, b, 4), dtype=torch.uint8, device=DEV)
    tern.tern_attention(pg.cache, b, qd, 256, 4, 64 ** -0.5, y, 256, ws)
    got = y.cpu().numpy().reshape(2 * new, 4, 64)
    spoilt = np.zeros((2 * new, 4), bool)
    spoilt[0, 1] = spoilt[2 * new - 1, 2] = True
    assert np.isnan(got[spoilt]).all()
    assert (got[~spoilt] == good[~spoilt]).all()
