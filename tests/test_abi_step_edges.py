"""Calls at the borders of the lookup's, rotation's, epilogue's and pages' checks:
status codes before any launch (no GPU needed: nothing below gets past them)."""

import pytest

from packed_bit_gemv_tern_amd import tern
from test_abi_step import (A16, ALIGN, INF, INVALID, NAN, ODD2, OK, RANGE, WORKSPACE, batch, compact, embed,  # noqa: F401
                           lib, linear, pool, rope, weights)

FLT_MAX = (2 - 2 ** -23) * 2.0 ** 127


def test_compact_without_rows(lib):  # noqa: F811
    """live and the lists are written, so they and refs are checked; table and len
    are not used, and without refs there is nothing to write about."""
    none = dict(S=0, ld_table=0, table=None)
    for kw in ({"live": None}, {"src": None}, {"dst": None}):
        assert compact(lib, pool(**none), length=None, **kw) == INVALID, kw
    for kw in ({"live": ODD2}, {"src": ODD2}, {"dst": ODD2}):
        assert compact(lib, pool(**none), length=None, **kw) == ALIGN, kw
    assert compact(lib, pool(refs=ODD2, **none)) == ALIGN
    for kw in ({"ws": None}, {"ws": A16 + 16}, {"n": 64}):
        assert compact(lib, pool(**none), **kw) == WORKSPACE, kw
    assert compact(lib, pool(refs=None, **none), live=None, ws=None) == OK


@pytest.mark.parametrize("M", [1, 8, 16])
@pytest.mark.parametrize("gate", [False, True])
def test_linear_epilogue_rows_that_no_launch_counts(lib, M, gate):  # noqa: F811
    """Up to 16 tokens take 64 rows to a workgroup at most, more could take 256: from
    2^30 rows on no launch of the former counts its threads."""
    up = weights() if gate else None
    for N in (2 ** 30, 2 ** 30 + 1, 2 ** 31 - 1000):
        assert linear(lib, up=up, N=N, M=M, ldr=N, ldy=N) == RANGE, N


@pytest.mark.parametrize("M", [17, 64, 128])
def test_linear_epilogue_rows_of_the_last_tile(lib, M):  # noqa: F811
    """Row numbers are 32 bits wide: the last tile's may not pass them."""
    for N in (2 ** 31 - 255, 2 ** 31 - 1):
        assert linear(lib, N=N, M=M, ldr=N, ldy=N) == RANGE, N


def test_every_finite_scale(lib):  # noqa: F811
    """Up to the largest float, and nothing past it (empty calls: nothing is launched)."""
    none = dict(b=batch(max_new=0))
    for x in (3.401e38, FLT_MAX, 2.0 ** -149):
        assert embed(lib, M=0, scale=x) == OK and embed(lib, M=0, scale=-x) == OK
        assert rope(lib, mag=x, **none) == OK and rope(lib, mag=-x, **none) == OK and rope(lib, eps=x, **none) == OK
        assert rope(lib, eps=-x, **none) == INVALID
    for x in (INF, -INF, NAN):
        assert embed(lib, M=0, scale=x) == INVALID
        assert rope(lib, mag=x, **none) == INVALID and rope(lib, eps=x, **none) == INVALID
