"""Calls at the borders of the lookup's, rotation's, epilogue's and pages' checks:
status codes before any launch (no GPU needed: nothing below gets past them)."""

from packed_bit_gemv_tern_amd import tern
from test_abi_step import A16, ALIGN, INVALID, ODD2, OK, WORKSPACE, compact, lib, pool  # noqa: F401


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
