"""Refusals of the embedding, rotation, epilogue and page calls: status codes
before any launch (no GPU needed: nothing below gets past the checks)."""
import ctypes

import pytest

from packed_bit_gemv_tern_amd import tern

A16, ODD8, ODD2 = 0x10000, 0x10008, 0x10002  # fake device addresses, never dereferenced
OK, INVALID, ALIGN, RANGE = tern.TERN_OK, tern.TERN_ERR_INVALID_ARG, tern.TERN_ERR_ALIGNMENT, tern.TERN_ERR_RANGE
UNSUPPORTED, WORKSPACE = tern.TERN_ERR_UNSUPPORTED, tern.TERN_ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return tern.library()


def embed(lib, W=A16, s_row=A16, N=100, K=64, ldw=64, ids=A16, M=2, scale=1.0, x=A16, ldx=64):
    return lib.tern_embed(W, s_row, N, K, ldw, ids, M, scale, x, ldx, None)


def test_embed_refusals(lib):
    for kw in ({"N": 0}, {"K": 0}, {"M": -1}, {"ldw": 63}, {"ldx": 63}, {"scale": NAN}, {"scale": INF}, {"scale": -INF},
               {"W": None}, {"s_row": None}, {"ids": None}, {"x": None}):
        assert embed(lib, **kw) == INVALID, kw
    for field in ("s_row", "ids", "x"):
        assert embed(lib, **{field: ODD2}) == ALIGN, field
    big = tern.TERN_MAX_K + 1
    for kw in ({"N": 2 ** 31}, {"K": big, "ldw": big, "ldx": big}, {"M": 2 ** 40}, {"M": 2 ** 62}):
        assert embed(lib, **kw) == RANGE, kw
    assert embed(lib, M=0, W=None, x=None) == OK


def batch(**kw):
    d = dict(table=None, ld_table=0, start=A16, len=A16, S=2, rows=2, max_new=1, max_len=0)
    return tern.tern_kv_batch(*{**d, **kw}.values())


def rope(lib, b=None, D=64, freq=A16, R=64, mag=1.0, q=A16, ldq=256, hq=4, qg=A16, qo=A16, ldqo=256, k=A16, ldk=128, h=2,
         kg=A16, ko=A16, ldko=128, eps=1e-6):
    return lib.tern_qk_norm_rope(batch() if b is None else b, D, freq, R, mag, q, ldq, hq, qg, qo, ldqo, k, ldk, h, kg, ko,
                                 ldko, eps, None)


def test_rope_refusals(lib):
    for kw in ({"hq": -1}, {"h": -1}, {"eps": 0.0}, {"eps": -1.0}, {"eps": NAN}, {"eps": INF}, {"mag": NAN},
               {"mag": INF}, {"ldq": 255}, {"ldqo": 255}, {"ldk": 127}, {"ldko": 127}, {"freq": None}, {"q": None},
               {"qo": None}, {"k": None}, {"ko": None}, {"b": batch(S=-1)}, {"b": batch(rows=-1)},
               {"b": batch(max_new=-1)}, {"b": batch(start=None)}, {"b": batch(len=None)}):
        assert rope(lib, **kw) == INVALID, kw
    for kw in ({"D": 96}, {"D": 0}, {"R": 72}, {"R": -8}, {"R": 4}, {"D": 128, "R": 136}):
        assert rope(lib, **kw) == UNSUPPORTED, kw
    for kw in ({"freq": ODD2}, {"q": ODD2}, {"qo": ODD2}, {"k": ODD2}, {"ko": ODD2}, {"qg": ODD2}, {"kg": ODD2},
               {"b": batch(start=ODD2)}, {"b": batch(len=ODD2)}):
        assert rope(lib, **kw) == ALIGN, kw
    for kw in ({"b": batch(rows=2 ** 31)}, {"b": batch(S=2 ** 31)}, {"b": batch(max_new=2 ** 31)},
               {"b": batch(rows=2 ** 30)}, {"hq": 2 ** 17, "ldq": 2 ** 30, "ldqo": 2 ** 30}):
        assert rope(lib, **kw) == RANGE, kw
    assert lib.tern_qk_norm_rope(None, 64, A16, 64, 1.0, A16, 256, 4, A16, A16, 256, A16, 128, 2, A16, A16, 128, 1e-6,
                                 None) == INVALID
    for kw in ({"b": batch(S=0, start=None)}, {"b": batch(rows=0)}, {"b": batch(max_new=0)},
               {"h": 0, "hq": 0, "q": None, "k": None}):
        assert rope(lib, **kw) == OK, kw


def weights(**kw):
    d = dict(packed=A16, s_row=A16, rowsum=A16, bias=A16)
    return tern.tern_weights(*{**d, **kw}.values())


def linear(lib, w=None, up=None, N=32, K=64, M=2, q=A16, ldq=64, s=A16, z=A16, act=0, res=A16, ldr=32, y=A16, ldy=32):
    return lib.tern_linear_epilogue(weights() if w is None else w, up, N, K, M, q, ldq, s, z, act, res, ldr, y, ldy, None)


def test_linear_epilogue_refusals(lib):
    for field in ("packed", "s_row", "rowsum"):
        assert linear(lib, w=weights(**{field: None})) == INVALID, field
        assert linear(lib, up=weights(**{field: None})) == INVALID, field
    for kw in ({"N": -1}, {"M": -1}, {"K": 0}, {"ldq": 63}, {"ldy": 31}, {"ldr": 31}, {"act": -1}, {"act": 3},
               {"q": None}, {"s": None}, {"z": None}, {"y": None}):
        assert linear(lib, **kw) == INVALID, kw
    for kw in ({"q": ODD8}, {"ldq": 72}, {"s": ODD2}, {"z": ODD2}, {"y": ODD2}, {"res": ODD2}):
        assert linear(lib, **kw) == ALIGN, kw
    for field, bad in (("packed", ODD8), ("s_row", ODD2), ("rowsum", ODD2), ("bias", ODD2)):
        assert linear(lib, w=weights(**{field: bad})) == ALIGN, field
        assert linear(lib, up=weights(**{field: bad})) == ALIGN, field
    big = tern.TERN_MAX_K + 1
    for kw in ({"K": big, "ldq": big + 15}, {"N": 2 ** 31, "ldy": 2 ** 31, "ldr": 2 ** 31}, {"M": 2 ** 31},
               {"N": 2 ** 30, "M": 2 ** 20, "ldy": 2 ** 30, "ldr": 2 ** 30}):
        assert linear(lib, **kw) == RANGE, kw
    assert lib.tern_linear_epilogue(None, None, 32, 64, 2, A16, 64, A16, A16, 0, None, 0, A16, 32, None) == INVALID
    assert linear(lib, M=0, q=None, y=None) == OK and linear(lib, N=0, w=weights(packed=None)) == OK


def pool(**kw):
    d = dict(refs=A16, table=A16, pages=64, ld_table=8, S=3, page_tokens=16)
    return tern.tern_kv_pool(*{**d, **kw}.values())


def fork(lib, p, length=A16, src=A16, dst=A16, n=2):
    return lib.tern_kv_fork(p, length, src, dst, n, None)


def truncate(lib, p, length=A16, keep=A16):
    return lib.tern_kv_truncate(p, length, keep, None)


def reserve(lib, p, length=A16, want=A16, granted=A16, src=A16, dst=A16, ws=A16, n=1 << 30):
    return lib.tern_kv_reserve(p, length, want, granted, src, dst, ws, n, None)


def compact(lib, p, length=A16, src=A16, dst=A16, moves=32, live=A16, ws=A16, n=1 << 30):
    return lib.tern_kv_compact(p, length, src, dst, moves, live, ws, n, None)


@pytest.mark.parametrize("call", [fork, truncate, reserve, compact])
def test_pool_refusals(lib, call):
    for kw, status in (({"pages": -1}, INVALID), ({"S": -1}, INVALID), ({"ld_table": -1}, INVALID),
                       ({"refs": None}, INVALID), ({"table": None}, INVALID), ({"refs": ODD2}, ALIGN),
                       ({"table": ODD2}, ALIGN), ({"page_tokens": 8}, UNSUPPORTED), ({"page_tokens": 24}, UNSUPPORTED),
                       ({"page_tokens": 256}, UNSUPPORTED), ({"pages": 2 ** 31}, RANGE), ({"S": 2 ** 31}, RANGE),
                       ({"S": 2 ** 25}, RANGE), ({"ld_table": tern.TERN_KV_MAX_LEN // 16 + 1}, RANGE)):
        assert call(lib, pool(**kw)) == status, kw
    assert call(lib, None) == INVALID
    assert call(lib, pool(S=0, refs=None)) == OK
    for name in call.__code__.co_varnames[2: call.__code__.co_argcount]:
        if name not in ("n", "moves", "ws"):
            assert call(lib, pool(), **{name: None}) == INVALID, name
            assert call(lib, pool(), **{name: ODD2}) == ALIGN, name


def test_pool_sizes_and_workspaces(lib):
    assert fork(lib, pool(), n=-1) == INVALID and fork(lib, pool(), n=2 ** 40) == RANGE
    assert fork(lib, pool(), n=0, src=None) == OK
    assert compact(lib, pool(), moves=-1) == INVALID and compact(lib, pool(), moves=2 ** 31) == RANGE
    for call in (reserve, compact):
        assert call(lib, pool(pages=0)) == INVALID and call(lib, pool(ld_table=0)) == INVALID
        for kw in ({"ws": None}, {"ws": A16 + 16}, {"n": 64}):
            assert call(lib, pool(), **kw) == WORKSPACE, kw
    for call in (fork, truncate):
        assert call(lib, pool(pages=0, refs=None)) == OK
    size = lib.tern_kv_pool_workspace_bytes
    assert size(pool()) >= 256 and size(pool(pages=10 ** 6)) >= 4 * 10 ** 6 and size(pool(S=10 ** 5)) >= 4 * 10 ** 5
    assert size(pool(page_tokens=20)) == 0 and size(None) == 0


def layers(n=2, **kw):
    d = dict(k=A16, v=A16, k_scale=A16, v_scale=A16, pages=8, heads=2, head_dim=64, page_tokens=16)
    return (tern.tern_kv_cache * n)(*[tern.tern_kv_cache(*{**d, **(kw if i == n - 1 else {})}.values()) for i in range(n)])


def copy(lib, dst=None, src=None, n_layers=2, a=A16, b=A16, n=3):
    return lib.tern_kv_copy(layers() if dst is None else dst, layers() if src is None else src, n_layers, a, b, n, None)


def test_copy_refusals(lib):
    for kw in ({"n_layers": -1}, {"n": -1}, {"a": None}, {"b": None}):
        assert copy(lib, **kw) == INVALID, kw
    for kw in ({"heads": 3}, {"head_dim": 128}, {"page_tokens": 32}, {"pages": 9}, {"k": None}, {"v": None},
               {"k_scale": None}, {"v_scale": None}, {"heads": 0}):
        assert copy(lib, dst=layers(**kw)) == INVALID and copy(lib, src=layers(**kw)) == INVALID, kw
    for kw in ({"k": ODD8}, {"v": ODD8}, {"k_scale": ODD2}, {"v_scale": ODD2}):
        assert copy(lib, dst=layers(**kw)) == ALIGN and copy(lib, src=layers(**kw)) == ALIGN, kw
    assert copy(lib, a=ODD2) == ALIGN and copy(lib, b=ODD2) == ALIGN
    for kw in ({"head_dim": 80}, {"page_tokens": 48}):
        assert copy(lib, dst=layers(1, **kw), src=layers(1, **kw), n_layers=1) == UNSUPPORTED, kw
    assert copy(lib, n=2 ** 40) == RANGE and copy(lib, n=2 ** 62) == RANGE
    assert copy(lib, n=0, a=None) == OK and copy(lib, n_layers=0) == OK
    none = ctypes.POINTER(tern.tern_kv_cache)()
    assert lib.tern_kv_copy(none, layers(), 2, A16, A16, 1, None) == INVALID
    assert lib.tern_kv_copy(layers(), none, 2, A16, A16, 1, None) == INVALID
    with pytest.raises(tern.TernError):
        tern.tern_kv_copy(tern.make_kv_layers(list(layers())), tern.make_kv_layers(list(layers(3))), None, None, 1, stream=0)
