"""Refusals of the norm, cache, attention and sampling calls: status codes
before any launch (no GPU needed: nothing below gets past the checks)."""
import pytest

from packed_bit_gemv_tern_amd import tern

A16, ODD8, ODD2 = 0x10000, 0x10008, 0x10002  # fake device addresses, never dereferenced
OK, INVALID, ALIGN, RANGE = tern.TERN_OK, tern.TERN_ERR_INVALID_ARG, tern.TERN_ERR_ALIGNMENT, tern.TERN_ERR_RANGE
UNSUPPORTED, WORKSPACE = tern.TERN_ERR_UNSUPPORTED, tern.TERN_ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return tern.library()


def norm(lib, x=A16, ldx=64, res=A16, ldr=64, gain=A16, eps=1e-6, M=2, K=64, h=A16, ldh=64, q=A16, ldq=64, s=A16,
         z=A16):
    return lib.tern_rmsnorm_quantize(x, ldx, res, ldr, gain, eps, M, K, h, ldh, q, ldq, s, z, None)


def test_norm_refusals(lib):
    for kw in ({"K": 0}, {"M": -1}, {"ldx": 63}, {"ldr": 63}, {"ldh": 63}, {"ldq": 63}, {"eps": 0.0}, {"eps": -1.0},
               {"eps": NAN}, {"eps": INF}, {"x": None}, {"gain": None}, {"q": None}, {"s": None}, {"z": None}):
        assert norm(lib, **kw) == INVALID, kw
    for kw in ({"q": ODD8}, {"ldq": 72}, {"x": ODD2}, {"res": ODD2}, {"gain": ODD2}, {"h": ODD2}, {"s": ODD2},
               {"z": ODD2}):
        assert norm(lib, **kw) == ALIGN, kw
    big = tern.TERN_MAX_K + 1
    assert norm(lib, K=big, ldx=big, ldr=big, ldh=big, ldq=big + 15) == RANGE
    assert norm(lib, M=2 ** 32) == RANGE
    assert norm(lib, M=0, x=None, q=None) == OK


def cache(**kw):
    d = dict(k=A16, v=A16, k_scale=A16, v_scale=A16, pages=8, heads=2, head_dim=64, page_tokens=16)
    return tern.tern_kv_cache(*{**d, **kw}.values())


def batch(**kw):
    d = dict(table=A16, ld_table=4, start=A16, len=A16, S=2, rows=2, max_new=1, max_len=0)
    return tern.tern_kv_batch(*{**d, **kw}.values())


def append(lib, c, b, k=A16, ldk=128, v=A16, ldv=128):
    return lib.tern_kv_append(c, b, k, ldk, v, ldv, None)


def attend(lib, c, b, q=A16, ldq=256, q_heads=4, scale=0.125, y=A16, ldy=256, ws=A16, n=1 << 30):
    return lib.tern_attention(c, b, q, ldq, q_heads, scale, y, ldy, ws, n, None)


CACHE = [({"pages": -1}, INVALID), ({"pages": 0}, INVALID), ({"heads": 0}, INVALID), ({"head_dim": 96}, UNSUPPORTED),
         ({"head_dim": 0}, UNSUPPORTED), ({"page_tokens": 8}, UNSUPPORTED), ({"page_tokens": 48}, UNSUPPORTED),
         ({"page_tokens": 256}, UNSUPPORTED), ({"pages": 2 ** 31}, RANGE), ({"k": None}, INVALID),
         ({"v": None}, INVALID), ({"k_scale": None}, INVALID), ({"v_scale": None}, INVALID), ({"k": ODD8}, ALIGN),
         ({"v": ODD8}, ALIGN), ({"k_scale": ODD2}, ALIGN), ({"v_scale": ODD2}, ALIGN)]
BATCH = [({"S": -1}, INVALID), ({"rows": -1}, INVALID), ({"max_new": -1}, INVALID), ({"max_len": -1}, INVALID),
         ({"ld_table": -1}, INVALID), ({"ld_table": 0}, INVALID), ({"table": None}, INVALID),
         ({"start": None}, INVALID), ({"len": None}, INVALID), ({"table": ODD2}, ALIGN), ({"start": ODD2}, ALIGN),
         ({"len": ODD2}, ALIGN), ({"ld_table": tern.TERN_KV_MAX_LEN // 16 + 1}, RANGE), ({"rows": 2 ** 31}, RANGE),
         ({"S": 2 ** 31}, RANGE)]


@pytest.mark.parametrize("call", [append, attend])
def test_cache_and_batch_refusals(lib, call):
    for kw, status in CACHE:
        assert call(lib, cache(**kw), batch()) == status, kw
    for kw, status in BATCH:
        assert call(lib, cache(), batch(**kw)) == status, kw
    assert call(lib, None, batch()) == INVALID and call(lib, cache(), None) == INVALID
    for kw in ({"S": 0, "start": None, "len": None}, {"rows": 0}, {"max_new": 0, "table": None}):
        assert call(lib, cache(k=None), batch(**kw)) == OK, kw
    # a launch counts its work-items in 32 bits
    assert call(lib, cache(), batch(S=2 ** 27, rows=2 ** 30, max_new=64)) == RANGE


def test_append_refusals(lib):
    for kw in ({"k": None}, {"v": None}, {"ldk": 127}, {"ldv": 127}):
        assert append(lib, cache(), batch(), **kw) == INVALID, kw
    assert append(lib, cache(), batch(), k=ODD2) == ALIGN
    assert append(lib, cache(), batch(), v=ODD2) == ALIGN


def test_attention_refusals(lib):
    for kw in ({"q": None}, {"y": None}, {"ldq": 255}, {"ldy": 255}, {"q_heads": 0}, {"q_heads": 3},
               {"q_heads": -2}, {"scale": NAN}, {"scale": INF}, {"scale": -INF}):
        assert attend(lib, cache(), batch(), **kw) == INVALID, kw
    assert attend(lib, cache(), batch(), q_heads=2 ** 17) == RANGE
    assert attend(lib, cache(), batch(), q=ODD2) == ALIGN
    assert attend(lib, cache(), batch(), y=ODD2) == ALIGN
    c, b = cache(), batch()
    assert lib.tern_attention_workspace_bytes(None, b, 4) == 0
    assert lib.tern_attention_workspace_bytes(c, None, 4) == 0
    assert lib.tern_attention_workspace_bytes(c, b, 3) == 0
    assert lib.tern_attention_workspace_bytes(cache(head_dim=80), b, 4) == 0


def sample(lib, x=A16, M=2, N=100, ldl=100, T=A16, u=A16, k=A16, p=A16, mp=A16, token=A16, prob=A16, kept=A16, ws=A16,
           n=1 << 40):
    return lib.tern_sample(x, M, N, ldl, T, u, k, p, mp, token, prob, kept, ws, n, None)


def test_sample_refusals(lib):
    for kw in ({"M": -1}, {"N": 0}, {"ldl": 99}, {"x": None}, {"T": None}, {"u": None}, {"token": None}):
        assert sample(lib, **kw) == INVALID, kw
    for field in ("x", "T", "u", "k", "p", "mp", "token", "prob", "kept"):
        assert sample(lib, **{field: ODD2}) == ALIGN, field
    assert sample(lib, N=tern.TERN_SAMPLE_MAX_N + 1, ldl=2 ** 20) == RANGE
    assert sample(lib, M=2 ** 32) == RANGE
    assert sample(lib, M=0, x=None, token=None) == OK
    assert lib.tern_sample_workspace_bytes(-1, 100) == 0
    assert lib.tern_sample_workspace_bytes(4, tern.TERN_SAMPLE_MAX_N + 1) == 0


def test_sizes_that_do_not_fit_64_bits(lib):
    """Row counts whose work-items pass 2^64 are refused too."""
    assert norm(lib, M=2 ** 54 + 1) == RANGE
    for M in (2 ** 44, 2 ** 54 + 1, 2 ** 62):
        assert sample(lib, M=M) == RANGE
        assert lib.tern_sample_workspace_bytes(M, 151936) == 0
