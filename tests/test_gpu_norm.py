"""Residual addition, RMS norm and int8 output against the oracle.

Sums are fp32 with one rounding, the norm is fp64 rounded once to fp32 and
the codes follow from correctly rounded divisions, so everything is compared
for equality: an fp64 value would have to lie within 2^-50 of a border between
two fp32 numbers to differ."""
import numpy as np
import pytest

from oracle import decode

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from packed_bit_gemv_tern_amd import tern  # noqa: E402
from gpu_util import DEV, to_dev  # noqa: E402


def rows(kind, M, K, rng):
    x = rng.normal(0, 1, (M, K))
    if kind == "outliers":
        x[:, ::17] *= 30
    elif kind == "zeros":
        x[:] = 0
    elif kind == "tiny":
        x *= 1e-24
    elif kind == "large":
        x *= 1e18
    elif kind == "positive":
        x = np.abs(x) + 0.5
    return x.astype(np.float32)


def padded(a, extra, shift=0):
    """A device copy of `a` with row stride K + extra, its first element
    `shift` floats past a 16-byte border; the view and its stride."""
    M, K = a.shape
    buf = torch.full((M * (K + extra) + shift + 4,), 7.5, dtype=torch.float32, device=DEV)
    view = buf[shift: shift + M * (K + extra)].reshape(M, K + extra)
    view[:, :K] = to_dev(a)
    return view


def check(M, K, kind="outliers", with_res=True, with_h=True, extra=0, shift=0, in_place=None, eps=1e-6):
    rng = np.random.default_rng([M, K, len(kind), with_res, extra])
    x, res = rows(kind, M, K, rng), rows("normal", M, K, rng) if with_res else None
    if kind in ("zeros", "tiny") and with_res:
        res *= 0
    gain = rng.uniform(-1.5, 1.5, K).astype(np.float32)
    rh, rq, rs, rz = decode.rmsnorm_quantize(x, res, gain, eps)
    xd = padded(x, extra, shift)
    rd = padded(res, extra, shift) if with_res else None
    ld = K + extra
    h = {None: padded(np.zeros((M, K), np.float32), extra, shift) if with_h else None, "x": xd, "res": rd}[in_place]
    ldq = (K + 15) // 16 * 16 + 16
    q = torch.full((M, ldq), 55, dtype=torch.int8, device=DEV)
    s, z = torch.empty(M, device=DEV), torch.empty(M, dtype=torch.int32, device=DEV)
    tern.tern_rmsnorm_quantize(xd, to_dev(gain), eps, M, K, ld, q, ldq, s, z, res=rd, ldr=ld if with_res else 0,
                               h=h, ldh=ld if h is not None else 0)
    torch.cuda.synchronize()
    qh = q.cpu().numpy()
    assert np.array_equal(qh[:, :K], rq)
    assert (qh[:, K:] == 55).all()
    assert np.array_equal(s.cpu().numpy().view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(z.cpu().numpy(), rz)
    if h is not None:
        hh = h.cpu().numpy()
        assert np.array_equal(hh[:, :K].view(np.uint32), rh.view(np.uint32))
        assert (hh[:, K:] == 7.5).all()
    if in_place != "x":
        assert np.array_equal(xd.cpu().numpy()[:, :K], x)


# one column, one token, both models' widths, odd widths, each register variant and the long rows
@pytest.mark.parametrize("M,K", [(1, 1), (2, 3), (1, 1024), (1, 4096), (3, 100), (37, 1019), (5, 4097), (4, 8192),
                                 (2, 12288), (2, 16384), (2, 16385), (1, 50001), (700, 1024), (300, 4096), (65, 2050)])
@pytest.mark.parametrize("with_res", [True, False])
def test_norm_sizes(M, K, with_res):
    check(M, K, with_res=with_res)


@pytest.mark.parametrize("kind", ["normal", "outliers", "zeros", "tiny", "large", "positive"])
@pytest.mark.parametrize("K", [512, 777, 20000])
def test_norm_values(kind, K):
    check(3, K, kind=kind)
    check(3, K, kind=kind, with_res=False, with_h=False)


# strides and alignments that take the element-by-element variant, and that do not
@pytest.mark.parametrize("extra,shift", [(4, 0), (3, 0), (0, 1), (5, 3), (4, 2)])
@pytest.mark.parametrize("M,K", [(1, 256), (9, 256), (9, 4096), (3, 5000)])
def test_norm_strides(M, K, extra, shift):
    check(M, K, extra=extra, shift=shift)


@pytest.mark.parametrize("K", [64, 1001, 4096, 17000])
@pytest.mark.parametrize("in_place", ["x", "res"])
def test_norm_in_place(K, in_place):
    check(5, K, in_place=in_place)
    check(5, K, in_place=in_place, extra=3)


@pytest.mark.parametrize("K", [5, 1024, 3000, 4096, 20000])
@pytest.mark.parametrize("M", [2, 300])
def test_norm_of_a_sum_that_is_not_kept(M, K):
    check(M, K, with_h=False)


def test_norm_eps_counts():
    check(2, 300, kind="tiny", eps=1e-3)
    check(2, 300, kind="normal", eps=2.0)
