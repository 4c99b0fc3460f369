"""The norm and rotation of queries and keys against the oracle's fp64."""
import numpy as np
import pytest

from oracle import step
from packed_bit_gemv_tern_amd import tern

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from gpu_util import DEV, to_dev  # noqa: E402


def freqs(R, base=1e6):
    return (base ** (-np.arange(R // 2) / max(R // 2, 1))).astype(np.float32)


def run(new, length, Hq, H, D, R, gains=True, extra=0, max_new=None, magnitude=1.0, in_place=False, seed=0, start=None,
        rows=None, shift=0, f=None, x=None):
    rng = np.random.default_rng([Hq, H, D, R, seed])
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32) if start is None else np.asarray(start, np.int32)
    length = np.asarray(length, np.int32)
    rows = int(start[-1]) if rows is None else rows
    max_new = max(new) if max_new is None else max_new
    f = freqs(R) if f is None else f
    keep = to_dev(start), to_dev(length)
    b = tern.make_kv_batch(None, 0, keep[0], keep[1], len(length), rows, max_new)
    host, dev, outs, args = {}, {}, {}, {}
    for name, heads in (("q", Hq), ("k", H)):
        ld = heads * D + extra
        host[name] = (3 * rng.standard_normal((rows, ld))).astype(np.float32) if x is None else x(name, rows, ld)
        dev[name] = torch.empty(rows * ld + 4, device=DEV)[shift: shift + rows * ld].view(rows, ld)
        dev[name].copy_(torch.from_numpy(host[name]))
        outs[name] = dev[name] if in_place else torch.full((rows * ld + 4,), 7.0, device=DEV)[
            shift: shift + rows * ld].view(rows, ld)
        host[name + "_gain"] = rng.uniform(0.5, 1.5, D).astype(np.float32) if gains else None
        dev[name + "_gain"] = to_dev(host[name + "_gain"]) if gains else None
        args.update({name: dev[name], "ld" + name: ld, name + "_out": outs[name], "ld" + name + "o": ld,
                     name + "_gain": dev[name + "_gain"]})
    tern.tern_qk_norm_rope(b, D, to_dev(f) if R else None, R, q_heads=Hq, heads=H, eps=1e-6, magnitude=magnitude, **args)
    places = step.positions(start, length, rows, max_new)
    for name, heads in (("q", Hq), ("k", H)):
        got = outs[name].cpu().numpy().astype(np.float64)
        ref = host[name].astype(np.float64) if in_place else np.full(got.shape, 7.0)
        tol = np.zeros(got.shape)
        for r, p in enumerate(places):
            for h in range(heads if p is not None else 0):
                at = slice(h * D, (h + 1) * D)
                y, size = step.norm_rope(host[name][r, at], host[name + "_gain"], 1e-6, p, f, magnitude)
                ref[r, at] = y
                # one rounding to fp32 (2^-24 of the value, or half the smallest subnormal), and fp64 steps on
                # sines and cosines good to 2^-44
                tol[r, at] = 2.0 ** -24 * np.abs(y) + 2.0 ** -42 * size + 2.0 ** -150
        assert (np.abs(got - ref) <= tol).all(), name
    return outs


@pytest.mark.parametrize("D,R", [(64, 64), (128, 128), (128, 64), (64, 32), (128, 8), (64, 40), (128, 120), (64, 0)])
@pytest.mark.parametrize("Hq,H", [(4, 1), (5, 5), (32, 8), (3, 0), (0, 2)])
def test_heads_and_parts(Hq, H, D, R):
    run([1, 5, 1], [9, 5, 1], Hq, H, D, R, magnitude=1.25 if R else 1.0)


@pytest.mark.parametrize("gains", [True, False])
@pytest.mark.parametrize("in_place", [True, False])
def test_in_place_strides_and_alignment(gains, in_place):
    for extra, shift in ((0, 0), (4, 0), (3, 0), (0, 1), (64, 2)):
        run([3, 2], [3, 70], 6, 2, 128, 128, gains=gains, in_place=in_place, extra=extra, shift=shift)


def test_far_positions():
    """Positions to the longest cache: angles in fp32 would be off by turns."""
    far = [1000003, 131072, 2 ** 24 + 1, 2 ** 30, 2 ** 31 - 1]
    run([2] * 5, far, 2, 2, 128, 128)
    run([2] * 5, far, 2, 2, 64, 64, f=np.linspace(0.9, 1.0, 32).astype(np.float32))
    run([2] * 5, far, 2, 2, 64, 64, f=-np.linspace(0.1, 1.0, 32).astype(np.float32), gains=False)


def test_rows_without_a_place():
    """Idle slots, lengths shorter than the new rows, rows past max_new, rows of
    no sequence, sequences whose rows leave the buffers."""
    for in_place in (False, True):
        run([1, 4, 1], [0, 2, -5], 4, 2, 64, 64, in_place=in_place)
        run([7, 3], [7, 9], 4, 2, 64, 64, max_new=4, in_place=in_place)
        run([0], [9, 9, 9, 30], 4, 2, 64, 64, start=[2, 4, 4, 3, 12], rows=9, max_new=9, in_place=in_place)
        run([0], [9, 9, 9], 4, 2, 64, 64, start=[-1, 4, 2, 6], rows=9, max_new=9, in_place=in_place)


def test_many_sequences_and_rows():
    new = [1 + (i % 3) for i in range(700)]
    run(new, [n + 13 * i for i, n in enumerate(new)], 2, 1, 64, 64)
    run([600], [600], 9, 3, 128, 128)


def test_values_at_the_ends_of_the_range():
    """Squares past fp32, zeros and tiny rows under the norm; a row of NaN or
    infinities spoils itself alone."""
    def x(name, rows, ld):
        v = np.ones((rows, ld), np.float32)
        v[0] *= 1e30
        v[1] = 0
        v[2] *= 1e-30
        v[3, ::2] = -3e38
        return v
    run([5], [5], 2, 2, 64, 64, x=x)
    rng = np.random.default_rng(0)
    a = rng.standard_normal((3, 128)).astype(np.float32)
    outs = []
    for bad in (np.nan, np.inf, 1.0):
        v = a.copy()
        v[1, 5] = bad
        t = to_dev(v)
        keep = to_dev(np.array([0, 3], np.int32)), to_dev(np.array([9], np.int32))
        b = tern.make_kv_batch(None, 0, *keep, 1, 3, 3)
        tern.tern_qk_norm_rope(b, 64, to_dev(freqs(64)), 64, q=t, ldq=128, q_heads=2, q_out=t, ldqo=128,
                               q_gain=to_dev(np.ones(64, np.float32)))
        outs.append(t.cpu().numpy())
    good = outs[2]
    for o in outs[:2]:
        assert np.isnan(o[1, :64]).any()
        assert np.array_equal(np.delete(o, 1, 0), np.delete(good, 1, 0)) and np.array_equal(o[1, 64:], good[1, 64:])
