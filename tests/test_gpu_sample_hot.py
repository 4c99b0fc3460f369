"""Rows whose cut falls among thousands of close logits, as of a hot temperature
over a large vocabulary: more tokens in one bin of the histogram than the list
holds, without a single tie."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
pytest.importorskip("torch")
from test_gpu_sample import draw  # noqa: E402

LIST = 2048  # tokens that are ordered at once


def listed(x, T, k, p):
    """Tokens in the bins (3/64 of an octave below the maximum) that the cuts
    fall in: that of the k-th token where it is split, and those in which top-p may
    end, for any part of that bin's weight."""
    v = (x.max() - x.astype(np.float64)) / T
    b = np.minimum(np.rint(v * 64 / np.log(2)) // 3, 1023).astype(int)
    n, m = np.bincount(b, minlength=1024), np.bincount(b, weights=np.exp(-v), minlength=1024)
    run, mass = np.cumsum(n), np.cumsum(m)
    kb = int(np.searchsorted(run, k or len(x)))
    split = run[kb] > (k or len(x))
    bins = {kb} if split else set()
    if p is not None:
        first = np.searchsorted(mass, p * (mass[kb] - m[kb] * split))
        bins |= set(range(int(first), int(np.searchsorted(mass, p * mass[kb])) + 1))
    return sum(n[i] for i in bins)


@pytest.mark.parametrize("M,N,sd,T,k,p", [
    (1, 151936, 2.2, 1.5, 50000, 0.9), (1, 151936, 2.2, 2.0, 20000, 0.95), (1, 262144, 2.2, 1.5, None, 0.95),
    (1, 524288, 2.2, 1.0, None, 0.95), (3, 151936, 1.5, 2.0, None, 0.9), (3, 151936, 1.0, 1.5, None, 0.8),
    (4, 151936, 1.0, 2.0, 60000, None), (3, 200003, 1.5, 2.0, 60000, 0.9)])
@pytest.mark.parametrize("min_p", [None, 0.02])
def test_close_logits_at_the_cut(M, N, sd, T, k, p, min_p):
    rng = np.random.default_rng([M, N, int(10 * T)])
    x = rng.normal(0, sd, (M, N)).astype(np.float32)
    args = {"top_k": None if k is None else [k + i for i in range(M)], "top_p": None if p is None else [p] * M}
    u = rng.random(M)
    if min_p is None:
        assert all(listed(x[i], T, k and k + i, p) > LIST for i in range(M))
        draw(x, [T] * M, u, **args)
    else:
        draw(x, [T] * M, u, min_p=[min_p] * M, **args)
