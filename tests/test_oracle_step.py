"""Pins of the plain forms in oracle/step.py: closed forms and invariants."""
import numpy as np
import pytest

from oracle import step


def test_embed_rows():
    W = np.array([[1, -2, 127], [0, 5, -127]], np.int8)
    out = step.embed(W, np.array([0.5, 0.25], np.float32), [1, -1, 0, 2], 2.0)
    assert out.tolist() == [[0.0, 2.5, -63.5], [0, 0, 0], [1, -2, 127], [0, 0, 0]]


def test_rotation_depends_on_distances_only():
    """Scores of rotated rows are those of the distance; a rotation keeps the norm."""
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 64)).astype(np.float32)
    f = (1e4 ** (-np.arange(32) / 32)).astype(np.float32)
    at = lambda x, p: step.norm_rope(x, None, 1e-6, p, f, 1.0)[0]  # noqa: E731
    near = at(q, 7) @ at(k, 3)
    for far in (0, 100, 10 ** 6):
        # (angles of 10^6 carry 2^-33 each, for 64 terms of a few units)
        assert abs(at(q, far + 7) @ at(k, far + 3) - near) < 1e-6
    assert abs(np.linalg.norm(at(q, 12345)) - np.linalg.norm(q.astype(np.float64))) < 1e-9
    assert np.array_equal(at(q, 0), q.astype(np.float64))


def test_norm_before_the_rotation():
    x = np.array([3.0] * 64, np.float32)
    y, _ = step.norm_rope(x, np.full(64, 2, np.float32), 1e-6, 0, np.zeros(0, np.float32), 1.0)
    assert np.allclose(y, 2.0, atol=1e-6)


def test_positions():
    assert step.positions([0, 2, 3, 3, 6], [10, 0, 4, 3], 8, 2) == [8, 9, None, 0, 1, None, None, None]
    assert step.positions([0, 9], [9], 8, 9) == [None] * 8


def test_gelu_against_64_bits():
    x = np.linspace(-12, 12, 4001).astype(np.float32)
    d = x.astype(np.float64)
    t = np.sqrt(2 / np.pi) * (d + 0.044715 * d ** 3)
    ref = d / (1 + np.exp(-2 * t))
    # e^(-2t): the argument is off by 4 roundings, |2t| 2^-24 each, the exp by 1.5 ulp; two more roundings;
    # where e^(-2t) passes 2^128 the result is 0 and |ref| below 12 / 2^128 < 2^-124
    tol = np.abs(ref) * (4 * np.abs(2 * t) + 3 + 2 + 1) * 2.0 ** -24 + 2.0 ** -124
    assert (np.abs(step.gelu(x) - ref) <= tol).all()


def check_pool(p, length):
    """refs count the entries of the held tokens."""
    n = [0] * len(p.refs)
    for s in range(len(p.table)):
        for j in range(p.count(length[s])):
            if p.page(s, j) is not None:
                n[p.page(s, j)] += 1
    assert n == p.refs


@pytest.mark.parametrize("seed", range(6))
def test_pool_keeps_its_counts_and_contents(seed):
    """Random forks, steps, ends and compactions: refs count entries, and every
    sequence finds its own tokens in its pages."""
    rng = np.random.default_rng(seed)
    S, P, columns, pages = 6, 16, 8, 30
    p = step.Pool(pages, S, columns, P, rng)
    length = [0] * S
    content = {}  # page -> {place: token}
    tokens = [[] for _ in range(S)]
    stamp = 0
    for _ in range(60):
        what = rng.integers(4)
        if what == 0:
            empty = [s for s in range(S) if not length[s]]
            if empty and max(length):
                a = int(np.argmax(length))
                p.fork(length, [a], [empty[0]])
                length[empty[0]], tokens[empty[0]] = length[a], list(tokens[a])
        elif what == 1:
            want = [n + int(rng.integers(0, 20)) for n in length]
            granted, src, dst = p.reserve(length, want)
            assert all(p.refs[b] == 1 for b in dst if b >= 0)
            for a, b in zip(src, dst):
                if b >= 0:
                    content[b] = dict(content[a])
            for s in range(S):
                if granted[s]:
                    for n in range(length[s], want[s]):
                        stamp += 1
                        tokens[s].append(stamp)
                        page = p.page(s, n // P)
                        assert p.refs[page] == 1
                        if n % P == 0:
                            content[page] = {}
                        content[page][n % P] = stamp
                    length[s] = max(length[s], want[s])
        elif what == 2:
            keep = [int(rng.integers(0, n + 2)) if rng.integers(2) else n for n in length]
            p.truncate(length, keep)
            length = [min(n, k) for n, k in zip(length, keep)]
            tokens = [t[:n] for t, n in zip(tokens, length)]
        else:
            src, dst, live = p.compact(length, int(rng.integers(0, pages // 2 + 1)))
            for a, b in zip(src, dst):
                if a >= 0:
                    content[b] = content.pop(a)
            assert live == sum(n > 0 for n in p.refs)
        check_pool(p, length)
        for s in range(S):
            assert [content[p.page(s, n // P)][n % P] for n in range(length[s])] == tokens[s]
    src, dst, live = p.compact(length, pages // 2)
    assert all(n > 0 for n in p.refs[:live]) and not any(p.refs[live:])
