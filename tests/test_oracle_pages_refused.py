"""The step over a pool of pages where rows are refused, on the oracle's lists: what
append would write into, and what truncate gives up."""
import numpy as np
import pytest

from oracle import step


def run(seed, idle):
    """Random steps of a pool that runs out; refused rows are idle slots (length 0) in
    append and truncate, or go on with the length that they wanted.  Returns the
    number of tokens written into pages that others hold, and of pages whose count is
    not that of the entries."""
    rng = np.random.default_rng(seed)
    S, P, columns, pages = 5, 16, 4, 9
    p = step.Pool(pages, S, columns, P, rng)
    length, shared, miscounted, refused = [0] * S, 0, 0, 0
    for _ in range(80):
        empty = [s for s in range(S) if not length[s]]
        if empty and max(length) and rng.integers(2):
            a = int(np.argmax(length))
            p.fork(length, [a], [empty[0]])
            length[empty[0]] = length[a]
        new = [int(n) for n in rng.integers(0, 9, S)]
        want = [n + m for n, m in zip(length, new)]
        granted, _, _ = p.reserve(length, want)
        now = [w if g or not idle else 0 for g, w in zip(granted, want)]
        refused += granted.count(0)
        for s in range(S):
            for t in range(max(now[s] - new[s], 0), now[s]):
                page = p.page(s, t // P) if t // P < columns else None
                shared += page is not None and p.refs[page] > 1
        kept = [w - int(rng.integers(0, m + 1)) for w, m in zip(want, new)]
        p.truncate(now, kept)
        length = [k if g else n for g, k, n in zip(granted, kept, length)]
        if rng.integers(3) == 0:
            s = int(rng.integers(S))
            p.truncate(length, [0 if i == s else n for i, n in enumerate(length)])
            length[s] = 0
        count = [0] * pages
        for s in range(S):
            for j in range(p.count(length[s])):
                if p.page(s, j) is not None:
                    count[p.page(s, j)] += 1
        miscounted += sum(a != b for a, b in zip(count, p.refs))
    assert refused > 5
    return shared, miscounted


@pytest.mark.parametrize("seed", range(8))
def test_refused_rows_as_idle_slots(seed):
    assert run(seed, True) == (0, 0)


def test_refused_rows_with_the_length_they_wanted():
    """What the idle slots are for."""
    shared, miscounted = np.sum([run(seed, False) for seed in range(8)], axis=0)
    assert shared > 0 and miscounted > 0
