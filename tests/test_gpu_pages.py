"""The pages under the cache against the oracle's lists: random runs of forks,
steps, ends and compactions with the contents that they move."""
import numpy as np
import pytest

from oracle import step
from packed_bit_gemv_tern_amd import tern

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from gpu_util import DEV, to_dev  # noqa: E402


class Both:
    """A pool on the host and on the device."""

    def __init__(self, pages, S, columns, P, seed=0):
        self.rng = np.random.default_rng([pages, S, columns, P, seed])
        self.host = step.Pool(pages, S, columns, P, self.rng)
        self.S, self.pages, self.columns = S, pages, columns
        self.upload()

    def upload(self):
        self.refs, self.table = (to_dev(np.asarray(a, np.int32)) for a in (self.host.refs, self.host.table))
        self.pool = tern.make_kv_pool(self.refs, self.table, self.columns, self.S, self.pages, self.host.P)
        self.ws = torch.full((tern.tern_kv_pool_workspace_bytes(self.pool),), 0x5A, dtype=torch.uint8, device=DEV)
        return self

    def check(self):
        assert self.refs.cpu().tolist() == self.host.refs
        assert self.table.cpu().tolist() == self.host.table

    def fork(self, length, src, dst):
        self.host.fork(length, src, dst)
        tern.tern_kv_fork(self.pool, dev(length), dev(src), dev(dst), len(src))
        self.check()

    def truncate(self, length, keep):
        self.host.truncate(length, keep)
        tern.tern_kv_truncate(self.pool, dev(length), dev(keep))
        self.check()

    def reserve(self, length, want):
        out = torch.full((3, self.S), -7, dtype=torch.int32, device=DEV)
        tern.tern_kv_reserve(self.pool, dev(length), dev(want), out[0], out[1], out[2], self.ws)
        ref = self.host.reserve(length, want)
        assert out.cpu().tolist() == [list(r) for r in ref]
        self.check()
        return ref

    def compact(self, length, moves):
        out, live = torch.full((2, max(moves, 1)), -7, dtype=torch.int32, device=DEV), dev([-7])
        tern.tern_kv_compact(self.pool, dev(length), out[0], out[1], moves, live, self.ws)
        src, dst, n = self.host.compact(length, moves)
        assert out.cpu().tolist() == [src, dst] if moves else True
        assert live.item() == n
        self.check()
        return src, dst


def dev(a):
    return to_dev(np.asarray(a, np.int32))


@pytest.mark.parametrize("pages,S,columns,P", [(30, 6, 8, 16), (200, 13, 9, 32), (9000, 70, 33, 64), (13000, 300, 17, 128),
                                               (1, 1, 1, 16), (3, 2, 4, 16),
                                               (16384, 40, 60, 16), (16385, 40, 60, 16), (40000, 300, 9, 32)])
def test_random_runs(pages, S, columns, P):
    b = Both(pages, S, columns, P)
    rng, length = b.rng, [0] * S
    for _ in range(25):
        what = rng.integers(4)
        if what == 0:
            empty = [s for s in range(S) if not length[s]]
            full = [s for s in range(S) if length[s]]
            if empty and full:
                dst = [int(d) for d in rng.permutation(empty)[: rng.integers(1, len(empty) + 1)]]
                src = [int(rng.choice(full)) for _ in dst]
                b.fork(length, src, dst)
                for s, d in zip(src, dst):
                    length[d] = length[s]
        elif what == 1:
            want = [n + int(rng.integers(-3, 2 * P)) for n in length]
            granted, _, _ = b.reserve(length, want)
            length = [max(n, w) if g else n for n, w, g in zip(length, want, granted)]
        elif what == 2:
            keep = [int(rng.integers(-2, n + 3)) if rng.integers(3) else n for n in length]
            b.truncate(length, keep)
            length = [max(0, min(n, k)) for n, k in zip(length, keep)]
        else:
            b.compact(length, int(rng.choice([0, 1, pages // 4, pages // 2, pages])))


def test_forks_that_are_passed_over():
    b = Both(40, 8, 4, 16)
    length = [40, 0, 0, 0, 33, 0, 0, 0]
    b.reserve([0] * 8, length)
    # the same row twice, rows outside the table, a chain, a row onto itself
    b.fork(length, [0, 4, 0, 4, -1, 8, 0, 5, 6], [1, 1, 2, 8, 3, 3, -1, 5, 6])
    b.fork(length, [0, 2], [2, 3])


def test_shared_last_page():
    """Three holders of one part-filled page: who copies it, and who keeps it."""
    b = Both(40, 5, 4, 16)
    length = [20, 0, 0, 0, 30]
    b.reserve([0] * 5, length)
    b.fork(length, [0, 0], [1, 2])
    length = [20, 20, 20, 0, 30]
    _, src, _ = b.reserve(length, [21, 20, 20, 0, 31])  # one of three writes: copies
    assert [a >= 0 for a in src] == [True, False, False, False, False]
    _, src, _ = b.reserve([21, 20, 20, 0, 31], [22, 24, 40, 0, 31])  # both others: the last keeps it
    assert [a >= 0 for a in src] == [False, True, False, False, False]
    # no more than a page's own place: nothing is taken
    assert b.reserve([22, 24, 40, 0, 31], [23, 25, 41, 0, 32]) == ([1] * 5, [-1] * 5, [-1] * 5)


def test_pool_that_runs_out():
    """Rows in order: one that does not fit, and the later ones that need pages
    or keep a shared one, get nothing; the others go on."""
    b = Both(7, 6, 8, 16)
    length = [20, 0, 10, 0, 0, 16]
    b.reserve([0] * 6, length)
    b.fork(length, [0], [1])
    length[1] = 20
    # three pages are free: row 0 would need four (its part-filled page is row 1's too), and row 1, which would keep
    # that page, must not write into it while row 0 has no copy
    assert b.reserve(length, [80, 21, 11, 5, 0, 17])[0] == [0, 0, 1, 0, 1, 0]
    # two fresh ones and the copy: all three, the page is row 1's alone
    granted, src, _ = b.reserve(length, [60, 21, 11, 5, 0, 17])
    assert granted == [1, 1, 1, 0, 1, 0] and [a >= 0 for a in src] == [True] + [False] * 5
    b.reserve([60, 21, 11, 0, 0, 16], [60, 22, 12, 0, 0, 16])
    # more tokens than the table has columns: refused alone
    c = Both(50, 3, 2, 16)
    assert c.reserve([0, 0, 0], [33, 32, 1])[0] == [0, 1, 1]


@pytest.mark.parametrize("S", [1025, 2048, 2049])
def test_many_sequences(S):
    """Batches on both sides of what one workgroup takes, few pages left."""
    b = Both(2 * S, S, 3, 16)
    want = [int(n) for n in b.rng.integers(0, 33, S)]
    granted, _, _ = b.reserve([0] * S, want)
    length = [w if g else 0 for w, g in zip(want, granted)]
    full = int(np.argmax(length))
    empty = [s for s in range(S) if length[s] == 0][:5]
    b.fork(length, [full] * len(empty), empty)
    for s in empty:
        length[s] = length[full]
    b.reserve(length, [n + 9 for n in length])


def test_pages_without_holders_and_bad_entries():
    """Ids outside the pool inside the held part hold nothing; a page given up
    more often than it was counted stays free."""
    b = Both(20, 3, 4, 16)
    b.host.table = [[5, 20, -1, 7], [2 ** 31 - 1, -2 ** 31, 5, 3], [7, 8, 9, 19]]
    b.host.refs[5], b.host.refs[7] = 2, 1
    b.upload()
    b.reserve([33, 30, 0], [34, 31, 0])
    b.fork([50, 30, 0], [0], [2])
    b.compact([50, 30, 50], 10)
    b.truncate([64, 64, 64], [0, 0, 0])
    b.truncate([64, 64, 64], [0, 0, 0])


def test_large_pool():
    """Many chunks of pages: ranks carried across workgroups."""
    pages, S, columns, P = 70001, 40, 1200, 16
    b = Both(pages, S, columns, P)
    free = b.rng.random(pages) < 0.3
    b.host.refs = [0 if f else 1 for f in free]
    b.upload()
    want = [int(b.rng.integers(0, columns * P + 1)) for _ in range(S)]
    b.reserve([0] * S, want)
    c = Both(pages, 2, 4, P, seed=1)
    c.host.refs = [int(r) for r in b.rng.integers(0, 2, pages)]
    c.upload()
    for moves in (100, pages // 2):
        c.compact([0, 0], moves)


@pytest.mark.parametrize("pages", [1, 2, 17, 4096, 4097, 12287, 12288, 12289, 16385])
@pytest.mark.parametrize("share", [0.0, 0.03, 0.5, 1.0])
def test_compact_sizes(pages, share):
    """Pools inside one workgroup and past it, nearly full to nearly empty, lists
    shorter and longer than the moves (compact compares every array)."""
    for moves in (0, 1, 5, pages // 2, pages + 3):
        c = Both(pages, 2, 4, 16, seed=2)
        c.host.refs = [int(r < share) * int(k) for r, k in zip(c.rng.random(pages), c.rng.integers(1, 4, pages))]
        used = [i for i, r in enumerate(c.host.refs) if r]
        if len(used) > 4:
            c.host.table = [used[:2] + used[-2:], [used[-1], -1, used[len(used) // 2], used[0]]]
        c.upload()
        c.compact([64, 40], moves)


@pytest.mark.parametrize("H,D,P,L", [(2, 64, 16, 3), (1, 128, 128, 2), (8, 128, 64, 2), (3, 64, 32, 41), (1, 64, 16, 81)])
def test_copy(H, D, P, L):
    rng = np.random.default_rng([H, D, P, L])
    pages = 12
    shapes = ((pages, H, P, D), (pages, H, D, P), (pages, H), (pages, H))
    make = lambda n, layers: [[torch.from_numpy(  # noqa: E731
        rng.integers(-127, 128, (n,) + s[1:]).astype(np.int8) if len(s) > 2 else rng.random((n,) + s[1:]).astype(np.float32)
    ).to(DEV) for s in shapes] for _ in range(layers)]
    a, b = make(pages, L), make(9, L)
    wrap = lambda layers, n: tern.make_kv_layers([tern.make_kv_cache(*t, n, H, D, P) for t in layers])  # noqa: E731
    # within one cache: pairs with ids outside are passed over
    src, dst = [3, -1, 0, 12, 5, 4, 2 ** 31 - 1], [7, 1, -1, 2, 12, 11, 6]
    ref = [[t.clone() for t in layer] for layer in a]
    for layer in ref:
        for t in layer:
            t[7], t[11] = t[3].clone(), t[4].clone()
    tern.tern_kv_copy(wrap(a, pages), wrap(a, pages), dev(src), dev(dst), len(src))
    # to a smaller one: 10 is no page of it
    src2, dst2 = [11, 7, 7, 1], [0, 8, 10, 3]
    ref2 = [[t.clone() for t in layer] for layer in b]
    for x, y in zip(ref2, ref):
        for t, u in zip(x, y):
            t[0], t[8], t[3] = u[11], u[7], u[1]
    tern.tern_kv_copy(wrap(b, 9), wrap(a, pages), dev(src2), dev(dst2), len(src2))
    for got, want in ((a, ref), (b, ref2)):
        for x, y in zip(got, want):
            assert all(torch.equal(t, u) for t, u in zip(x, y))


def test_copy_of_a_long_list():
    """More pairs than a step has, most of them empty."""
    n, pages = 5000, 64
    k = torch.randint(-127, 128, (pages, 1, 16, 64), dtype=torch.int8, device=DEV)
    v = torch.randint(-127, 128, (pages, 1, 64, 16), dtype=torch.int8, device=DEV)
    s = torch.rand((2, pages, 1), device=DEV)
    ref = [t.clone() for t in (k, v, s[0], s[1])]
    layer = tern.make_kv_layers([tern.make_kv_cache(k, v, s[0], s[1], pages, 1, 64, 16)])
    src, dst = np.full((2, n), -1, np.int32)
    at = [0, 17, 4095, 4999]
    src[at], dst[at] = [1, 2, 3, 4], [60, 61, 62, 63]
    tern.tern_kv_copy(layer, layer, dev(src), dev(dst), n)
    for t, r in zip((k, v, s[0], s[1]), ref):
        r[60:64] = r[1:5].clone()
        assert torch.equal(t, r)


def test_workspace_refusals():
    b = Both(5000, 3, 4, 16)
    n = tern.tern_kv_pool_workspace_bytes(b.pool)
    big = torch.empty(n + 512, dtype=torch.uint8, device=DEV)
    o = dev([0, 0, 0])
    for ws in (None, big[: n - 1], big[8: 8 + n]):
        for call in (lambda: tern.tern_kv_reserve(b.pool, o, o, o, o, o, ws),
                     lambda: tern.tern_kv_compact(b.pool, o, o, o, 3, o, ws)):
            with pytest.raises(tern.TernError) as e:
                call()
            assert e.value.status == tern.TERN_ERR_WORKSPACE
