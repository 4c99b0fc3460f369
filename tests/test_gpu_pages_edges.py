"""The pages under the cache at the borders of what the calls allow: pools
without rows, rows that a reserve refuses."""
import numpy as np
import pytest

from oracle import step as plain
from packed_bit_gemv_tern_amd import tern

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from gpu_util import DEV, to_dev  # noqa: E402


@pytest.mark.parametrize("pages", [0, 1, 40, 12288, 12289, 20000])
@pytest.mark.parametrize("moves", [0, 1, 300])
def test_compact_without_rows(pages, moves):
    """live and the lists of moves are written where no row holds a page, on both
    sides of the one workgroup's border and for a pool of no pages."""
    refs = torch.zeros(max(pages, 1), dtype=torch.int32, device=DEV)
    table = torch.empty((0, 4), dtype=torch.int32, device=DEV)
    p = tern.make_kv_pool(refs, table, 4, 0, pages, 16)
    ws = torch.full((tern.tern_kv_pool_workspace_bytes(p),), 0x5A, dtype=torch.uint8, device=DEV)
    out = torch.full((2, moves + 1), 3, dtype=torch.int32, device=DEV)
    live = torch.full((1,), 3, dtype=torch.int32, device=DEV)
    tern.tern_kv_compact(p, None, out[0], out[1], moves, live, ws)
    assert live.item() == 0
    assert out.cpu().tolist() == [[-1] * moves + [3]] * 2
    assert not refs.any()


def i32(a):
    return to_dev(np.asarray(a, np.int32))


HQ, H, D, P, LAYERS, S = 4, 2, 64, 16, 2, 3


class Steps:
    """Three slots over a pool and a cache of two layers, steps from given rows of q,
    k and v; the host keeps the lists of oracle/step.py."""

    def __init__(self, pages, columns):
        rng = np.random.default_rng([pages, columns])
        self.pages, self.columns = pages, columns
        # (what the fresh cache holds must not matter)
        self.k = to_dev(rng.integers(-127, 128, (LAYERS, pages, H, P, D)).astype(np.int8))
        self.v = to_dev(rng.integers(-127, 128, (LAYERS, pages, H, D, P)).astype(np.int8))
        self.scales = to_dev(rng.uniform(0.005, 0.03, (2, LAYERS, pages, H)).astype(np.float32))
        self.caches = [tern.make_kv_cache(self.k[i], self.v[i], self.scales[0, i], self.scales[1, i], pages, H, D, P)
                       for i in range(LAYERS)]
        self.layers = tern.make_kv_layers(self.caches)
        self.host = plain.Pool(pages, S, columns, P, rng)  # (entries that hold nothing: any ids)
        self.refs, self.table = i32(self.host.refs), i32(self.host.table)
        self.pool = tern.make_kv_pool(self.refs, self.table, columns, S, pages, P)
        self.pool_ws = torch.empty(tern.tern_kv_pool_workspace_bytes(self.pool), dtype=torch.uint8, device=DEV)
        self.lists = torch.empty((3, S), dtype=torch.int32, device=DEV)
        self.now = torch.empty(S, dtype=torch.int32, device=DEV)
        self.freq = to_dev((1e4 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32))
        self.length = [0] * S

    def state(self):
        return [self.k, self.v, self.scales, self.refs, self.table]

    def workspace(self, start, rows, max_new):
        batch = tern.make_kv_batch(self.table, self.columns, start, self.now, S, rows, max_new, 64)
        n = tern.tern_attention_workspace_bytes(self.caches[0], batch, HQ)
        return torch.empty(n, dtype=torch.uint8, device=DEV)

    def forward(self, qkv, start, held, want, kept, max_new, ws):
        """One step as the header lists it, all on the device.  Returns the rotated rows
        (8: those that are left as they were) and y."""
        rows = qkv.shape[1]
        tern.tern_kv_reserve(self.pool, held, want, self.lists[0], self.lists[1], self.lists[2], self.pool_ws)
        tern.tern_kv_copy(self.layers, self.layers, self.lists[1], self.lists[2], S)
        torch.mul(want, self.lists[0], out=self.now)
        batch = tern.make_kv_batch(self.table, self.columns, start, self.now, S, rows, max_new, 64)
        ld = (HQ + 2 * H) * D
        turned = torch.full((LAYERS, rows, (HQ + H) * D), 8.0, device=DEV)
        y = torch.full((LAYERS, rows, HQ * D), 8.0, device=DEV)
        for i, cache in enumerate(self.caches):
            q, k, v, t = qkv[i], qkv[i, :, HQ * D:], qkv[i, :, (HQ + H) * D:], turned[i]
            tern.tern_qk_norm_rope(batch, D, self.freq, D, q=q, ldq=ld, q_heads=HQ, q_out=t, ldqo=(HQ + H) * D, k=k,
                                   ldk=ld, heads=H, k_out=t[:, HQ * D:], ldko=(HQ + H) * D)
            tern.tern_kv_append(cache, batch, t[:, HQ * D:], (HQ + H) * D, v, ld)
            tern.tern_attention(cache, batch, t, (HQ + H) * D, HQ, D ** -0.5, y[i], HQ * D, ws)
        tern.tern_kv_truncate(self.pool, self.now, kept)
        return turned, y

    def step(self, qkv, new, kept=None, granted=None):
        """new: rows of each slot, in order; kept: tokens kept of those granted (all)."""
        start = np.concatenate([[0], np.cumsum(new)])
        want = [a + b for a, b in zip(self.length, new)]
        kept = want if kept is None else kept
        ws = self.workspace(i32(start), qkv.shape[1], max(new))
        out = self.forward(qkv, i32(start), i32(self.length), i32(want), i32(kept), max(new), ws)
        lists = self.host.reserve(self.length, want)
        assert self.lists.cpu().tolist() == [list(x) for x in lists]
        assert granted is None or lists[0] == granted
        now = [g * w for g, w in zip(lists[0], want)]
        assert self.now.cpu().tolist() == now
        self.host.truncate(now, kept)
        self.length = [min(w, t) if g else n for g, w, t, n in zip(lists[0], want, kept, self.length)]
        self.check()
        return out

    def fork(self, src, dst):
        tern.tern_kv_fork(self.pool, i32(self.length), i32([src]), i32([dst]), 1)
        self.host.fork(self.length, [src], [dst])
        self.length[dst] = self.length[src]
        self.check()

    def end(self, s):
        keep = [0 if i == s else n for i, n in enumerate(self.length)]
        tern.tern_kv_truncate(self.pool, i32(self.length), i32(keep))
        self.host.truncate(self.length, keep)
        self.length[s] = 0
        self.check()

    def check(self):
        assert self.refs.cpu().tolist() == self.host.refs
        assert self.table.cpu().tolist() == self.host.table
        count = [0] * self.pages
        for s in range(S):
            for j in range(self.host.count(self.length[s])):
                count[self.host.table[s][j]] += 1
        assert self.host.refs == count

    def tokens(self, s):
        """Codes and scales of a slot's tokens, as they lie in its pages."""
        n = self.length[s]
        ids = torch.tensor([self.host.page(s, j) for j in range(self.host.count(n))], device=DEV)
        k = self.k[:, ids].transpose(2, 3).flatten(1, 2)[:, :n]
        v = self.v[:, ids].permute(0, 1, 4, 2, 3).flatten(1, 2)[:, :n]
        return [t.clone() for t in (k, v, self.scales[:, :, ids])]


def rows_of(seed, n):
    return to_dev(np.random.default_rng(seed).standard_normal((LAYERS, n, (HQ + 2 * H) * D)).astype(np.float32))


@pytest.mark.parametrize("pages,columns,held,new", [(3, 4, 20, 1), (3, 4, 20, 6), (8, 2, 31, 3)])
def test_a_refused_row_leaves_what_it_shares(pages, columns, held, new):
    """Two rows share a part-filled page and are refused, for want of pages or of
    columns, beside a third that is served: no byte of the shared pages changes, the
    third row gets what it gets alone, and a later step gives both what they get in a
    pool that never refused."""
    a, b = Steps(pages, columns), Steps(12, columns)
    prompt, drafted, last = rows_of(1, held + 10), rows_of(2, 3 * new), rows_of(3, 2)
    for e in (a, b):
        e.step(prompt, [held, 0, 10], granted=[1, 1, 1])
        e.fork(0, 1)
    shared = torch.tensor([a.host.page(0, j) for j in range(2)], device=DEV)
    own = a.host.page(2, 0)
    before = [t.clone() for t in a.state()]
    turned, y = a.step(drafted, [new] * 3, kept=[held, held, 10], granted=[0, 0, 1])
    for t, u in zip(a.state()[:2], before):
        assert torch.equal(t[:, shared], u[:, shared])
        assert not torch.equal(t[:, own], u[:, own])  # (the third row's tokens went there)
    assert torch.equal(a.scales[:, :, shared], before[2][:, :, shared])
    assert (turned[:, : 2 * new] == 8.0).all() and not y[:, : 2 * new].any()
    # the third row alone, from the same state
    after = [t.clone() for t in a.state()]
    for t, u in zip(a.state(), before):
        t.copy_(u)
    ws = a.workspace(i32([0] * 4), 3 * new, new)
    alone = a.forward(drafted, i32([2 * new] * 3 + [3 * new]), i32([0, 0, 10]), i32([0, 0, 10 + new]), i32([0, 0, 10]),
                      new, ws)
    for t, u in zip((turned, y), alone):
        assert torch.equal(t[:, 2 * new:], u[:, 2 * new:])
    for t, u in zip(a.state()[:4], after):
        assert torch.equal(t, u)
    a.table.copy_(after[4])
    for e in (a, b):
        e.end(2)
    outs = [e.step(last, [1, 1, 0], granted=[1, 1, 1]) for e in (a, b)]
    assert all(torch.equal(t, u) for t, u in zip(*outs))
    for s in range(2):
        for t, u in zip(a.tokens(s), b.tokens(s)):
            assert torch.equal(t, u)


def test_refused_rows_in_a_graph_replayed():
    """One captured step, replayed while a pool runs out, rows end and the refused ones
    are served: every replay equals the eager step from the same state, and the host's
    lists."""
    e = Steps(4, 4)
    e.step(rows_of(4, 30), [20, 0, 10], granted=[1, 1, 1])
    e.fork(0, 1)
    qkv, start = rows_of(5, 3), i32([0, 1, 2, 3])
    held, want, kept = (torch.zeros(S, dtype=torch.int32, device=DEV) for _ in range(3))
    ws = e.workspace(start, 3, 1)
    first = [t.clone() for t in e.state()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        e.forward(qkv, start, held, want, kept, 1, ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = e.forward(qkv, start, held, want, kept, 1, ws)
    for t, f in zip(e.state(), first):
        t.copy_(f)
    seen = set()
    for i in range(24):
        if i == 14:
            e.end(2)
        qkv.copy_(rows_of([6, i], 3))
        new = [1, 1, int(i < 14)]
        lengths = [e.length, [n + m for n, m in zip(e.length, new)]]
        held.copy_(i32(lengths[0])), want.copy_(i32(lengths[1])), kept.copy_(i32(lengths[1]))
        before = [t.clone() for t in e.state()]
        eager = [t.clone() for t in e.forward(qkv, start, held, want, kept, 1, ws)]
        after = [t.clone() for t in e.state()]
        for t, b in zip(e.state(), before):
            t.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        for t, u in zip([*out, *e.state()], [*eager, *after]):
            assert torch.equal(t, u), "replay %d" % i
        granted = e.host.reserve(*lengths)[0]
        assert e.lists[0].cpu().tolist() == granted
        e.host.truncate([x * w for x, w in zip(granted, lengths[1])], lengths[1])
        e.length = [w if x else n for x, n, w in zip(granted, *lengths)]
        e.check()
        seen.add(tuple(granted))
    assert (1, 1, 1) in seen and len(seen) > 1
