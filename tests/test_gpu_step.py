"""A step from token ids to token ids with nothing left to the caller: lookup,
norm, linears, norm and rotation of q and k, pages, cache, attention, the gated
feed-forward with its epilogues, head and sampling; two layers over one pool of
pages; branches, drafted tokens taken back, sequences that end, compaction; eager,
captured in a HIP graph and replayed, and two users on two streams."""
import numpy as np
import pytest

from oracle import step as plain
from packed_bit_gemv_tern_amd import tern

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from gpu_util import DEV, gpu_pack, to_dev  # noqa: E402

HID, HQ, H, D, FFN, VOCAB, P, LAYERS, EPS = 256, 4, 2, 64, 320, 515, 16, 2, 1e-6


def i32(a):
    return to_dev(np.asarray(a, np.int32))


class Linear:
    def __init__(self, rng, N, K):
        w = rng.choice(np.array([-1, 0, 1], np.int8), p=[0.2, 0.6, 0.2], size=(N, K))
        self.N, self.K = N, K
        self.packed, self.rowsum, _ = gpu_pack(w)
        self.s = to_dev((rng.uniform(0.5, 1.5, N) * 1.5 / np.sqrt(K)).astype(np.float32))
        self.weights = tern.make_weights(self.packed, self.s, self.rowsum)

    def __call__(self, q, s, z, **kw):
        M = q.shape[0]
        y = torch.empty((M, self.N), device=DEV)
        tern.tern_linear_epilogue(self.weights, self.N, self.K, M, q, q.shape[1], s, z, y, self.N, **kw)
        return y


class Engine:
    """Slots of sequences over a pool of pages; the host keeps the tokens of each
    slot and what the lists of oracle/step.py say about the pages."""

    def __init__(self, seed, slots=4, pages=26, columns=8):
        rng = np.random.default_rng(seed)
        self.rng, self.slots, self.pages, self.columns = rng, slots, pages, columns
        width, kv = HQ * D, H * D
        self.layers = [dict(qkv=Linear(rng, width + 2 * kv, HID), o=Linear(rng, HID, width), gate=Linear(rng, FFN, HID),
                            up=Linear(rng, FFN, HID), down=Linear(rng, HID, FFN),
                            gains=[to_dev(rng.uniform(0.5, 1.5, n).astype(np.float32)) for n in (HID, HID, D, D)])
                       for _ in range(LAYERS)]
        self.gain = to_dev(rng.uniform(0.5, 1.5, HID).astype(np.float32))
        self.W = to_dev(rng.integers(-127, 128, (VOCAB, HID)).astype(np.int8))
        self.sW = to_dev(rng.uniform(0.005, 0.02, VOCAB).astype(np.float32))
        self.rowsum = torch.empty(VOCAB, dtype=torch.int32, device=DEV)
        tern.tern_head_rowsum(self.W, VOCAB, HID, HID, self.rowsum)
        self.freq = to_dev((1e4 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32))
        # (what the fresh cache holds must not matter)
        self.k = torch.randint(-127, 128, (LAYERS, pages, H, P, D), dtype=torch.int8, device=DEV)
        self.v = torch.randint(-127, 128, (LAYERS, pages, H, D, P), dtype=torch.int8, device=DEV)
        self.scales = torch.rand((2, LAYERS, pages, H), device=DEV)
        self.caches = [tern.make_kv_cache(self.k[i], self.v[i], self.scales[0, i], self.scales[1, i], pages, H, D, P)
                       for i in range(LAYERS)]
        self.cache_layers = tern.make_kv_layers(self.caches)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
        self.table = torch.full((slots, columns), -1, dtype=torch.int32, device=DEV)
        self.pool = tern.make_kv_pool(self.refs, self.table, columns, slots, pages, P)
        self.pool_ws = torch.empty(tern.tern_kv_pool_workspace_bytes(self.pool), dtype=torch.uint8, device=DEV)
        self.lists = torch.empty((3, slots), dtype=torch.int32, device=DEV)
        self.host = plain.Pool(pages, slots, columns, P)
        self.length = [0] * slots

    def check(self):
        assert self.refs.cpu().tolist() == self.host.refs
        got, want = self.table.cpu().tolist(), self.host.table
        for s, n in enumerate(self.length):
            j = self.host.count(n)
            assert got[s][:j] == want[s][:j]

    def state(self):
        return [self.k, self.v, self.scales, self.refs, self.table]

    def norm(self, x, gain, res=None):
        M = x.shape[0]
        h, q = torch.empty((M, HID), device=DEV), torch.empty((M, HID), dtype=torch.int8, device=DEV)
        s, z = torch.empty(M, device=DEV), torch.empty(M, dtype=torch.int32, device=DEV)
        tern.tern_rmsnorm_quantize(x, gain, EPS, M, HID, HID, q, HID, s, z, res=res, ldr=HID if res is not None else 0,
                                   h=h, ldh=HID)
        return h, q, s, z

    def quantise(self, x):
        M, K = x.shape
        q = torch.empty((M, K), dtype=torch.int8, device=DEV)
        s, z = torch.empty(M, device=DEV), torch.empty(M, dtype=torch.int32, device=DEV)
        tern.tern_quantize_act(x, M, K, K, q, K, s, z)
        return q, s, z

    def forward(self, ids, start, held, want, rows, max_new, u, ws=None):
        """ids (M), start (slots + 1), held and want (slots): device int32.
        Returns the residual stream behind the last layer and the sampled tokens."""
        tern.tern_kv_reserve(self.pool, held, want, self.lists[0], self.lists[1], self.lists[2], self.pool_ws)
        tern.tern_kv_copy(self.cache_layers, self.cache_layers, self.lists[1], self.lists[2], self.slots)
        M, width, kv = ids.shape[0], HQ * D, H * D
        ld = width + 2 * kv
        batch = tern.make_kv_batch(self.table, self.columns, start, want, self.slots, rows, max_new, 128)
        h = torch.empty((M, HID), device=DEV)
        tern.tern_embed(self.W, self.sW, VOCAB, HID, HID, ids, M, h, HID, scale=4.0)
        if ws is None:
            ws = self.workspaces(batch, M)
        for lay, cache in zip(self.layers, self.caches):
            _, q, s, z = self.norm(h, lay["gains"][0])
            qkv = lay["qkv"](q, s, z)
            k, v = qkv[:, width: width + kv], qkv[:, width + kv:]
            tern.tern_qk_norm_rope(batch, D, self.freq, D, q=qkv, ldq=ld, q_heads=HQ, q_gain=lay["gains"][2], q_out=qkv,
                                   ldqo=ld, k=k, ldk=ld, heads=H, k_gain=lay["gains"][3], k_out=k, ldko=ld, eps=EPS)
            tern.tern_kv_append(cache, batch, k, ld, v, ld)
            y = torch.zeros((M, width), device=DEV)
            tern.tern_attention(cache, batch, qkv, ld, HQ, D ** -0.5, y, width, ws[0])
            h = lay["o"](*self.quantise(y), res=h, ldr=HID)
            _, q, s, z = self.norm(h, lay["gains"][1])
            f = lay["gate"](q, s, z, up=lay["up"].weights, act=tern.TERN_ACT_SILU)
            h = lay["down"](*self.quantise(f), res=h, ldr=HID)
        _, q, s, z = self.norm(h, self.gain)
        logits = torch.empty((M, VOCAB), device=DEV)
        for r in range(0, M, 8):
            n = min(8, M - r)
            tern.tern_head_gemv(self.W, self.sW, self.rowsum, VOCAB, HID, HID, n, q[r:], HID, s[r:], z[r:], logits[r:],
                                VOCAB)
        token = torch.empty(M, dtype=torch.int32, device=DEV)
        tern.tern_sample(logits, M, VOCAB, VOCAB, torch.ones(M, device=DEV), u, token, ws[1])
        return h, token

    def workspaces(self, batch, M):
        return [torch.empty(n, dtype=torch.uint8, device=DEV) for n in (
            tern.tern_attention_workspace_bytes(self.caches[0], batch, HQ), tern.tern_sample_workspace_bytes(M, VOCAB))]

    def step(self, new):
        """new: lists of token ids for each slot.  Returns each slot's rows of the
        residual stream and its tokens."""
        n = [len(x) for x in new]
        start = np.concatenate([[0], np.cumsum(n)])
        want = [a + b for a, b in zip(self.length, n)]
        # (always 64 rows, most of them of no sequence, and 40 new ones at most: the attention picks its kernel by
        # these, and its kernels round differently)
        ids = [t for x in new for t in x]
        h, token = self.forward(i32(ids + [-1] * (64 - len(ids))), i32(start), i32(self.length), i32(want), 64, 40,
                                torch.zeros(64, device=DEV))
        granted, src, dst = self.host.reserve(self.length, want)
        assert self.lists.cpu().tolist() == [granted, src, dst] and all(granted)
        self.length = want
        self.check()
        return [(h[a:b].cpu(), token[a:b].cpu()) for a, b in zip(start[:-1], start[1:])]

    def keep(self, keep):
        tern.tern_kv_truncate(self.pool, i32(self.length), i32(keep))
        self.host.truncate(self.length, keep)
        self.length = [min(a, max(b, 0)) for a, b in zip(self.length, keep)]
        self.check()

    def fork(self, src, dst):
        tern.tern_kv_fork(self.pool, i32(self.length), i32(src), i32(dst), len(src))
        self.host.fork(self.length, src, dst)
        for a, b in zip(src, dst):
            self.length[b] = self.length[a]
        self.check()

    def compact(self):
        n = self.pages // 2
        src, dst, live = torch.empty((2, n), dtype=torch.int32, device=DEV).unbind(0) + (i32([0]),)
        tern.tern_kv_compact(self.pool, i32(self.length), src, dst, n, live, self.pool_ws)
        tern.tern_kv_copy(self.cache_layers, self.cache_layers, src, dst, n)
        a, b, n_live = self.host.compact(self.length, n)
        assert (src.cpu().tolist(), dst.cpu().tolist(), live.item()) == (a, b, n_live)
        self.check()
        return sum(x >= 0 for x in a)


def test_pages_do_not_show_in_the_results():
    """A run with branches, drafts taken back, ends and compactions gives, bit for
    bit, what each sequence gives alone in a fresh engine of the same weights and
    calls: where a sequence's tokens lie, and who shared them, does not matter."""
    a = Engine(1)
    rng = np.random.default_rng(0)
    ids = lambda n: [int(x) for x in rng.integers(0, VOCAB, n)]  # noqa: E731
    prompt, other = ids(21), ids(33)
    calls = {s: [] for s in range(4)}  # what each slot was given: ("step", ids) or ("keep", n)
    seen = {s: [] for s in range(4)}

    def go(new):
        for s, out in enumerate(a.step(new)):
            if new[s]:
                calls[s].append(("step", new[s]))
                seen[s].append(out)

    def cut(keep):
        a.keep(keep)
        for s in range(4):
            calls[s].append(("keep", keep[s]))

    def branch(src, dst):
        a.fork(src, dst)
        for x, y in zip(src, dst):
            calls[y], seen[y] = list(calls[x]), list(seen[x])

    go([prompt, [], other, []])
    branch([0, 0], [1, 3])
    go([ids(1), ids(1), ids(1), ids(1)])  # the branches part: the part-filled page is copied twice, kept once
    go([ids(6), ids(5), ids(6), ids(1)])  # drafted tokens, some of them over a page's end
    cut([24, 27, 39, 23])
    go([ids(2), ids(1), ids(1), ids(2)])
    calls[2], seen[2] = [], []
    a.keep([a.length[0], a.length[1], 0, a.length[3]])  # slot 2 ends: pages below those of others are free
    assert a.compact() > 0
    go([ids(1), ids(1), [], ids(12)])
    branch([3], [2])
    go([ids(1), ids(7), ids(8), ids(1)])
    a.compact()
    go([ids(1)] * 4)
    for s in range(4):
        b = Engine(1)
        assert torch.equal(a.W, b.W)
        outs = []
        for what, x in calls[s]:
            if what == "step":
                outs.append(b.step([[], [], x, []])[2])
            else:
                b.keep([0, 0, x, 0])
        for (h, t), (h1, t1) in zip(seen[s], outs):
            assert torch.equal(h, h1) and torch.equal(t, t1)
        assert len(outs) == len(seen[s]) > 3


def test_step_in_a_graph_replayed():
    """One token for each slot (one idle), captured once: replayed with other
    tokens, lengths and pages, a branch among them, eager work in between; every
    replay equals the eager step from the same state."""
    e = Engine(2)
    rng = np.random.default_rng(1)
    e.step([[int(x) for x in rng.integers(0, VOCAB, n)] for n in (15, 3, 20, 0)])
    e.fork([2], [3])
    ids, held, want, start = i32([1, 2, 3, 4]), i32(e.length), i32([n + 1 for n in e.length]), i32([0, 1, 2, 3, 4])
    u = torch.zeros(4, device=DEV)
    ws = e.workspaces(tern.make_kv_batch(e.table, e.columns, start, want, 4, 4, 1, 128), 4)
    first = [t.clone() for t in e.state()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        e.forward(ids, start, held, want, 4, 1, u, ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = e.forward(ids, start, held, want, 4, 1, u, ws)
    for t, f in zip(e.state(), first):
        t.copy_(f)
    length = list(e.length)
    for i in range(6):
        grow = [1, int(i != 2), 1, 1]  # (an idle slot in the third)
        ids.copy_(torch.from_numpy(rng.integers(0, VOCAB, 4).astype(np.int32)))
        held.copy_(torch.tensor(length, dtype=torch.int32))
        want.copy_(torch.tensor([a + b for a, b in zip(length, grow)], dtype=torch.int32))
        u.copy_(torch.from_numpy(rng.random(4).astype(np.float32)))
        before = [t.clone() for t in e.state()]
        eager = [t.clone() for t in e.forward(ids, start, held, want, 4, 1, u)]
        after = [t.clone() for t in e.state()]
        for t, b in zip(e.state(), before):
            t.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, eager):
            assert torch.equal(x, y), "replay %d" % i
        for x, y in zip(e.state(), after):
            assert torch.equal(x, y), "replay %d: state" % i
        length = [a + b for a, b in zip(length, grow)]


def test_two_streams():
    """Two engines in flight at once: what each gives alone."""
    outs = []
    for together in (False, True):
        engines = [Engine(3 + i) for i in range(2)]
        streams = [torch.cuda.Stream() if together else torch.cuda.current_stream() for _ in range(2)]
        torch.cuda.synchronize()
        got = []
        n = [40, 1, 17, 9]
        for rep in range(4):
            for i, e in enumerate(engines):
                rng = np.random.default_rng([rep, i])
                with torch.cuda.stream(streams[i]):
                    start = i32(np.concatenate([[0], np.cumsum(n)]))
                    held, want = i32([rep * x for x in n]), i32([(rep + 1) * x for x in n])
                    got.append(e.forward(i32(rng.integers(0, VOCAB, sum(n))), start, held, want, sum(n), max(n),
                                         torch.zeros(sum(n), device=DEV)))
            n = [1, 1, 1, 1] if rep == 2 else n
        torch.cuda.synchronize()
        outs.append([[t.cpu() for t in o] for o in got])
    for x, y in zip(*outs):
        assert all(torch.equal(a, b) for a, b in zip(x, y))
