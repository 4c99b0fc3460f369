"""The decode step's operators together, as they are used: norm and int8
codes, ternary linears, the cache's append and its attention, the int8 head
and sampling; prompts first, then single tokens; eager, captured in a HIP graph
and on two streams.  Each call is checked against the oracle on the inputs
that it had: bit for bit, the attention within the roundings of fp32."""
import numpy as np
import pytest

import oracle
from oracle import decode
from packed_bit_gemv_tern_amd import tern

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from gpu_util import DEV, gpu_pack, to_dev  # noqa: E402
from kv_util import Paged  # noqa: E402

HID, HQ, HKV, D, FFN, VOCAB, P = 512, 8, 2, 64, 768, 1003, 16
EPS = 1e-6


def bits(a):
    a = np.ascontiguousarray(a)
    return a.view(np.uint32) if a.dtype == np.float32 else a


def same(gpu, ref, what):
    got = gpu.cpu().numpy() if torch.is_tensor(gpu) else gpu
    assert np.array_equal(bits(got), bits(np.asarray(ref, got.dtype))), what


class Linear:
    def __init__(self, rng, N, K):
        w = rng.choice(np.array([-1, 0, 1], np.int8), p=[0.2, 0.6, 0.2], size=(N, K))
        self.s_row = rng.uniform(0.01, 0.1, N).astype(np.float32)
        self.N, self.K = N, K
        self.packed, self.rowsum, _ = gpu_pack(w)
        self.s_dev = to_dev(self.s_row)
        self.rp, self.rr, _ = oracle.pack(w)

    def __call__(self, q, s, z, y=None):
        M = q.shape[0]
        y = torch.empty((M, self.N), device=DEV) if y is None else y
        tern.tern_gemm_smallM(self.packed, self.s_dev, self.rowsum, self.N, self.K, M, q, q.shape[1], s, z, y, self.N)
        return y

    def check(self, y, q, s, z, what):
        ref = oracle.linear(self.rp, self.s_row, self.rr, self.K, q.cpu().numpy()[:, : self.K], s.cpu().numpy(),
                            z.cpu().numpy())[1]
        same(y, ref, what)


class Model:
    """One layer and a head, with a table of int8 token embeddings."""

    def __init__(self, seed, seqs):
        rng = np.random.default_rng(seed)
        width, kvw = HQ * D, HKV * D
        self.qkv = Linear(rng, width + 2 * kvw, HID)
        self.o, self.gate, self.up, self.down = (Linear(rng, *nk) for nk in (
            (HID, width), (FFN, HID), (FFN, HID), (HID, FFN)))
        self.gains = [to_dev(rng.uniform(0.5, 1.5, HID).astype(np.float32)) for _ in range(3)]
        W = rng.integers(-127, 128, (VOCAB, HID)).astype(np.int8)
        self.W, self.s_head = to_dev(W), to_dev(rng.uniform(1e-3, 1e-2, VOCAB).astype(np.float32))
        self.Wh, self.sh = W, self.s_head.cpu().numpy()
        self.rowsum = torch.empty(VOCAB, dtype=torch.int32, device=DEV)
        tern.tern_head_rowsum(self.W, VOCAB, HID, HID, self.rowsum)
        self.pg = Paged(seqs, 6, HKV, D, P, seed=seed).upload()

    def norm(self, i, x, res, check):
        M = x.shape[0]
        h = torch.empty((M, HID), device=DEV)
        q = torch.empty((M, HID), dtype=torch.int8, device=DEV)
        s, z = torch.empty(M, device=DEV), torch.empty(M, dtype=torch.int32, device=DEV)
        tern.tern_rmsnorm_quantize(x, self.gains[i], EPS, M, HID, HID, q, HID, s, z, res=res,
                                   ldr=0 if res is None else HID, h=h, ldh=HID)
        if check:
            ref = decode.rmsnorm_quantize(x.cpu().numpy(), None if res is None else res.cpu().numpy(),
                                          self.gains[i].cpu().numpy(), EPS)
            for got, want, what in zip((h, q, s, z), ref, "hqsz"):
                same(got, want, "norm %d %s" % (i, what))
        return h, q, s, z

    def quantise(self, x):
        M, K = x.shape
        q = torch.empty((M, K), dtype=torch.int8, device=DEV)
        s, z = torch.empty(M, device=DEV), torch.empty(M, dtype=torch.int32, device=DEV)
        tern.tern_quantize_act(x, M, K, K, q, K, s, z)
        return q, s, z

    def step(self, x, batch, params, last, check=True, workspaces=None):
        """x: fp32 embeddings of the new rows.  Returns (tokens, probs, kept)
        of the rows `last`."""
        pg, width, kvw = self.pg, HQ * D, HKV * D
        M = x.shape[0]
        h, q, s, z = self.norm(0, x, None, check)
        qkv = self.qkv(q, s, z)
        ld = width + 2 * kvw
        k, v = qkv[:, width: width + kvw], qkv[:, width + kvw:]
        tern.tern_kv_append(pg.cache, batch, k, ld, v, ld)
        y = torch.zeros((M, width), device=DEV)
        ws = workspaces or [torch.empty(n, dtype=torch.uint8, device=DEV) for n in (
            tern.tern_attention_workspace_bytes(pg.cache, batch, HQ), tern.tern_sample_workspace_bytes(8, VOCAB))]
        tern.tern_attention(pg.cache, batch, qkv, ld, HQ, D ** -0.5, y, width, ws[0])
        if check:
            self.qkv.check(qkv, q, s, z, "qkv")
            kh, vh = (a.cpu().numpy().reshape(M, HKV, D) for a in (k, v))
            decode.kv_append(pg.host, pg.table, pg.start, pg.length, kh, vh, pg.max_new)
            pg.check()
            ref = np.zeros((M, HQ, D))
            size = decode.attention(pg.host, pg.table, pg.start, pg.length,
                                    qkv[:, :width].cpu().numpy().reshape(M, HQ, D), D ** -0.5, pg.max_new, ref)
            # (as in test_gpu_attention.py, for at most 6 pages of 16)
            tol = 2 * size[..., 1:] * (size[..., :1] * (2 ** -21 + 24 * 2 ** -24) + 2 ** -22 + 2 ** -21 + 2 ** -16)
            assert (np.abs(y.cpu().numpy().reshape(M, HQ, D) - ref) <= tol).all()
        qo = self.quantise(y)
        attn = self.o(*qo)
        h2, q, s, z = self.norm(1, attn, h, check)
        g, u = self.gate(q, s, z), self.up(q, s, z)
        hf = torch.nn.functional.silu(g) * u
        qf = self.quantise(hf)
        ffn = self.down(*qf)
        h3, q3, s3, z3 = self.norm(2, ffn, h2, check)
        if check:
            self.o.check(attn, *qo, "o")
            self.gate.check(g, q, s, z, "gate")
            self.down.check(ffn, *qf, "down")
        ql, sl, zl = q3[last].contiguous(), s3[last].contiguous(), z3[last].contiguous()
        m = ql.shape[0]
        logits = torch.empty((m, VOCAB), device=DEV)
        tern.tern_head_gemv(self.W, self.s_head, self.rowsum, VOCAB, HID, HID, m, ql, HID, sl, zl, logits, VOCAB)
        token = torch.empty(m, dtype=torch.int32, device=DEV)
        prob, kept = torch.empty(m, device=DEV), torch.empty(m, dtype=torch.int32, device=DEV)
        T, uu, tk, tp, mp = params
        tern.tern_sample(logits, m, VOCAB, VOCAB, T, uu, token, ws[1], top_k=tk, top_p=tp, min_p=mp, prob=prob,
                         kept=kept)
        if check:
            same(logits, oracle.head(self.Wh, self.sh, oracle.head_rowsum(self.Wh), ql.cpu().numpy(),
                                     sl.cpu().numpy(), zl.cpu().numpy())[1], "logits")
            for i in range(m):
                ref = decode.sample(logits[i].cpu().numpy(), *(a[i].cpu().numpy() for a in params))
                assert (int(token[i]), int(kept[i])) == (ref[0], ref[2])
                assert abs(float(prob[i]) - ref[1]) <= 2 ** -23 * ref[1]
        return token, prob, kept

    def embed(self, token):
        return self.W[token.long()].float() * self.s_head[token.long()][:, None] * 8


def sampling(rng, m):
    f = lambda a: to_dev(np.asarray(a, np.float32))  # noqa: E731
    return (f(rng.uniform(0.5, 1.2, m)), f(rng.random(m)), to_dev(rng.integers(1, 60, m).astype(np.int32)),
            f(rng.uniform(0.6, 0.99, m)), f(rng.uniform(0.0, 0.05, m)))


def test_prompt_then_tokens():
    rng = np.random.default_rng(1)
    m = Model(1, 3)
    new = [21, 1, 34]
    length = list(new)
    ids = rng.integers(0, VOCAB, sum(new))
    last = [sum(new[: i + 1]) - 1 for i in range(3)]
    batch = m.pg.batch(new, length, max_len=64)
    token, _, _ = m.step(m.embed(torch.from_numpy(ids).to(DEV)), batch, sampling(rng, 3), last)
    for _ in range(4):
        length = [n + 1 for n in length]
        batch = m.pg.batch([1, 1, 1], length, max_len=64)
        token, _, _ = m.step(m.embed(token), batch, sampling(rng, 3), [0, 1, 2])


def test_drafted_tokens_in_one_pass_match_single_ones():
    """Five drafted tokens verified at once: the rows' logits are those of
    five single steps up to the attention's roundings and the codes that move
    with them, so the checks inside each step are the test; here the cache
    lengths and masks of the two ways are exercised side by side."""
    rng = np.random.default_rng(2)
    m = Model(2, 2)
    ids = torch.from_numpy(rng.integers(0, VOCAB, 40)).to(DEV)
    m.step(m.embed(ids), m.pg.batch([17, 23], [17, 23]), sampling(rng, 2), [16, 39])
    m.step(m.embed(ids[:10]), m.pg.batch([5, 5], [22, 28]), sampling(rng, 8), list(range(8)))
    m.step(m.embed(ids[:2]), m.pg.batch([1, 1], [23, 29]), sampling(rng, 2), [0, 1])


def test_step_in_a_graph_replayed():
    """One decode step captured once and replayed with new embeddings, lengths,
    pages and random numbers in the same buffers, one slot idle; eager work
    between the replays; every replay equals the eager step on a copy."""
    rng = np.random.default_rng(3)
    m = Model(3, 3)
    ids = torch.from_numpy(rng.integers(0, VOCAB, 30)).to(DEV)
    m.step(m.embed(ids), m.pg.batch([9, 20, 1], [9, 20, 1]), sampling(rng, 3), [8, 28, 29], check=False)
    batch = m.pg.batch([1, 1, 1], [10, 21, 0], max_len=96)
    table, start, length = m.pg.keep
    x, params = m.embed(ids[:3]), list(sampling(rng, 3))
    ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in (
        tern.tern_attention_workspace_bytes(m.pg.cache, batch, HQ), tern.tern_sample_workspace_bytes(8, VOCAB))]
    last = torch.arange(3, device=DEV)
    state = (m.pg.k, m.pg.v, m.pg.ks, m.pg.vs)
    keep = [t.clone() for t in state]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.step(x, batch, params, last, check=False, workspaces=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = m.step(x, batch, params, last, check=False, workspaces=ws)
    for t, k in zip(state, keep):
        t.copy_(k)
    lengths = [[10, 21, 0], [11, 22, 2], [12, 0, 3], [17, 23, 4], [33, 24, 5]]
    for i, ln in enumerate(lengths):
        length.copy_(torch.tensor(ln, dtype=torch.int32))
        x.copy_(m.embed(ids[3 * i: 3 * i + 3]))
        for t, n in zip(params, sampling(rng, 3)):
            t.copy_(n)
        before = [t.clone() for t in state]
        eager = [t.clone() for t in m.step(x, batch, params, last, check=False)]
        after = [t.clone() for t in state]
        for t, b in zip(state, before):
            t.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b), "replay %d" % i
        for a, b in zip(state, after):
            assert torch.equal(a, b), "replay %d: cache" % i


def test_two_streams_with_their_own_workspaces():
    """Calls in flight on two streams at once, a workspace each: what each
    gives alone."""
    rng = np.random.default_rng(4)
    models = [Model(5 + i, 2) for i in range(2)]
    steps = []
    for m in models:
        ids = torch.from_numpy(rng.integers(0, VOCAB, 62)).to(DEV)
        batch = m.pg.batch([31, 31], [31, 31], max_len=10 ** 5)
        steps.append((m.embed(ids), batch, sampling(rng, 2), torch.tensor([30, 61], device=DEV)))
    alone = [[t.clone() for t in m.step(*a, check=False)] for m, a in zip(models, steps)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in models]
    outs = [None, None]
    for _ in range(5):
        for i, (m, a) in enumerate(zip(models, steps)):
            with torch.cuda.stream(streams[i]):
                outs[i] = m.step(*a, check=False)
    torch.cuda.synchronize()
    for o, r in zip(outs, alone):
        assert all(torch.equal(x, y) for x, y in zip(o, r))


def test_workspace_refusals():
    pg = Paged(1, 200, 1, 64, 16).upload()
    b = pg.batch([1], [3000], max_len=3000)
    n = tern.tern_attention_workspace_bytes(pg.cache, b, 4)
    assert n > 256
    q, y = torch.zeros((1, 256), device=DEV), torch.zeros((1, 256), device=DEV)
    big = torch.empty(n + 512, dtype=torch.uint8, device=DEV)
    for ws in (None, big[: n - 1], big[8: 8 + n]):
        with pytest.raises(tern.TernError) as e:
            tern.tern_attention(pg.cache, b, q, 256, 4, 0.1, y, 256, ws)
        assert e.value.status == tern.TERN_ERR_WORKSPACE
    x, t = torch.zeros((2, 100), device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    n = tern.tern_sample_workspace_bytes(2, 100)
    for ws in (None, big[:256], torch.empty(n + 512, dtype=torch.uint8, device=DEV)[8: 8 + n]):
        with pytest.raises(tern.TernError) as e:
            tern.tern_sample(x, 2, 100, 100, x[:, 0], x[:, 0], t, ws)
        assert e.value.status == tern.TERN_ERR_WORKSPACE
