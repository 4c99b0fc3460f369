"""Sampling against the oracle: token and number of kept tokens equal, the
probability within two fp32 roundings."""
import numpy as np
import pytest

from oracle import decode

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from packed_bit_gemv_tern_amd import tern  # noqa: E402
from gpu_util import DEV, to_dev  # noqa: E402


def draw(x, T, u, top_k=None, top_p=None, min_p=None, extra=0):
    """(token, prob, kept) of the library, checked against the oracle's."""
    M, N = x.shape
    xd = torch.full((M, N + extra), float("inf"), device=DEV)
    xd[:, :N] = to_dev(x)
    dev = [None if a is None else to_dev(np.asarray(a, t)) for a, t in (
        (T, np.float32), (u, np.float32), (top_k, np.int32), (top_p, np.float32), (min_p, np.float32))]
    token = torch.full((M,), -7, dtype=torch.int32, device=DEV)
    kept = torch.full((M,), -7, dtype=torch.int32, device=DEV)
    prob = torch.full((M,), -7.0, device=DEV)
    ws = torch.full((tern.tern_sample_workspace_bytes(M, N),), 255, dtype=torch.uint8, device=DEV)
    tern.tern_sample(xd, M, N, N + extra, dev[0], dev[1], token, ws, top_k=dev[2], top_p=dev[3], min_p=dev[4],
                     prob=prob, kept=kept)
    torch.cuda.synchronize()
    got = token.cpu().numpy(), prob.cpu().numpy(), kept.cpu().numpy()
    for i in range(M):
        at = lambda a: None if a is None else np.float32(a[i]) if a is not top_k else int(a[i])  # noqa: E731
        ref = decode.sample(x[i], at(T), at(u), at(top_k), at(top_p), at(min_p))
        assert (got[0][i], got[2][i]) == (ref[0], ref[2]), (i, got[0][i], got[2][i], ref)
        assert abs(got[1][i] - ref[1]) <= 2 ** -23 * ref[1], (i, got[1][i], ref)
    return got


def logits(rng, M, N, kind="peaked"):
    x = rng.normal(0, 2.2, (M, N))
    if kind == "peaked":
        for r in x:
            at = rng.integers(0, N, max(1, min(N, 200)))
            r[at] = rng.uniform(4, 14, len(at))
    elif kind == "coarse":      # many equal logits, as from a head of few bits
        x = np.rint(x * 4) / 4
    elif kind == "flat":
        x = x * 0 + 1.5
    elif kind == "masked":
        x[rng.random((M, N)) < 0.9] = -np.inf
    return x.astype(np.float32)


FILTERS = {
    "none": {},
    "k": {"top_k": True},
    "p": {"top_p": True},
    "min_p": {"min_p": True},
    "kp": {"top_k": True, "top_p": True},
    "all": {"top_k": True, "top_p": True, "min_p": True},
}


def params(rng, M, names):
    out = {"T": rng.uniform(0.3, 1.5, M), "u": rng.random(M)}
    if "top_k" in names:
        out["top_k"] = rng.integers(1, 300, M)
    if "top_p" in names:
        out["top_p"] = rng.uniform(0.1, 0.999, M)
    if "min_p" in names:
        out["min_p"] = rng.uniform(0.001, 0.3, M)
    return out


@pytest.mark.parametrize("names", list(FILTERS))
@pytest.mark.parametrize("kind", ["peaked", "coarse", "flat", "masked"])
@pytest.mark.parametrize("M,N", [(3, 1), (5, 2), (4, 100), (6, 1025), (3, 32003), (2, 151936)])
def test_filters(names, kind, M, N):
    rng = np.random.default_rng([M, N, len(names), len(kind)])
    draw(logits(rng, M, N, kind), **params(rng, M, FILTERS[names]), extra=int(N % 3))


def test_many_rows_with_their_own_parameters():
    rng = np.random.default_rng(5)
    M, N = 200, 5000
    p = params(rng, M, ("top_k", "top_p", "min_p"))
    p["top_k"][::2] = 0
    p["top_p"][::3] = 1.0
    p["min_p"][::5] = 0.0
    p["T"][::7] = 0.0
    draw(logits(rng, M, N), **p)


def test_every_random_number_reaches_its_token():
    """Eight equal tokens: u = i / 8 starts token i, and just under it ends
    the one before."""
    x = np.full((16, 8), 3.0, np.float32)
    edge = np.arange(8) / 8
    u = np.concatenate([edge, np.nextafter(edge.astype(np.float32) + np.float32(0.125), np.float32(0))])
    tok, prob, kept = draw(x, np.ones(16), u)
    assert tok.tolist() == list(range(8)) * 2 and (prob == 0.125).all() and (kept == 8).all()


def test_ties_at_the_cut_go_to_the_lowest_index():
    x = np.zeros((4, 300), np.float32)
    x[:, 100:110] = 5.0
    tok, _, kept = draw(x, np.ones(4), [0.0, 0.3, 0.6, 0.9999], top_k=[3] * 4)
    assert (kept == 3).all() and set(tok) <= {100, 101, 102}
    draw(x, np.ones(4), [0.0, 0.3, 0.6, 0.9999], top_p=[0.5] * 4)
    draw(x, np.ones(4), [0.1, 0.3, 0.6, 0.9999], top_k=[200] * 4, top_p=[0.9999] * 4)


def test_greedy_and_extremes():
    rng = np.random.default_rng(6)
    x = logits(rng, 12, 4000)
    x[0, :] = -np.inf                      # nothing to draw
    x[1, :] = np.nan
    x[2, 7] = np.inf                       # all of the weight
    x[3, [5, 900]] = np.inf
    x[4, ::2] = np.nan
    x[5, :] = -np.inf
    x[5, 3999] = -1e30                     # one token left
    x[6, :] = np.float32(-3.4e38)
    x[7, 10], x[7, 20] = 0.0, -0.0
    x[7, 30:] = -50.0
    T = np.ones(12)
    T[8], T[9], T[10], T[11] = 0.0, np.nan, 1e-30, np.inf
    for extra in ({}, {"top_k": [2] * 12}, {"top_p": [0.3] * 12}, {"min_p": [0.9] * 12}):
        tok, prob, kept = draw(x, T, rng.random(12), **extra)
        assert tok[0] == -1 and tok[1] == -1 and kept[0] == 0
        assert tok[2] == 7 and prob[2] == 1.0


def test_parameters_out_of_range_are_no_filter():
    rng = np.random.default_rng(7)
    x = logits(rng, 4, 1000)
    u = rng.random(4)
    a = draw(x, np.ones(4), u)
    b = draw(x, np.ones(4), u, top_k=[0, -5, 1000, 2 ** 31 - 1], top_p=[1.0, 2.0, np.nan, np.inf],
             min_p=[0.0, -1.0, np.nan, 0.0])
    assert all(np.array_equal(p, q) for p, q in zip(a, b))
    draw(x, np.ones(4), u, top_p=[0.0, -1.0, 1e-30, 0.5], min_p=[1.0, 0.0, 7.0, 2.0])


def test_rows_alike_draw_alike():
    """The same row, many times: the sums do not depend on their order."""
    rng = np.random.default_rng(8)
    x = np.repeat(logits(rng, 1, 151936), 40, 0)
    tok, prob, kept = draw(x[:2], [0.9] * 2, [0.77] * 2, top_p=[0.95] * 2)
    xd = to_dev(x)
    f = lambda v: torch.full((40,), v, device=DEV)  # noqa: E731
    token = torch.empty(40, dtype=torch.int32, device=DEV)
    p, ws = f(0.0), torch.empty(tern.tern_sample_workspace_bytes(40, 151936), dtype=torch.uint8, device=DEV)
    tern.tern_sample(xd, 40, 151936, 151936, f(0.9), f(0.77), token, ws, top_p=f(0.95), prob=p)
    assert (token == int(tok[0])).all() and (p == float(prob[0])).all()


def test_cut_far_below_the_maximum():
    """A cut among tokens whose weight is next to nothing: the first k are
    counted all the same, and a tiny min_p is heeded."""
    rng = np.random.default_rng(9)
    x = rng.uniform(-80, 0, (6, 3000)).astype(np.float32)
    x[:, 77] = 1.0
    T, u = [0.5, 1.0, 0.2, 0.5, 1.0, 0.2], rng.random(6)
    for k in (500, 2999, 3000):
        draw(x, T, u, top_k=[k] * 6)
        draw(x, T, u, top_k=[k] * 6, min_p=[1e-20, 1e-16, 1e-30, 1e-12, 3e-14, 1e-5])
        draw(x, T, u, top_k=[k] * 6, top_p=[0.999] * 6)


@pytest.mark.parametrize("n", [1, 2, 500, 2047, 2048, 2049, 2500])
def test_cut_among_many_close_logits(n):
    """Lists at, under and over the length that is ordered at once."""
    rng = np.random.default_rng(n)
    x = np.full((3, 9000), -20.0, np.float32)
    for r in x:
        r[rng.permutation(9000)[:n]] = rng.uniform(1.0, 1.02, n)
    u = rng.random(3)
    draw(x, [1.0] * 3, u, top_k=[max(1, n // 2)] * 3)
    draw(x, [1.0] * 3, u, top_p=[0.4] * 3)
    draw(x, [1.0] * 3, u, top_k=[max(1, n - 1)] * 3, top_p=[0.7] * 3, min_p=[0.5] * 3)


@pytest.mark.parametrize("names", ["none", "kp", "min_p"])
def test_longest_rows_and_unaligned_ones(names):
    rng = np.random.default_rng(10)
    N = tern.TERN_SAMPLE_MAX_N
    draw(logits(rng, 1, N), **params(rng, 1, FILTERS[names]))
    # a row that starts 4 bytes past a 16-byte border
    x, p = logits(rng, 1, 50001), params(rng, 1, FILTERS[names])
    buf = torch.zeros(50005, device=DEV)
    buf[1:50002] = to_dev(x[0])
    dev = {k: to_dev(np.asarray(v, np.int32 if k == "top_k" else np.float32)) for k, v in p.items()}
    token = torch.empty(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(tern.tern_sample_workspace_bytes(1, 50001), dtype=torch.uint8, device=DEV)
    tern.tern_sample(buf[1:], 1, 50001, 50001, dev["T"], dev["u"], token, ws, top_k=dev.get("top_k"),
                     top_p=dev.get("top_p"), min_p=dev.get("min_p"))
    one = lambda k: None if k not in p else dev[k].cpu().numpy()[0]  # noqa: E731
    assert int(token[0]) == decode.sample(x[0], one("T"), one("u"), one("top_k"), one("top_p"), one("min_p"))[0]


def test_cuts_of_some_rows_and_not_of_others_at_every_chunk_length():
    """One tile per chunk, four, and sixteen: rows with and without filters,
    greedy and empty ones side by side."""
    rng = np.random.default_rng(11)
    for M, N in ((2, 100000), (40, 60000), (300, 33000)):
        x = logits(rng, M, N)
        x[1::9] = -np.inf
        p = params(rng, M, ("top_k", "top_p", "min_p"))
        p["top_k"][::2] = 0
        p["top_p"][::3] = 1.0
        p["min_p"][::5] = 0.0
        p["T"][::7] = 0.0
        draw(x, **p)
