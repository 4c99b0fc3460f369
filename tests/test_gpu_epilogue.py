"""A linear with its epilogue against the oracle's fp32 steps, bit for bit, and
against fp64; every number of tokens, ragged K, odd N, strides."""
import numpy as np
import pytest

import oracle
from oracle import step
from packed_bit_gemv_tern_amd import tern

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from gpu_util import DEV, gpu_pack, pad_cols, to_dev  # noqa: E402

ACT = {None: tern.TERN_ACT_NONE, "silu": tern.TERN_ACT_SILU, "gelu": tern.TERN_ACT_GELU}


class Side:
    def __init__(self, rng, N, K, bias, hi=0.02):
        w = rng.choice(np.array([-1, 0, 1], np.int8), p=[0.2, 0.6, 0.2], size=(N, K))
        self.s_row = rng.uniform(0.002, hi, N).astype(np.float32)
        self.bias = rng.standard_normal(N).astype(np.float32) if bias else None
        self.packed, self.rowsum, _ = gpu_pack(w)
        self.keep = to_dev(self.s_row), None if self.bias is None else to_dev(self.bias)
        self.dev = tern.make_weights(self.packed, self.keep[0], self.rowsum, self.keep[1])
        self.rp, self.rr, _ = oracle.pack(w)

    @property
    def host(self):
        return self.rp, self.s_row, self.rr, self.bias


def run(M, N, K, gate=False, act=None, bias=False, res=None, extra=0, seed=0, rows=None, sides=None, q=None):
    """rows: the output rows that are checked (all)."""
    rng = np.random.default_rng([M, N, K, seed])
    w = sides[0] if sides else Side(rng, N, K, bias)
    up = (sides[1] if sides else Side(rng, N, K, bias)) if gate else None
    q = rng.integers(-128, 128, (M, K)).astype(np.int8) if q is None else q
    s = rng.uniform(0.01, 0.03, M).astype(np.float32)
    z = rng.integers(-255, 256, M).astype(np.int32)
    ld = N + extra
    y = torch.full((M, ld), float("nan"), device=DEV)
    r = rng.standard_normal((M, ld)).astype(np.float32) if res else None
    rd = None
    if res == "in place":
        y.copy_(to_dev(r))
        rd = y
    elif res:
        rd = to_dev(r)
    qp = pad_cols(q)
    # a single token's row of activations ends with its last column
    qd = to_dev(qp) if M > 1 else to_dev(q)
    tern.tern_linear_epilogue(w.dev, N, K, M, qd, qp.shape[1], to_dev(s), to_dev(z), y, ld,
                              up=None if up is None else up.dev, act=ACT[act], res=rd, ldr=ld if res else 0)
    got = y.cpu().numpy()
    pick = slice(None) if rows is None else rows
    cut = lambda h: (h[0][pick], h[1][pick], h[2][pick], None if h[3] is None else h[3][pick])  # noqa: E731
    ref = step.linear_epilogue(cut(w.host), None if up is None else cut(up.host), K, q, s, z, act,
                               None if r is None else np.ascontiguousarray(r[:, :N][:, pick]))
    mine = np.ascontiguousarray(got[:, :N][:, pick])
    bad = np.argwhere(mine.view(np.uint32) != ref.astype(np.float32).view(np.uint32))
    assert not len(bad), "(%d, %d): %r, not %r; %d of %d" % (*bad[0], mine[tuple(bad[0])], ref[tuple(bad[0])], len(bad),
                                                             mine.size)
    assert np.array_equal(got[:, N:], r[:, N:]) if res == "in place" else np.isnan(got[:, N:]).all()
    return got


@pytest.mark.parametrize("M", [1, 2, 3, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 127, 128, 129, 200, 257, 300])
def test_tokens(M):
    run(M, 96, 320, gate=True, act="silu")
    run(M, 70, 200, act="gelu", bias=True, res="apart", extra=3)


@pytest.mark.parametrize("K", [1, 15, 16, 17, 63, 64, 65, 100, 127, 128, 192, 255, 256, 257, 500, 512, 1019, 1024, 2048, 4096,
                               4100, 12288])
@pytest.mark.parametrize("M", [1, 7, 40, 140])
def test_columns(M, K):
    run(M, 33, K, gate=True, act="silu", res="apart")
    run(M, 48, K, bias=True)


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 31, 33, 64, 127, 128, 129, 255, 256, 257, 300, 1003])
@pytest.mark.parametrize("M", [1, 5, 70, 150])
def test_rows(M, N):
    run(M, N, 128, gate=True, act="gelu", bias=True, res="in place", extra=5)
    run(M, N, 192, act="silu")


@pytest.mark.parametrize("M", [1, 16, 50, 130])
@pytest.mark.parametrize("act", [None, "silu", "gelu"])
@pytest.mark.parametrize("gate", [False, True])
def test_every_epilogue(M, act, gate):
    for bias in (False, True):
        for res in (None, "apart", "in place"):
            run(M, 80, 256, gate=gate, act=act, bias=bias, res=res, extra=16)


def test_several_tiles_and_workgroups():
    run(300, 1100, 640, gate=True, act="silu")
    run(600, 520, 320, res="apart")
    run(70, 4000, 128, gate=True)


@pytest.mark.parametrize("M", [1, 8, 64, 512])
def test_model_shapes(M):
    """The 8B's feed-forward: gate and up, then down onto the residual stream,
    a sample of the rows."""
    pick = np.r_[0:40, 6000:6040, 12248:12288]
    run(M, 12288, 4096, gate=True, act="silu", rows=pick if M < 512 else pick[::6])
    run(M, 4096, 12288, res="in place", rows=pick[:60:3] // 3)


@pytest.mark.parametrize("M,N,K,gate", [
    (300, 4001, 1019, False), (601, 2500, 1030, False), (300, 2501, 2049, True), (1001, 1003, 2050, True),
    (1000, 2497, 1019, False), (577, 4000, 321, False), (600, 2500, 1019, True), (290, 4000, 2048, True),
    (2050, 6001, 700, False), (3000, 4100, 130, False), (2100, 6145, 65, False), (1500, 9001, 577, False),
    (130, 2500, 1019, False), (130, 4001, 1019, True), (1, 70001, 300, True), (9, 65537, 129, False), (16, 66000, 1019, True),
    (1000, 2501, 1019, True), (1001, 4003, 321, True), (600, 4000, 1019, True), (2000, 4003, 130, True)])
def test_large_odd_sizes(M, N, K, gate):
    """Every shape of workgroup at sizes that none divides (tiles with K split, of
    64 tokens, of 128, rows for more tokens, for very many rows): their edges."""
    pick = np.unique(np.r_[0:70, 120:136, 250:262, N // 2: N // 2 + 30, N - 140: N])
    run(M, N, K, gate=gate, act="silu", res="apart" if K % 2 else None, bias=K % 2 == 0, extra=K % 4, rows=pick)


@pytest.mark.parametrize("M,N,K,gate", [
    (1, 300, 16, True), (5, 300, 6416, True), (16, 1003, 12304, False), (9, 1003, 4112, True), (16, 330, 3344, False),
    (16, 4001, 1040, True), (3, 9001, 112, False), (13, 9001, 1296, True), (2, 9001, 6160, False),
    (1, 24593, 272, False), (7, 24593, 304, True), (16, 24593, 48, False),
    (17, 1003, 4099, True), (33, 300, 6401, False), (40, 1003, 1009, True), (130, 2500, 1019, True),
    (17, 4001, 4099, False), (32, 4001, 7001, False), (50, 2003, 4112, False),
    (50, 4001, 4112, True), (64, 4001, 6403, False), (33, 2501, 6416, True),
    (50, 9001, 4112, False), (300, 4001, 1019, False), (130, 4001, 2050, True), (300, 2501, 2049, True),
    (250, 4001, 4099, False), (256, 4001, 12304, False), (200, 4001, 7001, True), (200, 2003, 2047, True),
    (1100, 1003, 1019, False)])
def test_streams(M, N, K, gate):
    """The shapes whose waves share K (16 rows in four, eight and sixteen waves, 64
    rows; 32 tokens, 32 rows x 32 tokens in four and eight waves; tiles of 64 rows):
    steps that some waves have and others not, pieces and blocks that end inside,
    odd edges."""
    pick = np.unique(np.r_[0:min(N, 70), N // 2: N // 2 + 30, N - 70: N])
    run(M, N, K, gate=gate, act="silu", res="apart" if M % 2 else None, bias=M % 2 == 0, extra=M % 4, rows=pick)


def test_strides_past_32_bits():
    """Rows of activations so far apart that a block of them passes 2^31 bytes,
    and outputs behind 2^31 elements."""
    M, N, K = 100, 64, 128
    rng = np.random.default_rng(9)
    side = Side(rng, N, K, False)
    q = to_dev(rng.integers(-128, 128, (M, K)).astype(np.int8))
    s, z = to_dev(rng.uniform(0.01, 0.03, M).astype(np.float32)), torch.zeros(M, dtype=torch.int32, device=DEV)
    want = torch.empty((M, N), device=DEV)
    tern.tern_linear_epilogue(side.dev, N, K, M, q, K, s, z, want, N)
    ld = 24 << 20
    far_q = torch.empty(M * ld, dtype=torch.int8, device=DEV)
    far_y = torch.empty(M * ld, device=DEV)
    far_q.view(M, ld)[:, :K] = q
    tern.tern_linear_epilogue(side.dev, N, K, M, far_q, ld, s, z, far_y, ld)
    assert torch.equal(far_y.view(M, ld)[:, :N], want)


def test_equals_the_chain_of_calls():
    """The gated linear gives what the two linears and the stack launch's gate
    give: its codes, scale and zero point, bit for bit."""
    rng = np.random.default_rng(5)
    M, N, K = 24, 512, 1024
    g, u, down = Side(rng, N, K, False), Side(rng, N, K, False), Side(rng, 64, N, False)
    q = to_dev(rng.integers(-128, 128, (M, K)).astype(np.int8))
    s, z = to_dev(rng.uniform(0.01, 0.03, M).astype(np.float32)), to_dev(rng.integers(-8, 9, M).astype(np.int32))
    h = torch.empty((M, N), device=DEV)
    tern.tern_linear_epilogue(g.dev, N, K, M, q, K, s, z, h, N, up=u.dev, act=tern.TERN_ACT_SILU)
    fused = [torch.empty((M, N), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV),
             torch.empty(M, dtype=torch.int32, device=DEV)]
    tern.tern_quantize_act(h, M, N, N, fused[0], N, fused[1], fused[2])
    ys = [torch.empty((M, N), device=DEV) for _ in range(2)]
    for side, y in zip((g, u), ys):
        tern.tern_gemm_smallM(side.packed, side.keep[0], side.rowsum, N, K, M, q, K, s, z, y, N)
    chain = [torch.empty_like(t) for t in fused]
    out = torch.empty((M, 64), device=DEV)
    desc = tern.make_desc(down.packed, down.keep[0], down.rowsum, 64, N, chain[0], N, chain[1], chain[2], out, 64,
                          x=ys[0], ldx=N, x_up=ys[1])
    ws = torch.empty(tern.tern_linear_stack_workspace_bytes(1, M), dtype=torch.uint8, device=DEV)
    tern.tern_linear_stack(tern.tern_linear_stack_prepare([desc], M, ws))
    for a, b in zip(fused, chain):
        assert torch.equal(a, b)


def test_activations_at_the_ends_of_their_range():
    """Outputs from -1e6 to 1e6: gates that vanish, exponentials that overflow."""
    rng = np.random.default_rng(6)
    sides = [Side(rng, 64, 256, True, hi=40.0) for _ in range(2)]
    for act in ("silu", "gelu"):
        for M in (3, 80):
            got = run(M, 64, 256, gate=True, act=act, sides=sides, seed=act == "gelu")
            assert np.isfinite(got).all()


def test_zero_sums_and_zero_scales():
    rng = np.random.default_rng(7)
    for M in (2, 90):
        side = Side(rng, 40, 128, False)
        q = np.zeros((M, 128), np.int8)
        # (a sum of zero, less z times the row sum)
        run(M, 40, 128, act="silu", sides=[side], q=q)
        side.keep[0][::2] = 0
        side.s_row[::2] = 0
        run(M, 40, 128, act="gelu", sides=[side])


def test_unaligned_outputs():
    """y and res rows of any 4-byte alignment."""
    rng = np.random.default_rng(8)
    for M in (4, 130):
        N, K = 256, 128
        side = Side(rng, N, K, False)
        q, s, z = (to_dev(a) for a in (rng.integers(-128, 128, (M, K)).astype(np.int8),
                                       rng.uniform(0.01, 0.03, M).astype(np.float32), np.zeros(M, np.int32)))
        want = torch.empty((M, N), device=DEV)
        r = to_dev(rng.standard_normal((M, N)).astype(np.float32))
        tern.tern_linear_epilogue(side.dev, N, K, M, q, K, s, z, want, N, res=r, ldr=N)
        for ld, shift in ((N, 1), (N + 1, 0), (N + 2, 3)):
            y = torch.zeros(M * ld + 4, device=DEV)
            rr = torch.zeros(M * ld + 4, device=DEV)
            view = lambda t: t[shift: shift + M * ld].view(M, ld)  # noqa: E731
            view(rr)[:, :N] = r
            tern.tern_linear_epilogue(side.dev, N, K, M, q, K, s, z, view(y), ld, res=view(rr), ldr=ld)
            assert torch.equal(view(y)[:, :N], want)
            assert not view(y)[:, N:].any() and not y[:shift].any() and not y[shift + M * ld:].any()
