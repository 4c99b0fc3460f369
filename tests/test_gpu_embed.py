"""The embedding lookup against the oracle, bit for bit: widths that no vector
load divides, strides, unaligned tables and rows, ids outside the table."""
import numpy as np
import pytest

from oracle import step
from packed_bit_gemv_tern_amd import tern

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from gpu_util import DEV, to_dev  # noqa: E402


def run(rng, M, N, K, ldw, ldx, scale=1.0, shift=0, xshift=0, ids=None):
    W = rng.integers(-128, 128, (N, ldw)).astype(np.int8)
    flat = np.zeros(N * ldw + 16, np.int8)
    flat[shift: shift + N * ldw] = W.ravel()
    s = rng.uniform(1e-3, 1e-2, N).astype(np.float32)
    ids = rng.integers(0, N, M).astype(np.int32) if ids is None else np.asarray(ids, np.int32)
    x = torch.full((M * ldx + 8,), float("nan"), device=DEV)
    tern.tern_embed(to_dev(flat)[shift:], to_dev(s), N, K, ldw, to_dev(ids), M, x[xshift:], ldx, scale=scale)
    got = x.cpu().numpy()
    rows = got[xshift: xshift + M * ldx].reshape(M, ldx)
    ref = step.embed(W[:, :K], s, ids, scale)
    assert np.array_equal(rows[:, :K].view(np.uint32), ref.view(np.uint32))
    assert np.isnan(rows[:, K:]).all() and np.isnan(got[:xshift]).all() and np.isnan(got[xshift + M * ldx:]).all()


@pytest.mark.parametrize("K", [1, 3, 4, 15, 16, 64, 100, 255, 256, 260, 1000, 1019, 1024, 4095, 4096, 4100, 5000, 12288])
@pytest.mark.parametrize("M", [1, 5, 33])
def test_rows(M, K):
    rng = np.random.default_rng([M, K])
    run(rng, M, 71, K, K, K, scale=float(np.sqrt(K)))


@pytest.mark.parametrize("ldw,ldx,shift,xshift", [(80, 64, 0, 0), (64, 68, 0, 0), (65, 64, 0, 0), (64, 65, 0, 0),
                                                  (64, 64, 1, 0), (64, 64, 4, 0), (64, 64, 0, 1), (67, 71, 3, 3)])
def test_strides_and_alignments(ldw, ldx, shift, xshift):
    run(np.random.default_rng(1), 9, 30, 64, ldw, ldx, shift=shift, xshift=xshift)


def test_ids_outside_the_table_and_repeated():
    ids = [0, -1, 29, 30, 29, 29, -2 ** 31, 2 ** 31 - 1, 3, 0]
    for K in (64, 61):
        run(np.random.default_rng(2), len(ids), 30, K, K, K, ids=ids, scale=-0.5)


def test_table_past_32_bit_offsets():
    """Rows behind the first 2^31 bytes of a table."""
    N, K = 150000, 16384
    W = torch.zeros((N, K), dtype=torch.int8, device=DEV)
    rows = [0, 131071, 131072, N - 1]
    for i, r in enumerate(rows):
        W[r] = i + 1
    s = torch.full((N,), 0.5, device=DEV)
    x = torch.empty((4, K), device=DEV)
    tern.tern_embed(W, s, N, K, K, to_dev(np.array(rows, np.int32)), 4, x, K)
    assert torch.equal(x, torch.tensor([[0.5], [1.0], [1.5], [2.0]], device=DEV).expand(4, K))


def test_many_rows():
    rng = np.random.default_rng(3)
    N, K, M = 300, 40, 70001
    W = rng.integers(-127, 128, (N, K)).astype(np.int8)
    s = rng.uniform(0.1, 1, N).astype(np.float32)
    ids = rng.integers(-1, N, M).astype(np.int32)
    x = torch.empty((M, K), device=DEV)
    tern.tern_embed(to_dev(W), to_dev(s), N, K, K, to_dev(ids), M, x, K)
    ref = np.where((ids >= 0)[:, None], W[ids].astype(np.float32) * s[ids][:, None], np.float32(0))
    assert np.array_equal(x.cpu().numpy(), ref)
