"""A linear with its epilogue at the borders of what its header allows."""
import numpy as np
import pytest

from packed_bit_gemv_tern_amd import tern

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from gpu_util import DEV, to_dev  # noqa: E402
from test_gpu_epilogue import Side  # noqa: E402


@pytest.mark.parametrize("M", [2, 16, 17, 40, 70, 140, 300])
@pytest.mark.parametrize("K,ldq", [(1, 16), (67, 80), (1019, 1024), (1008, 1040), (1024, 1088)])
def test_bytes_behind_a_row(M, K, ldq):
    """What stands behind K in a row of activations does not matter."""
    rng = np.random.default_rng([M, K])
    N = 130
    w, up = Side(rng, N, K, True), Side(rng, N, K, False)
    q = rng.integers(-128, 128, (M, K)).astype(np.int8)
    s, z = to_dev(rng.uniform(0.01, 0.03, M).astype(np.float32)), to_dev(rng.integers(-255, 256, M).astype(np.int32))
    outs = []
    for fill in (0, -128, 127, None):
        rows = np.full((M, ldq), fill, np.int8) if fill is not None else rng.integers(-128, 128, (M, ldq)).astype(np.int8)
        rows[:, :K] = q
        y = torch.full((2, M, N), float("nan"), device=DEV)
        d = to_dev(rows)
        tern.tern_linear_epilogue(w.dev, N, K, M, d, ldq, s, z, y[0], N, up=up.dev, act=tern.TERN_ACT_GELU)
        tern.tern_linear_epilogue(w.dev, N, K, M, d, ldq, s, z, y[1], N)
        outs.append(y)
    plain = torch.empty((M, N), device=DEV)
    tern.tern_gemm_smallM(w.packed, w.keep[0], w.rowsum, N, K, M, d, ldq, s, z, plain, N)
    assert torch.equal(outs[0][1], plain + w.keep[1])
    assert all(torch.equal(outs[0], y) for y in outs[1:])
