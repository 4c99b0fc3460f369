"""The pages under the cache at the borders of what the calls allow: pools
without rows, rows that a reserve refuses."""
import pytest

from packed_bit_gemv_tern_amd import tern

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from gpu_util import DEV  # noqa: E402


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
