"""Drafted tokens verified in one pass against the same tokens one by one: the
cache bit for bit, each row's attention within both ways' roundings."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from packed_bit_gemv_tern_amd import tern  # noqa: E402
from attention_util import reference  # noqa: E402
from gpu_util import DEV, to_dev  # noqa: E402
from kv_util import Paged  # noqa: E402


def step(pg, new, length, k, v, q):
    """Append and attention of the given rows."""
    b = pg.batch(new, length)
    rows, heads, D = q.shape
    dev = [to_dev(a.reshape(rows, -1)) for a in (k, v, q)]
    y = torch.full((rows, heads * D), 77.0, device=DEV)
    tern.tern_kv_append(pg.cache, b, dev[0], pg.heads * D, dev[1], pg.heads * D)
    ws = torch.full((tern.tern_attention_workspace_bytes(pg.cache, b, heads),), 255, dtype=torch.uint8, device=DEV)
    tern.tern_attention(pg.cache, b, dev[2], heads * D, heads, D ** -0.5, y, heads * D, ws)
    torch.cuda.synchronize()
    return y.cpu().numpy().reshape(q.shape)


@pytest.mark.parametrize("held", [(0, 0), (1, 30), (13, 200), (16, 31), (1021, 2500)])
@pytest.mark.parametrize("new,group,P,D", [(5, 4, 16, 64), (2, 1, 32, 128), (8, 4, 64, 128), (17, 8, 16, 128)])
def test_one_pass_and_single_tokens(held, new, group, P, D):
    """The new tokens shrink, so a page's scale is that of the first one to
    reach it, whichever way they come."""
    pg = Paged(2, -(-(max(held) + new) // P), 2, D, P, seed=new).upload()
    rng = pg.rng
    shrink = (0.99 ** np.arange(new))[None, :, None, None]
    k, v = (np.float32(np.sign(rng.normal(0, 1, (2, 1, 2, D))) * rng.uniform(0.2, 1, (2, new, 2, D)) * shrink)
            for _ in range(2))
    for a in (k, v):
        a[:, :, :, 3] = 1.5 * shrink[..., 0]  # (the largest element of every row)
    q = np.float32(rng.normal(0, 2, (2, new, 2 * group, D)))
    before = [t.clone() for t in (pg.k, pg.v, pg.ks, pg.vs)]
    flat = lambda a: np.ascontiguousarray(a.reshape((-1,) + a.shape[2:]))  # noqa: E731
    at_once = step(pg, [new, new], [h + new for h in held], flat(k), flat(v), flat(q))
    for name, t in (("k", pg.k), ("v", pg.v), ("k_scale", pg.ks), ("v_scale", pg.vs)):
        getattr(pg.host, name)[:] = t.cpu().numpy()
    tol = reference(pg, flat(q), D ** -0.5)[1]
    after = [t.clone() for t in (pg.k, pg.v, pg.ks, pg.vs)]
    for t, b in zip((pg.k, pg.v, pg.ks, pg.vs), before):
        t.copy_(b)
    single = np.stack([step(pg, [1, 1], [h + i + 1 for h in held], *(np.ascontiguousarray(a[:, i]) for a in (k, v, q)))
                       for i in range(new)], 1)
    for t, b in zip((pg.k, pg.v, pg.ks, pg.vs), after):
        assert torch.equal(t, b)
    assert (np.abs(flat(single) - at_once) <= 2 * tol).all()
