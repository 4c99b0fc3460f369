"""What bench.py's lines for the step's operators multiply: data that was made, and
stays the same from call to call."""
import pytest

import bench
from packed_bit_gemv_tern_amd import tern

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_operands_of_the_linears(monkeypatch):
    """Every linear of the feed-forward's lines sees quantised activations, none of them
    memory that nobody wrote, and leaves its residual as it was."""
    empty, linear, seen = torch.empty, tern.tern_linear_epilogue, []
    poison = {torch.float32: float("nan"), torch.int8: 0x55, torch.int32: 0x55555555}

    def poisoned(*size, **kw):
        t = empty(*size, **kw)
        return t.fill_(poison.get(t.dtype, 0x55))

    def checked(w, N, K, M, q, ldq, s, z, y, ldy, res=None, **kw):
        assert z.abs().max() <= 255 and (s > 0).all() and torch.isfinite(s).all()
        assert (q != q[0, 0]).any()
        before = None if res is None else res.clone()
        linear(w, N, K, M, q, ldq, s, z, y, ldy, res=res, **kw)
        assert torch.isfinite(y).all()
        assert res is None or torch.equal(res, before)
        seen.append((M, res is not None))

    def once(fn, calls, **kw):
        fn(0)
        return [1.0] * 10
    monkeypatch.setattr(torch, "empty", poisoned)
    monkeypatch.setattr(tern, "tern_linear_epilogue", checked)
    monkeypatch.setattr(bench, "_event_times", once)
    bench.step_operators(lambda rec: print(rec["workload"], flush=True))
    assert {m for m, _ in seen} == {1, 8, 64, 512, 2048} and any(r for _, r in seen)
