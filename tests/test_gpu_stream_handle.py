"""The binding launches on torch's current stream unless it is given one."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from packed_bit_gemv_tern_amd import tern  # noqa: E402


def test_current_stream_is_followed():
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    assert tern._stream(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(a):
        assert tern._stream(None) == a.cuda_stream
        with torch.cuda.stream(b):
            assert tern._stream(None) == b.cuda_stream
        assert tern._stream(b) == b.cuda_stream
        assert tern._stream(b.cuda_stream) == b.cuda_stream
    assert tern._stream(None) == torch.cuda.current_stream().cuda_stream
