"""What a layer's creation writes is in place on every stream when it returns."""
import pytest

from test_gpu_layer import _cuda, _layer  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_layer_is_ready_on_every_stream():
    """Behind work queued on the default stream, and on the stream current at
    its creation, a new layer's status block is cleared and its workspace free
    when the constructor returns: both streams have nothing left to do."""
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    lay = _layer(heads=2, d=64, page_size=16)
    assert torch.cuda.default_stream().query()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        other = _layer(heads=2, d=64, page_size=16)
        assert side.query() and torch.cuda.default_stream().query()
    assert lay.get_status(side) == 0 and other.get_status() == 0
