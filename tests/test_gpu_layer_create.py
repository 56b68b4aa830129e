"""What a layer's creation writes is in place on every stream when it returns."""
import pytest

from test_gpu_layer import _bits, _cache, _cuda, _layer, _rand, _starts  # noqa: F401

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


def test_layers_share_a_workspace():
    """Layers whose calls follow one another on a stream, on the larger one's
    workspace: the same bits as with workspaces of their own."""
    from clustered_sparse_attention_head_b200.layer import AttnLayer, LayerConfig
    cfgs = [LayerConfig(heads=4, d=d, page_size=16, causal_block=1) for d in (64, 128)]
    own = [AttnLayer(c) for c in cfgs]
    ws = max((lay.ws for lay in own), key=torch.numel)
    shared = [AttnLayer(c, workspace=ws) for c in cfgs]
    args = []
    for c in cfgs:
        kp, vp, bt = _cache(own[0] if c.d == 64 else own[1], [3000])
        args.append((_rand(60, 4, c.d, seed=7), kp, vp, bt, _starts([60]), torch.tensor([3000], dtype=torch.int32).cuda()))
    want = [lay.ac_cache_attn(*a) for lay, a in zip(own, args)]
    for _ in range(3):
        got = [lay.ac_cache_attn(*a) for lay, a in zip(shared, args)]
        assert all(torch.equal(_bits(a), _bits(b)) for a, b in zip(got, want))
    assert all(lay.get_status() == 0 for lay in own + shared)
