"""A sequence's attention does not depend on what the stacked tensors hold for
other sequences, to the bit."""
import pytest

from test_gpu_layer import _bits, _cache, _cuda, _layer, _rand, _starts  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("heads, kv_heads, d, new, kv", [
    (40, 40, 128, 20, 1500),    # rows 20 .. of our tile are the next sequence's
    (200, 40, 64, 30, 1100),    # 25 tokens a tile: the second one holds 5 of ours and 20 of the next sequence's
    (120, 40, 128, 50, 1300),   # 42 tokens a tile, rows 126 and 127 are nobody's
])
def test_neighbours_queries(heads, kv_heads, d, new, kv):
    """Every other sequence's queries are made 40 times as large: in our tiles
    their scores grow from chunk to chunk by more than the threshold at which a
    row's reference maximum moves, ours do not.  Ours keep their bits.  (More
    units than the GPU has SMs: none is cut down to a single chunk.)"""
    seqs = 4
    lay = _layer(heads=heads, kv_heads=kv_heads, d=d, page_size=64, causal_block=1)
    kp, vp, bt = _cache(lay, [kv] * seqs)
    for s in range(seqs):  # later pages hold larger keys
        pages = bt[s][:-(-kv // 64)].long()
        kp[pages] *= torch.linspace(0.5, 1.5, len(pages), device="cuda")[:, None, None, None].to(kp.dtype)
    q = _rand(seqs, new, heads, d, seed=7)
    lens = torch.tensor([kv] * seqs, dtype=torch.int32).cuda()
    outs = []
    for scale in (0.0, 1.0, 40.0):
        x = q.clone()
        x[1::2] *= scale
        out, lse = lay.ac_cache_attn(x.flatten(0, 1), kp, vp, bt, _starts([new] * seqs), lens, max_q=new, max_kv=kv, lse=True)
        outs.append([_bits(t.unflatten(0, (seqs, new))[::2]) for t in (out, lse)])
    assert lay.get_status() == 0
    for got in outs[1:]:
        assert torch.equal(got[0], outs[0][0]) and torch.equal(got[1], outs[0][1])
