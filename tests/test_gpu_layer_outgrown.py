"""A token stream that outgrows its table of positions is reported."""
import pytest

from test_gpu_layer import _cache, _cuda, _layer, _rand, _starts  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _append(rope_dims, rope_max, kv, new, pos=None):
    lay = _layer(heads=2, d=64, norm="none", page_size=16, rope_dims=rope_dims, rope_max=rope_max)
    kp, vp, bt = _cache(lay, [kv])
    k, v, q = (_rand(new, 2, 64, seed=i) for i in (1, 2, 3))
    if pos is not None:
        pos = pos.int().cuda()
    qo = lay.ac_cache_append(k, v, kp, vp, bt, _starts([new]), torch.tensor([kv], dtype=torch.int32).cuda(), q=q,
                             table=lay.ac_rope_table(), pos=pos)
    place = torch.arange(kv - new, kv).cuda()
    return lay, q, qo, k, kp[bt[0].long()[place // 16], :, place % 16]


def test_one_axis():
    """Positions 0 .. 49 fit the table; the token at 50 is written unrotated, as
    before, and recorded."""
    from clustered_sparse_attention_head_b200 import _abi
    lay, *_ = _append((64,), (50,), 50, 7)
    assert lay.get_status() == 0
    lay, q, qo, k, kc = _append((64,), (50,), 51, 7)
    assert lay.get_status() == _abi.AC_ERR_INVALID_ARG
    assert torch.equal(qo[-1], q[-1]) and torch.equal(kc[-1], k[-1])
    assert not torch.equal(qo[-2], q[-2])
    assert lay.get_status() == 0
    # a negative position given with the call still says "not rotated", without an error
    pos = torch.arange(44, 51)[:, None]
    pos[-1] = -1
    lay, q, qo, k, kc = _append((64,), (50,), 51, 7, pos)
    assert lay.get_status() == 0
    assert torch.equal(qo[-1], q[-1]) and torch.equal(kc[-1], k[-1])


def test_text_behind_a_grid():
    """On a grid of several axes the tokens behind it are text: no error."""
    lay, q, qo, k, kc = _append((16, 24), (5, 10), 53, 7)
    assert lay.get_status() == 0
    assert torch.equal(qo[-3:], q[-3:]) and torch.equal(kc[-3:], k[-3:])
