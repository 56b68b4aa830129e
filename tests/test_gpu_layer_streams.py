"""The layer calls on another stream than the current one: what they allocate
belongs to that stream, what they return may be freed on either."""
import pytest

from test_gpu_layer import ROPES, _cache, _cuda, _layer, _rand, _starts  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

PAUSE = 200_000_000  # clock cycles, about 0.1 s


def _calls():
    """Name -> call(stream) returning a list of tensors."""
    lay = _layer(heads=8, d=64, norm="layer", page_size=16, causal_block=1, **ROPES["grid64"])
    n = 700
    kp, vp, bt = _cache(lay, [n])
    x = _rand(1, n, 24, 64, seed=2)
    w, b = _rand(64, seed=3), _rand(64, seed=4)
    table = lay.ac_rope_table()
    kv, st = torch.tensor([n], dtype=torch.int32).cuda(), _starts([n])
    q, k, v = x[:, :, :8], x[:, :, 8:16], x[0, :, 16:]
    g = _rand(1, 8, n, 64, seed=5)

    def back(stream):
        r = lay.ac_qk_norm_rope_backward(g, g, q, k, table=table, w_q=w, w_k=w, b_q=b, b_k=b, stream=stream)
        return [r[name] for name in ("q", "k", "w_q", "b_q", "w_k", "b_k")]

    return lay, {
        "table": lambda s: [lay.ac_rope_table(stream=s)],
        "forward": lambda s: list(lay.ac_qk_norm_rope(q, k, table=table, w_q=w, w_k=w, b_q=b, b_k=b, stream=s)),
        "backward": back,
        "append": lambda s: [lay.ac_cache_append(k[0], v, kp, vp, bt, st, kv, q=q[0], table=table, w_q=w, w_k=w, stream=s)],
        "attn": lambda s: list(lay.ac_cache_attn(q[0], kp, vp, bt, st, kv, lse=True, stream=s)),
    }


@pytest.mark.parametrize("name", ["table", "forward", "backward", "append", "attn"])
def test_outputs_are_the_streams_own(name):
    """Blocks that the current stream has freed but not yet written, behind a
    pause, are not the outputs of a call on another stream."""
    lay, calls = _calls()
    call = calls[name]
    calls["append"](None)
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(side)
    torch.cuda.synchronize()
    torch.cuda._sleep(PAUSE)
    # more of each size than the allocator has free by chance
    held = [torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in want for _ in range(6)]
    for t in held:
        t.fill_(3)
    del held, t
    got = call(side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert lay.get_status() == 0


@pytest.mark.parametrize("name", ["forward", "backward", "append", "attn"])
def test_outputs_are_kept_for_the_caller(name):
    """A result that the caller's stream still has to read is not handed to the
    next call on the side stream when the caller lets go of it."""
    lay, calls = _calls()
    call = calls[name]
    calls["append"](None)
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(PAUSE)
    copies = [t.clone() for t in got]  # behind the pause
    del got
    with torch.cuda.stream(side):
        for t in want:
            for _ in range(3):
                torch.empty_like(t).fill_(5)
    torch.cuda.synchronize()
    for a, b in zip(copies, want):
        assert torch.equal(a, b)
