"""ac_qk_norm_rope under torch's autograd: its outputs carry the gradients of
ac_qk_norm_rope_backward to every input that asks for one."""
import pytest

import layer_util as U
from test_gpu_layer import ROPES, _bits, _cuda, _layer, _rand  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

NAMES = ("q", "k", "w_q", "w_k", "b_q", "b_k")


def _case(norm="layer", dt="bf16", rope="grid64", heads=6, kv_heads=3, batch=2, n=29):
    lay = _layer(heads=heads, kv_heads=kv_heads, d=64, dtype=dt, norm=norm, **ROPES[rope])
    x = _rand(batch, n, heads + kv_heads, 64, dtype=lay.dtype, seed=3, scale=2.0)
    w = {name: _rand(64, dtype=lay.dtype, seed=13 + i) for i, name in enumerate(NAMES[2:])} if norm != "none" else {}
    g = _rand(batch, heads, n, 64, dtype=lay.dtype, seed=8), _rand(batch, kv_heads, n, 64, dtype=lay.dtype, seed=9)
    return lay, x, w, g, lay.ac_rope_table()


@pytest.mark.parametrize("norm, dt, rope", [("layer", "bf16", "grid64"), ("rms", "f32", "half"), ("none", "bf16", "line")])
def test_same_gradients_as_the_call(norm, dt, rope):
    lay, x, w, (gq, gk), table = _case(norm, dt, rope)
    want = lay.ac_qk_norm_rope_backward(gq, gk, x[:, :, :6], x[:, :, 6:], table=table, **w)
    plain = lay.ac_qk_norm_rope(x[:, :, :6], x[:, :, 6:], table=table, **w)
    px = x.clone().requires_grad_()
    pw = {name: t.clone().requires_grad_() for name, t in w.items()}
    qo, ko = lay.ac_qk_norm_rope(px[:, :, :6], px[:, :, 6:], table=table, **pw)
    assert qo.requires_grad and ko.requires_grad
    assert torch.equal(qo, plain[0]) and torch.equal(ko, plain[1])
    torch.autograd.backward((qo, ko), (gq, gk))
    assert torch.equal(_bits(px.grad[:, :, :6]), _bits(want["q"])) and torch.equal(_bits(px.grad[:, :, 6:]), _bits(want["k"]))
    for name, t in pw.items():
        assert torch.equal(_bits(t.grad), _bits(want[name])), name
    assert lay.get_status() == 0


def test_only_what_asks():
    """One input with a gradient, one output used, and none under no_grad."""
    lay, x, w, (gq, gk), table = _case()
    q, k = x[:, :, :6].clone().requires_grad_(), x[:, :, 6:].clone()
    qo, ko = lay.ac_qk_norm_rope(q, k, table=table, **w)
    qo.backward(gq)
    want = lay.ac_qk_norm_rope_backward(gq, None, q.detach(), None, table=table, w_q=w["w_q"])
    assert torch.equal(q.grad, want["q"]) and k.grad is None
    wk = w["w_k"].clone().requires_grad_()
    none, ko = lay.ac_qk_norm_rope(None, k, table=table, w_k=wk, b_k=w["b_k"])
    assert none is None
    ko.backward(gk)
    want = lay.ac_qk_norm_rope_backward(None, gk, None, k, table=table, w_k=w["w_k"])
    assert torch.equal(wk.grad, want["w_k"])
    with torch.no_grad():
        assert not lay.ac_qk_norm_rope(q, k, table=table, **w)[0].requires_grad
    assert not lay.ac_qk_norm_rope(q.detach(), k, table=table, **w)[0].requires_grad
    assert lay.get_status() == 0


def test_gradients_of_any_strides():
    """A sum's gradient (strides of 0), a transposed one and a sliced one, whose
    rows begin on odd elements."""
    lay, x, w, (gq, _), table = _case()
    q = x[:, :, :6].clone().requires_grad_()
    pos = torch.stack(torch.meshgrid(torch.arange(2), torch.arange(3), torch.arange(4), indexing="ij"), -1).flatten(0, 2)
    pos = torch.cat([pos, torch.full((5, 3), -1)]).int().cuda()

    def grad(loss):
        q.grad = None
        loss(lay.ac_qk_norm_rope(q, None, table=table, pos=pos, w_q=w["w_q"])[0]).backward()
        return q.grad

    def want(g):
        return lay.ac_qk_norm_rope_backward(g, None, q.detach(), None, table=table, pos=pos, w_q=w["w_q"])["q"]

    assert torch.equal(grad(lambda y: y.sum()), want(torch.ones_like(gq)))
    gt = gq.transpose(1, 2).contiguous()
    assert torch.equal(grad(lambda y: (y.transpose(1, 2) * gt).sum()), want(gq))
    odd = torch.zeros(2, 6, 29, 65, dtype=lay.dtype, device="cuda")
    odd[..., 1:] = gq
    y = lay.ac_qk_norm_rope(q, None, table=table, pos=pos, w_q=w["w_q"])[0]
    q.grad = None
    torch.autograd.backward(y, odd[..., 1:])
    assert torch.equal(q.grad, want(gq))
    assert lay.get_status() == 0


def test_a_training_step():
    """Scores of q and k in torch behind the call: its gradients are the 64-bit
    forms' of the upstream gradients that torch arrives with, and a second
    backward adds to them."""
    lay, x, w, _, table = _case("rms", "f32", heads=4, kv_heads=4)
    x = x.requires_grad_()
    w = {name: t.requires_grad_() for name, t in w.items() if name.startswith("w")}
    pos = U.grid_pos(29, lay.cfg.rope_max)
    for step in (1, 2):
        qo, ko = lay.ac_qk_norm_rope(x[:, :, :4], x[:, :, 4:], table=table, **w)
        qo.retain_grad()
        ko.retain_grad()
        torch.softmax(qo @ ko.transpose(2, 3) / 8, -1).square().sum().backward()
        for name, g, part in (("q", qo.grad, slice(0, 4)), ("k", ko.grad, slice(4, 8))):
            dx, dw, _ = U.backward(lay.cfg, g.double().cpu().transpose(1, 2), x.detach()[:, :, part].double().cpu(),
                                   w["w_" + name].detach().double().cpu(), pos)
            for got, ref in ((x.grad[:, :, part], dx), (w["w_" + name].grad, dw)):
                # the bounds of the call's own tests come to under 1,000 roundings of the largest value
                err = (got.double().cpu() - step * ref).abs().max()
                assert err <= step * 1000 * U.EPS32 * ref.abs().max(), (name, float(err))
    w["w_q"].grad.mul_(0.5)  # as an optimiser or a clipping of norms would
    assert lay.get_status() == 0


def test_given_outputs_and_changed_inputs():
    """Outputs given by the caller cannot join the graph (as with torch's own out=):
    an input that asks for a gradient is refused then, not cut off; and an input
    changed in place before backward() is torch's error."""
    lay, x, w, (gq, _), table = _case()
    q = x[:, :, :6].clone().requires_grad_()
    with pytest.raises(ValueError, match="q_out"):
        lay.ac_qk_norm_rope(q, None, table=table, q_out=torch.empty_like(gq))
    with torch.no_grad():
        out = torch.empty_like(gq)
        assert lay.ac_qk_norm_rope(q, None, table=table, q_out=out)[0] is out
    h = q * 1
    y = lay.ac_qk_norm_rope(h, None, table=table, w_q=w["w_q"])[0]
    with torch.no_grad():
        h.mul_(2)
    with pytest.raises(RuntimeError):
        y.backward(gq)


def test_other_stream_and_graph():
    """Forward on a side stream, backward where torch puts it; and a captured
    forward and backward replayed on new inputs."""
    lay, x, w, (gq, gk), table = _case()
    want = lay.ac_qk_norm_rope_backward(gq, gk, x[:, :, :6], x[:, :, 6:], table=table, w_q=w["w_q"])
    px = x.clone().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        qo, ko = lay.ac_qk_norm_rope(px[:, :, :6], px[:, :, 6:], table=table, w_q=w["w_q"])
    torch.cuda.current_stream().wait_stream(side)
    torch.autograd.backward((qo, ko), (gq, gk))
    torch.cuda.synchronize()
    assert torch.equal(px.grad[:, :, :6], want["q"])
    px.grad = None
    qo, ko = lay.ac_qk_norm_rope(px[:, :, :6], px[:, :, 6:], table=table, w_q=w["w_q"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.autograd.backward((qo, ko), (gq, gk))
    torch.cuda.synchronize()
    assert torch.equal(px.grad[:, :, :6], want["q"])
    # one graph of both passes
    static = x.clone().requires_grad_()

    def step():
        a, b = lay.ac_qk_norm_rope(static[:, :, :6], static[:, :, 6:], table=table, w_q=w["w_q"])
        return torch.autograd.grad((a, b), static, (gq, gk))[0]

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (21, 22):
        new = _rand(*x.shape, dtype=lay.dtype, seed=seed)
        with torch.no_grad():
            static.copy_(new)
        graph.replay()
        ref = lay.ac_qk_norm_rope_backward(gq, gk, new[:, :, :6], new[:, :, 6:], table=table, w_q=w["w_q"])
        assert torch.equal(got[:, :, :6], ref["q"]) and torch.equal(got[:, :, 6:], ref["k"])
    assert lay.get_status() == 0
