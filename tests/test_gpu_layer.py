"""Per-head norm with rotary positions, its gradients, the append to a paged
cache and the attention over it, against plain forms in 64 bits
(layer_util.py); their refusals, odd views, streams and graphs; and a run of
them together with the clustered attention."""
import math

import numpy as np
import pytest

import layer_util as U

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from clustered_sparse_attention_head_b200 import build
    build()


def _layer(**kw):
    from clustered_sparse_attention_head_b200.layer import AttnLayer, LayerConfig
    return AttnLayer(LayerConfig(**kw))


def _rand(*shape, dtype=torch.bfloat16, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def _near(got, ref, tol, what):
    got = got.double().cpu()
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(((got - ref).abs() / tol.clamp(min=1e-300))[bad].max()))


def _bits(t):
    return t.view(torch.int16 if t.element_size() == 2 else torch.int32)


WAN = dict(rope_dims=(44, 42, 42), rope_max=(3, 5, 7))
ROPES = {
    "no": dict(),
    "grid": WAN,
    "grid64": dict(rope_dims=(16, 24, 24), rope_max=(2, 3, 4)),
    "line": dict(rope_dims=(32,), rope_max=(200,)),
    "half": dict(rope_dims=(48,), rope_max=(200,), rope_layout="half", rope_theta=5e5),
    "half3": dict(rope_dims=(16, 24, 24), rope_max=(2, 3, 4), rope_layout="half"),
    "two": dict(rope_dims=(2, 20), rope_max=(9, 8)),
}


def _inputs(cfg, batch, n, dt, wdt, seed=3, offset=0.0):
    h = cfg.heads + 2 * cfg.kv_heads
    x = _rand(batch, n, h, cfg.d, dtype=dt, seed=seed, scale=2.0) + torch.tensor(offset, dtype=dt).cuda()
    if n > 2:
        x[0, 1] = 0  # a row of zeros
    q, k = x[:, :, :cfg.heads], x[:, :, cfg.heads:cfg.heads + cfg.kv_heads]
    w = [_rand(cfg.d, dtype=wdt, seed=seed + i) for i in range(4)]
    return q, k, w


CASES = [
    # heads, kv heads, d, type, weights' type, norm, rotation, batch, tokens
    (1, 1, 128, "bf16", None, "rms", "grid", 1, 1),
    (5, 5, 128, "bf16", "f32", "rms", "grid", 1, 110),      # 105 tokens on the grid, 5 behind it
    (40, 40, 128, "bf16", None, "layer", "grid", 1, 77),
    (30, 30, 64, "bf16", None, "layer", "grid64", 2, 27),
    (8, 2, 64, "bf16", None, "none", "half", 3, 33),
    (9, 3, 128, "f32", None, "rms", "half", 2, 19),
    (3, 1, 64, "f32", None, "layer", "half3", 1, 26),
    (4, 4, 64, "f32", "bf16", "rms", "line", 1, 200),
    (2, 2, 128, "f32", None, "none", "two", 1, 80),
    (7, 7, 128, "bf16", None, "rms", "no", 1, 65),
    (16, 4, 128, "bf16", None, "rms", "line", 1, 4099),     # 3,899 tokens behind the 200 positions
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_norm_rope(case):
    hq, hk, d, dt, wdt, norm, rope, batch, n = case
    lay = _layer(heads=hq, kv_heads=hk, d=d, dtype=dt, w_dtype=wdt, norm=norm, **ROPES[rope])
    cfg = lay.cfg
    q, k, (wq, wk, bq, bk) = _inputs(cfg, batch, n, lay.dtype, lay.w_dtype)
    table = lay.ac_rope_table() if cfg.rope_dims else None
    qo, ko = lay.ac_qk_norm_rope(q, k, table=table, w_q=wq, w_k=wk, b_q=bq, b_k=bk)
    assert lay.get_status() == 0
    pos = U.grid_pos(n, cfg.rope_max) if cfg.rope_dims else None
    for x, w, b, got in ((q, wq, bq, qo), (k, wk, bk, ko)):
        x, w, b = (t.double().cpu() for t in (x, w, b))
        ref = U.forward(cfg, x, w, b, pos)
        _near(got.transpose(1, 2), ref, U.forward_tol(cfg, x, w, b, ref, lay.dtype), "forward")
    # without weights: 1 and 0
    qo, none = lay.ac_qk_norm_rope(q, None, table=table)
    assert none is None
    x = q.double().cpu()
    ref = U.forward(cfg, x, None, None, pos)
    _near(qo.transpose(1, 2), ref, U.forward_tol(cfg, x, None, None, ref, lay.dtype), "no weights")


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
def test_table_far_positions(scaling):
    """Angles of positions up to 2^20 come from 64 bits: cos and sin are within
    one rounding to fp32 and 2^-52 x angle of the definition's."""
    lay = _layer(heads=1, d=64, rope_dims=(64,), rope_max=(1 << 20,), rope_scaling=scaling, rope_factor=8.0,
                 rope_orig=4096)
    table = lay.ac_rope_table()
    f, _, mag = U.frequencies(lay.cfg)
    rows = torch.tensor([0, 1, 2, 4095, 65537, (1 << 20) - 1])
    got = table.view(1 << 20, 32, 2)[rows.cuda()].double().cpu()
    ang = rows.double()[:, None] * f
    for i, ref in enumerate((ang.cos() * mag, ang.sin() * mag)):
        # pow on the host, its product and the reduction: a few roundings of 2^-53 of the angle
        tol = U.EPS32 * ref.abs() + 8 * 2.0 ** -53 * ang + 2.0 ** -50
        assert ((got[..., i] - ref).abs() <= tol).all(), scaling


def test_explicit_positions():
    """Per-sample and shared positions; a negative coordinate leaves the token
    unrotated; one past the table is clamped and recorded."""
    from clustered_sparse_attention_head_b200 import _abi
    lay = _layer(heads=3, d=64, norm="rms", rope_dims=(16, 24), rope_max=(50, 60), rope_layout="interleaved")
    q, k, (wq, wk, _, _) = _inputs(lay.cfg, 2, 21, lay.dtype, lay.w_dtype)
    table = lay.ac_rope_table()
    g = torch.Generator().manual_seed(5)
    pos = torch.stack([torch.randint(0, 50, (2, 21), generator=g), torch.randint(0, 60, (2, 21), generator=g)], -1)
    pos[0, 3, 0] = -1
    pos[1, 4] = torch.tensor([49, 59])
    for p in (pos, pos[0]):
        qo, _ = lay.ac_qk_norm_rope(q, k, table=table, pos=p.int().cuda(), w_q=wq, w_k=wk)
        assert lay.get_status() == 0
        x, w = q.double().cpu(), wq.double().cpu()
        ref = U.forward(lay.cfg, x, w, None, p)
        _near(qo.transpose(1, 2), ref, U.forward_tol(lay.cfg, x, w, None, ref, lay.dtype), "positions")
    bad = pos.clone()
    bad[1, 7, 1] = 60
    qo, _ = lay.ac_qk_norm_rope(q, k, table=table, pos=bad.int().cuda(), w_q=wq, w_k=wk)
    assert lay.get_status() == _abi.AC_ERR_INVALID_ARG
    assert lay.get_status() == 0
    bad[1, 7, 1] = 59
    same, _ = lay.ac_qk_norm_rope(q, k, table=table, pos=bad.int().cuda(), w_q=wq, w_k=wk)
    assert torch.equal(qo, same)


def test_unrotated_elements_pass_infinities():
    """Elements outside the rotated part, and whole tokens behind the grid, go
    through unchanged with NONE, infinities too."""
    lay = _layer(heads=2, d=64, norm="none", rope_dims=(32,), rope_max=(4,))
    q = _rand(1, 6, 2, 64)
    q[0, 0, 0, 40] = math.inf
    q[0, 5, 1, 3] = -math.inf
    qo, _ = lay.ac_qk_norm_rope(q, None, table=lay.ac_rope_table())
    assert torch.equal(qo[0, :, :, 32:], q[0, :, :, 32:].transpose(0, 1))
    assert torch.equal(qo[0, :, 4:], q[0, 4:].transpose(0, 1))


def test_views_in_place_and_empty():
    lay = _layer(heads=6, kv_heads=2, d=128, norm="rms", **WAN)
    q, k, (wq, wk, _, _) = _inputs(lay.cfg, 2, 37, lay.dtype, lay.w_dtype)
    table = lay.ac_rope_table()
    want = lay.ac_qk_norm_rope(q, k, table=table, w_q=wq, w_k=wk)
    # head-major inputs, and outputs inside larger buffers
    qh, kh = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k))
    big = torch.full((2, 9, 41, 128), 7.0, dtype=lay.dtype, device="cuda")
    got = lay.ac_qk_norm_rope(qh, kh, table=table, w_q=wq, w_k=wk, q_out=big[:, :6, 2:39], k_out=big[:, 7:, 2:39])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (big[:, 6] == 7).all() and (big[:, :, :2] == 7).all() and (big[:, :, 39:] == 7).all()
    # in place in the packed projection
    x = torch.cat([q, k], 2)
    a, b = x[:, :, :6], x[:, :, 6:]
    lay.ac_qk_norm_rope(a, b, table=table, w_q=wq, w_k=wk, q_out=a.transpose(1, 2), k_out=b.transpose(1, 2))
    assert torch.equal(a.transpose(1, 2), want[0]) and torch.equal(b.transpose(1, 2), want[1])
    # a broadcast input (token stride 0)
    one = q[:, :1].expand(2, 37, 6, 128)
    got, _ = lay.ac_qk_norm_rope(one, None, table=table, w_q=wq)
    ref, _ = lay.ac_qk_norm_rope(one.contiguous(), None, table=table, w_q=wq)
    assert torch.equal(got, ref)
    # no tokens
    e, _ = lay.ac_qk_norm_rope(q[:, :0], k[:, :0], table=table)
    assert e.shape == (2, 6, 0, 128)
    assert lay.get_status() == 0


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_backward(case):
    hq, hk, d, dt, wdt, norm, rope, batch, n = case
    lay = _layer(heads=hq, kv_heads=hk, d=d, dtype=dt, w_dtype=wdt, norm=norm, **ROPES[rope])
    cfg = lay.cfg
    q, k, (wq, wk, bq, bk) = _inputs(cfg, batch, n, lay.dtype, lay.w_dtype)
    if n > 2 and norm != "none":
        q[0, 1], k[0, 1] = 0.5, 0.5  # 1 / sqrt(eps) of a zero row scales any rounding by 1,000
        q[0, 1, :, ::2] = -0.25
        k[0, 1, :, ::2] = -0.25
    gq, gk = _rand(batch, hq, n, d, dtype=lay.dtype, seed=8), _rand(batch, hk, n, d, dtype=lay.dtype, seed=9)
    table = lay.ac_rope_table() if cfg.rope_dims else None
    args = dict(table=table, w_q=wq, w_k=wk, b_q=bq, b_k=bk) if norm != "none" else dict(table=table)
    res = lay.ac_qk_norm_rope_backward(gq, gk, q, k, **args)
    assert lay.get_status() == 0
    pos = U.grid_pos(n, cfg.rope_max) if cfg.rope_dims else None
    for name, g, x, w in (("q", gq, q, wq), ("k", gk, k, wk)):
        g, x, w = g.double().cpu().transpose(1, 2), x.double().cpu(), w.double().cpu()
        dx, dw, db = U.backward(cfg, g, x, w, pos)
        if norm == "none":
            big = g.abs().amax(-1, keepdim=True)
            _near(res[name], dx, U.half_step(lay.dtype) * dx.abs() + 8 * U.EPS32 * big, "dx")
            continue
        y, r = U.normed(cfg, x)
        xin = x.abs().amax(-1, keepdim=True) * r
        e = 2 * g.abs().amax(-1, keepdim=True) * w.abs().max()
        # g' and n are within 32 roundings of their rows' largest values (forward_tol);
        # the two means add 10 roundings of e and of e n^2 each
        tol = U.half_step(lay.dtype) * dx.abs() + 128 * U.EPS32 * r * e * (1 + xin * y.abs().amax(-1, keepdim=True))
        _near(res[name], dx, tol, "dx")
        gt = U.turn(cfg, g, pos, back=True).abs()
        rows = gt.shape[0] * gt.shape[1] * gt.shape[2]
        # sequential fp32 sums of at most `rows` terms, each within 64 roundings of max|g'| max|n|
        most = (2 * g.abs().amax(-1, keepdim=True) * xin).sum((0, 1, 2))
        st = U.half_step(lay.w_dtype)
        _near(res["w_" + name], dw, st * dw.abs() + (min(rows, 4096) + 64) * U.EPS32 * most, "dw")
        most = (2 * g.abs().amax(-1, keepdim=True)).sum((0, 1, 2))
        _near(res["b_" + name], db, st * db.abs() + (min(rows, 4096) + 64) * U.EPS32 * most, "db")


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_backward_against_differences(norm):
    """Directional derivatives of sum(g y) by central differences of the 64-bit
    forward form, for the inputs, weights and biases."""
    lay = _layer(heads=4, kv_heads=2, d=64, dtype="f32", norm=norm, **ROPES["half3"])
    cfg = lay.cfg
    q, k, (wq, wk, bq, bk) = _inputs(cfg, 1, 30, torch.float32, torch.float32)
    q[0, 1], k[0, 1] = _rand(4, 64, dtype=torch.float32, seed=1), _rand(2, 64, dtype=torch.float32, seed=2)
    gq, gk = _rand(1, 4, 30, 64, dtype=torch.float32, seed=8), _rand(1, 2, 30, 64, dtype=torch.float32, seed=9)
    res = lay.ac_qk_norm_rope_backward(gq, gk, q, k, table=lay.ac_rope_table(), w_q=wq, w_k=wk, b_q=bq, b_k=bk)
    pos = U.grid_pos(30, cfg.rope_max)
    for name, g, x, w, b in (("q", gq, q, wq, bq), ("k", gk, k, wk, bk)):
        g, x, w, b = (t.double().cpu() for t in (g.transpose(1, 2), x, w, b))
        gen = torch.Generator().manual_seed(4)
        vx, vw, vb = (torch.randn(t.shape, generator=gen, dtype=torch.float64) for t in (x, w, b))
        h = 1e-5
        f = [(g * U.forward(cfg, x + s * h * vx, w + s * h * vw, b + s * h * vb, pos)).sum() for s in (1, -1)]
        want = (f[0] - f[1]) / (2 * h)
        parts = [(res[n].double().cpu() * v) for n, v in ((name, vx), ("w_" + name, vw), ("b_" + name, vb))]
        got = sum(p.sum() for p in parts)
        size = sum(p.abs().sum() for p in parts)
        # fp32 gradients: 256 roundings of every term; differences: h^2 curvature, far below
        assert abs(got - want) <= 256 * U.EPS32 * size + 1e-7 * size, (got, want)


def test_backward_views():
    lay = _layer(heads=6, kv_heads=3, d=64, norm="layer", **ROPES["grid64"])
    q, k, (wq, wk, bq, bk) = _inputs(lay.cfg, 2, 29, lay.dtype, lay.w_dtype)
    gq, gk = _rand(2, 6, 29, 64, seed=8), _rand(2, 3, 29, 64, seed=9)
    table = lay.ac_rope_table()
    args = dict(table=table, w_q=wq, w_k=wk)
    want = lay.ac_qk_norm_rope_backward(gq, gk, q, k, b_q=bq, b_k=bk, **args)
    again = lay.ac_qk_norm_rope_backward(gq, gk, q, k, b_q=bq, b_k=bk, **args)
    for name in want:  # the same bits every time
        assert torch.equal(_bits(want[name]), _bits(again[name])), name
    # a packed gradient, and a gradient written over its own upstream
    packed = torch.full((2, 29, 12, 64), 3.0, dtype=lay.dtype, device="cuda")
    got = lay.ac_qk_norm_rope_backward(gq, gk, q, k, dq=packed[:, :, :6], dk=packed[:, :, 6:9], **args)
    assert torch.equal(packed[:, :, :6], want["q"]) and torch.equal(packed[:, :, 6:9], want["k"])
    assert (packed[:, :, 9:] == 3).all() and got["b_q"] is None
    g2 = gq.clone()
    got = lay.ac_qk_norm_rope_backward(g2, None, q, None, table=table, w_q=wq, dq=g2.transpose(1, 2))
    assert torch.equal(g2.transpose(1, 2), want["q"]) and got["k"] is None
    # one gradient for every token (stride 0)
    one = gq[:, :, :1].expand(2, 6, 29, 64)
    a = lay.ac_qk_norm_rope_backward(one, None, q, None, table=table, w_q=wq)
    b = lay.ac_qk_norm_rope_backward(one.contiguous(), None, q, None, table=table, w_q=wq)
    assert torch.equal(a["q"], b["q"]) and torch.equal(a["w_q"], b["w_q"])
    # no tokens: gradients of zero
    z = lay.ac_qk_norm_rope_backward(gq[:, :, :0], gk[:, :, :0], q[:, :0], k[:, :0], b_q=bq, b_k=bk, **args)
    assert all((z[n] == 0).all() for n in ("w_q", "b_q", "w_k", "b_k"))
    assert lay.get_status() == 0


# ------------------------------------------------------------------ the cache
def _cache(lay, kv, spare=2, seed=0, fill=None, table_pages=None):
    """Pools and a shuffled block table for sequences of lengths kv."""
    page = lay.cfg.page_size
    need = [-(-n // page) for n in kv]
    total = sum(need) + spare
    kp = _rand(total, lay.kv_heads, page, lay.d, dtype=lay.dtype, seed=seed + 1)
    vp = _rand(total, lay.kv_heads, page, lay.d, dtype=lay.dtype, seed=seed + 2)
    order = np.random.default_rng(seed).permutation(total)
    table = np.full((len(kv), table_pages or max(max(need), 1)), 10 ** 9, np.int32)  # never-read entries are wild
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return kp, vp, torch.from_numpy(table).cuda()


def _starts(new):
    return torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32).cuda()


@pytest.mark.parametrize("dt, d, hq, hk, norm, rope, page", [
    ("bf16", 128, 4, 4, "rms", "grid", 16),
    ("bf16", 64, 8, 2, "layer", "half", 32),
    ("f32", 128, 3, 3, "none", "line", 64),
    ("bf16", 128, 5, 5, "rms", "no", 128),
    ("f32", 64, 30, 30, "rms", "grid64", 16),
])
def test_append(dt, d, hq, hk, norm, rope, page):
    lay = _layer(heads=hq, kv_heads=hk, d=d, dtype=dt, norm=norm, page_size=page, **ROPES[rope])
    cfg = lay.cfg
    new, kv = [1, 0, 17, 40, 3], [1, 33, 17, 131, 64]
    kp, vp, bt = _cache(lay, kv)
    extra = 3  # rows behind the last sequence
    T = sum(new)
    x = _rand(T + extra, hq + 2 * hk, d, dtype=lay.dtype, seed=5)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    w = [_rand(d, dtype=lay.dtype, seed=20 + i) for i in range(4)]
    table = lay.ac_rope_table() if cfg.rope_dims else None
    kp0, vp0 = kp.clone(), vp.clone()
    qo = torch.full((T + extra, hq, d), 9.0, dtype=lay.dtype, device="cuda")
    kw = dict(w_q=w[0], w_k=w[1], b_q=w[2], b_k=w[3])
    got = lay.ac_cache_append(k, v, kp, vp, bt, _starts(new), torch.tensor(kv, dtype=torch.int32).cuda(), q=q,
                              table=table, q_out=qo, **kw)
    assert got is qo and lay.get_status() == 0
    assert (qo[T:] == 9).all()
    place = torch.cat([torch.arange(n - m, n) for m, n in zip(new, kv)])
    pos = U.grid_pos(max(kv), cfg.rope_max)[place] if cfg.rope_dims else None
    for xx, ww, bb, name in ((q[:T], w[0], w[2], "q"), (k[:T], w[1], w[3], "k")):
        xx, ww, bb = xx.double().cpu()[None], ww.double().cpu(), bb.double().cpu()
        ref = U.forward(cfg, xx, ww, bb, pos)
        tol = U.forward_tol(cfg, xx, ww, bb, ref, lay.dtype)[0]
        seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
        pages = bt.cpu()[seq, place // page].long()
        mine = qo[:T] if name == "q" else kp.cpu()[pages, :, place % page]
        _near(mine, ref[0], tol, name)
    assert torch.equal(vp.cpu()[pages, :, place % page], v[:T].cpu())
    # everything else is as it was
    for pool, old in ((kp, kp0), (vp, vp0)):
        keep = torch.ones(pool.shape[0], page, dtype=torch.bool)
        keep[pages, place % page] = False
        a, b = pool.cpu().transpose(1, 2)[keep], old.cpu().transpose(1, 2)[keep]
        assert torch.equal(a, b)
    # keys and values alone, positions given
    kp2, vp2 = kp0.clone(), vp0.clone()
    p = pos.int().cuda() if pos is not None else None
    if p is not None:
        p = torch.cat([p, torch.zeros(extra, p.shape[1], dtype=torch.int32, device="cuda")])
    assert lay.ac_cache_append(k, v, kp2, vp2, bt, _starts(new), torch.tensor(kv, dtype=torch.int32).cuda(),
                               table=table, pos=p, w_k=w[1], b_k=w[3]) is None
    assert torch.equal(kp2, kp) and torch.equal(vp2, vp)


def test_append_bad_pages_and_lengths():
    """A wild page id, and a token outside its block table, are skipped and
    recorded; the other tokens arrive and the queries are all written."""
    from clustered_sparse_attention_head_b200 import _abi
    lay = _layer(heads=2, d=64, norm="none", page_size=16)
    kp, vp, bt = _cache(lay, [40, 40, 40])
    k, v, q = (_rand(12, 2, 64, seed=i) for i in (1, 2, 3))
    start = _starts([4, 4, 4])
    for kv, wild in (([40, 40, 40], -1), ([40, 40, 40], kp.shape[0]), ([40, 49, 40], None), ([40, 2, 40], None)):
        table = bt.clone()
        if wild is not None:
            table[1, 2] = wild
        kp0, vp0 = kp.clone(), vp.clone()
        qo = lay.ac_cache_append(k, v, kp0, vp0, table, start, torch.tensor(kv, dtype=torch.int32).cuda(), q=q)
        assert lay.get_status() == _abi.AC_ERR_INVALID_ARG
        assert torch.equal(qo, q)
        b = bt.cpu().long()
        for s in (0, 2):
            assert torch.equal(kp0[b[s, 2], :, 4:8], k[4 * s:4 * s + 4].transpose(0, 1))
            assert torch.equal(vp0[b[s, 2], :, 4:8], v[4 * s:4 * s + 4].transpose(0, 1))
        changed = (kp0 != kp).any(-1).any(1).sum()  # cache rows that changed
        assert int(changed) == 8 + {49: 3, 2: 2}.get(kv[1], 0)


ATTN = [
    # heads, kv heads, d, page, block, window, new, kv
    (1, 1, 64, 16, 0, 0, [1], [1]),
    (8, 8, 128, 16, 1, 0, [1, 1, 1], [1, 130, 777]),
    (32, 8, 128, 16, 1, 0, [1, 1], [513, 64]),
    (6, 2, 64, 32, 1, 0, [5, 0, 33], [5, 40, 300]),
    (5, 1, 128, 64, 7, 0, [50, 3], [190, 3]),
    (10, 2, 64, 128, 0, 0, [129], [257]),
    (3, 3, 128, 16, 1, 20, [70, 1], [200, 90]),
    (4, 4, 64, 16, 0, 5, [40], [40]),
    (2, 2, 128, 32, 64, 100, [128, 64], [256, 320]),
    (2, 2, 128, 16, 1, 0, [260], [700]),
    (4, 1, 64, 1024, 1, 0, [100], [1100]),
    (7, 1, 128, 16, 1, 0, [20, 19], [20, 400]),
    (12, 12, 64, 16, 300, 0, [300], [900]),
    (2, 1, 128, 16, 1, 0, [3, 5, 2], [0, 2, 2]),   # fewer keys than new tokens: some see none
    (40, 40, 128, 64, 8, 0, [8], [72]),
    (1, 1, 128, 16, 1, 1, [9], [30]),              # every token sees itself alone
    (16, 16, 64, 16, 1, 0, [1] * 9, [3, 0, 16, 17, 31, 128, 129, 255, 1000]),
    (32, 8, 128, 32, 1, 0, [4, 1, 3, 0], [4, 900, 2500, 7]),   # 16 rows a key head
    (16, 2, 64, 64, 0, 0, [2, 1], [5000, 33]),
    (3, 1, 128, 16, 1, 37, [5, 4], [700, 40]),                 # 15 rows, windows that begin inside a block
    (16, 1, 64, 16, 5, 0, [1], [4099]),
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "-".join(str(x) for x in c[:6]) + f"-{sum(c[6])}-{sum(c[7])}")
def test_attn(case):
    hq, hk, d, page, block, window, new, kv = case
    lay = _layer(heads=hq, kv_heads=hk, d=d, page_size=page, causal_block=block, window=window)
    kp, vp, bt = _cache(lay, kv, table_pages=max(1, -(-max(kv) // page)) + 2)
    # rows at or beyond a sequence's length hold anything
    kpn, vpn = kp.clone(), vp.clone()
    used = torch.zeros(kp.shape[0], page, dtype=torch.bool)
    for s, n in enumerate(kv):
        j = torch.arange(n)
        used[bt.cpu()[s][j // page].long(), j % page] = True
    for pool, val in ((kpn, math.nan), (vpn, math.inf)):
        pool.transpose(1, 2)[~used.cuda()] = val
    T = sum(new)
    x = _rand(T + 2, 3 * hq, d, seed=7, scale=1.5)
    q = x[:, hq:2 * hq]  # a view with foreign rows on both sides
    q[T:] = math.nan
    out = torch.full((hq, T + 2, d), 5.0, dtype=lay.dtype, device="cuda").transpose(0, 1)
    got, lse = lay.ac_cache_attn(q, kpn, vpn, bt, _starts(new), torch.tensor(kv, dtype=torch.int32).cuda(),
                                 max_q=max(new), max_kv=max(kv), out=out, lse=True)
    assert got is out and lay.get_status() == 0
    assert (got[T:] == 5).all()
    ref, rl, absv, big, _ = U.attend(lay.cfg, q[:T].double().cpu(), kp.double().cpu(), vp.double().cpu(), bt.cpu(),
                                     _starts(new).cpu(), kv)
    _near(got[:T], ref, U.attend_tol(ref, absv, big), "out")
    lse = lse[:T].double().cpu()
    none = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), none) and (lse[none] < 0).all()
    # the sum's 1.1e-4 by weight, the score's error, log2's and the product's roundings
    tol = 1.2e-4 + 136 * U.EPS32 * big + 8 * U.EPS32 * rl.abs()
    assert ((lse - rl).abs() <= tol)[~none].all()
    # the shapes' own bounds, no lse: the same within the tolerance of both
    got2 = lay.ac_cache_attn(q[:T], kpn, vpn, bt, _starts(new), torch.tensor(kv, dtype=torch.int32).cuda())
    assert lay.get_status() == 0
    _near(got2, ref, U.attend_tol(ref, absv, big), "default bounds")


@pytest.mark.parametrize("d, heads, kv_heads, new, kv, block", [
    (64, 40, 40, [300, 257], [2100, 2300], 1),      # more units than SMs, the last ones cut in pieces
    (128, 20, 20, [513, 1], [1500, 700], 50),
    (128, 2, 2, [1], [21000], 1),                   # a cluster of 16 CTAs
    (64, 1, 1, [2], [60000], 0),                    # too few units for the GPU: tiles cut along the keys
])
def test_attn_many_units(d, heads, kv_heads, new, kv, block):
    """Call after call the same bits, whichever CTA takes which unit, and right."""
    lay = _layer(heads=heads, kv_heads=kv_heads, d=d, page_size=64, causal_block=block)
    kp, vp, bt = _cache(lay, kv)
    q = _rand(sum(new), heads, d, seed=7)
    kvt = torch.tensor(kv, dtype=torch.int32).cuda()
    args = (q, kp, vp, bt, _starts(new), kvt)
    got = [lay.ac_cache_attn(*args, max_q=max(new), max_kv=max(kv)) for _ in range(3)]
    assert lay.get_status() == 0
    assert torch.equal(_bits(got[0]), _bits(got[1])) and torch.equal(_bits(got[0]), _bits(got[2]))
    ref, _, absv, big, _ = U.attend(lay.cfg, q.double().cpu(), kp.double().cpu(), vp.double().cpu(), bt.cpu(),
                                    _starts(new).cpu(), kv)
    _near(got[0], ref, U.attend_tol(ref, absv, big), "out")


def test_attn_large_scores_and_scale():
    """Scores in the hundreds whose maximum moves late, and a scale of its own."""
    lay = _layer(heads=2, d=64, page_size=16, causal_block=1, scale=0.37)
    kp, vp, bt = _cache(lay, [400])
    grow = torch.ones(kp.shape[0], device="cuda")
    grow[bt[0].long()] = torch.linspace(0.1, 12, bt.shape[1], device="cuda")  # later pages hold larger keys
    kp *= grow[:, None, None, None].to(kp.dtype)
    q = _rand(150, 2, 64, seed=3, scale=4.0)
    kv = torch.tensor([400], dtype=torch.int32).cuda()
    got = lay.ac_cache_attn(q, kp, vp, bt, _starts([150]), kv)
    ref, _, absv, big, _ = U.attend(lay.cfg, q.double().cpu(), kp.double().cpu(), vp.double().cpu(), bt.cpu(),
                                    _starts([150]).cpu(), [400])
    _near(got, ref, U.attend_tol(ref, absv, big), "large scores")


def test_attn_bounds_and_bad_pages():
    from clustered_sparse_attention_head_b200 import _abi
    lay = _layer(heads=4, kv_heads=2, d=64, page_size=16, causal_block=1)
    new, kv = [6, 40], [90, 200]
    kp, vp, bt = _cache(lay, kv)
    q = _rand(46, 4, 64, seed=7)
    kvt = torch.tensor(kv, dtype=torch.int32).cuda()
    dbl = (kp.double().cpu(), vp.double().cpu())

    def check(got, seen_only, **kw):
        table = kw.pop("table", bt).cpu()
        ref, _, absv, big, seen = U.attend(lay.cfg, q.double().cpu(), *dbl, table, _starts(new).cpu(), kv, **kw)
        _near(got[seen.cuda()] if seen_only else got, ref[seen] if seen_only else ref,
              U.attend_tol(ref, absv, big)[seen] if seen_only else U.attend_tol(ref, absv, big), kw)

    # the bounds cut longer sequences, and say so
    out = torch.full((46, 4, 64), 2.0, dtype=lay.dtype, device="cuda")
    lay.ac_cache_attn(q, kp, vp, bt, _starts(new), kvt, max_q=10, out=out)
    assert lay.get_status() == _abi.AC_ERR_INVALID_ARG
    check(out, True, max_q=10)
    assert (out[16:] == 2).all()
    got = lay.ac_cache_attn(q, kp, vp, bt, _starts(new), kvt, max_kv=150)
    assert lay.get_status() == _abi.AC_ERR_INVALID_ARG
    check(got, False, max_kv=150)
    # wild page ids read the nearest page
    for wild in (-5, 10 ** 9):
        table = bt.clone()
        table[1, 3] = wild
        got = lay.ac_cache_attn(q, kp, vp, table, _starts(new), kvt)
        assert lay.get_status() == _abi.AC_ERR_INVALID_ARG
        check(got, False, table=table)
    # a length below zero is none
    got = lay.ac_cache_attn(q, kp, vp, bt, _starts(new), torch.tensor([-4, 200], dtype=torch.int32).cuda())
    assert lay.get_status() == _abi.AC_ERR_INVALID_ARG
    assert (got[:6] == 0).all()
    assert lay.get_status() == 0
    # no keys at all, and no tokens
    got, lse = lay.ac_cache_attn(q, kp, vp, bt, _starts(new), torch.zeros_like(kvt), lse=True)
    assert (got == 0).all() and (lse == -math.inf).all() and lay.get_status() == 0
    got, lse = lay.ac_cache_attn(q, kp[:0], vp[:0], bt[:, :0], _starts(new), torch.zeros_like(kvt), lse=True)
    assert (got == 0).all() and (lse == -math.inf).all() and lay.get_status() == 0
    assert lay.ac_cache_attn(q[:0], kp, vp, bt, _starts([0, 0]), kvt).shape == (0, 4, 64)


def test_attn_malformed_starts():
    """Starts that fall, overlap or leave the tensor: no access outside the
    buffers; rows of well-formed sequences come out right."""
    lay = _layer(heads=2, d=64, page_size=16, causal_block=1)
    kp, vp, bt = _cache(lay, [40, 40, 40])
    q, kv = _rand(30, 2, 64, seed=7), torch.tensor([40, 40, 40], dtype=torch.int32).cuda()
    for starts in ([-3, 10, 20, 30], [0, 10, 20, 90], [0, 20, 10, 30], [5, 5, 5, 5], [40, 50, 60, 70]):
        st = torch.tensor(starts, dtype=torch.int32).cuda()
        got = lay.ac_cache_attn(q, kp, vp, bt, st, kv)
        lay.get_status()
        a, b = starts[1], starts[2]
        if starts[0] <= 0 <= a <= b <= 30 and starts[3] >= b:
            ref, _, absv, big, _ = U.attend(lay.cfg, q.double().cpu(), kp.double().cpu(), vp.double().cpu(), bt.cpu(),
                                            [0, a, b, b], [40, 40, 0])
            _near(got[a:b], ref[a:b], U.attend_tol(ref, absv, big)[a:b], starts)
        k = _rand(30, 2, 64, seed=8)
        none = _layer(heads=2, d=64, page_size=16, norm="none")
        none.ac_cache_append(k, k, kp.clone(), vp.clone(), bt, st, kv)
        none.get_status()
    torch.cuda.synchronize()


def test_cache_offsets_past_32_bits():
    """Pools of more than 2^32 bytes (and 2^31 elements): pages at their far end."""
    lay = _layer(heads=8, kv_heads=8, d=128, page_size=64, causal_block=1, norm="none")
    pages = (1 << 31) // (8 * 64 * 128) + 40
    kp = torch.zeros(pages, 8, 64, 128, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    bt = torch.tensor([[pages - 1, 3, pages - 30]], dtype=torch.int32).cuda()
    k, v, q = (_rand(150, 8, 128, seed=i) for i in (1, 2, 3))
    kv = torch.tensor([150], dtype=torch.int32).cuda()
    lay.ac_cache_append(k, v, kp, vp, bt, _starts([150]), kv)
    got = lay.ac_cache_attn(q, kp, vp, bt, _starts([150]), kv)
    assert lay.get_status() == 0
    rows = bt[0].long()
    small = torch.tensor([[0, 1, 2]])
    ref, _, absv, big, _ = U.attend(lay.cfg, q.double().cpu(), kp[rows].double().cpu(), vp[rows].double().cpu(), small,
                                    [0, 150], [150])
    _near(got, ref, U.attend_tol(ref, absv, big), "far pages")
    del kp, vp
    torch.cuda.empty_cache()


def test_strides_past_32_bits():
    """Heads 2^30 elements apart: the third one's rows lie beyond 2^31 elements."""
    buf = torch.zeros(2 ** 31 + 2 ** 20, dtype=torch.bfloat16, device="cuda")
    far = 2 ** 30
    lay = _layer(heads=3, d=128, norm="rms", page_size=16, causal_block=1, rope_dims=(128,), rope_max=(99,))
    table = lay.ac_rope_table()
    x = _rand(1, 20, 3, 128, seed=1)
    want, _ = lay.ac_qk_norm_rope(x, None, table=table)
    out = torch.as_strided(buf, (1, 3, 20, 128), (8, far, 128, 1))
    lay.ac_qk_norm_rope(x, None, table=table, q_out=out)
    assert torch.equal(out, want)
    back = lay.ac_qk_norm_rope_backward(want, None, x, None, table=table)["q"]
    assert torch.equal(lay.ac_qk_norm_rope_backward(out, None, x, None, table=table)["q"], back)
    kp, vp, bt = _cache(lay, [40])
    kv = torch.tensor([40], dtype=torch.int32).cuda()
    q, near = out[0].transpose(0, 1), want[0].transpose(0, 1).contiguous()
    buf2 = torch.zeros_like(buf)  # outputs whose span holds their input's are refused
    for new in (3, 20):  # the kernel for few rows, and tiles
        ref = lay.ac_cache_attn(near[:new], kp, vp, bt, _starts([new]), kv)
        o = torch.as_strided(buf2, (new, 3, 128), (128, far, 1))
        lay.ac_cache_attn(q[:new], kp, vp, bt, _starts([new]), kv, out=o)
        assert torch.equal(o, ref)
    lay.ac_cache_append(q, q, kp, vp, bt, _starts([20]), kv, table=table)
    kp2, vp2 = kp.clone(), vp.clone()
    lay.ac_cache_append(near, near, kp2, vp2, bt, _starts([20]), kv, table=table)
    assert torch.equal(kp, kp2) and torch.equal(vp, vp2) and lay.get_status() == 0
    del buf, buf2, out, q, o
    torch.cuda.empty_cache()


# ------------------------------------------------------- streams, graphs, runs
def test_other_stream():
    lay = _layer(heads=8, d=64, page_size=16, causal_block=1, **ROPES["grid64"])
    kp, vp, bt = _cache(lay, [24])
    x = _rand(1, 24, 24, 64, seed=2)
    table = lay.ac_rope_table()
    kv = torch.tensor([24], dtype=torch.int32).cuda()
    st = _starts([24])

    def step(stream):
        qo = lay.ac_cache_append(x[0, :, 8:16], x[0, :, 16:], kp, vp, bt, st, kv, q=x[0, :, :8], table=table,
                                 stream=stream)
        out = lay.ac_cache_attn(qo, kp, vp, bt, st, kv, stream=stream)
        q2, k2 = lay.ac_qk_norm_rope(x[:, :, :8], x[:, :, 8:16], table=table, stream=stream)
        g = lay.ac_qk_norm_rope_backward(q2, k2, x[:, :, :8], x[:, :, 8:16], table=table, stream=stream)
        return out, q2, k2, g["q"], g["k"]

    want = step(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert lay.get_status(side) == 0


def test_graph_replay_with_new_lengths():
    """Append and attention captured once; every replay reads the lengths, the
    starts and the block table of that moment."""
    lay = _layer(heads=4, kv_heads=2, d=128, page_size=16, causal_block=1, **dict(rope_dims=(128,), rope_max=(500,)))
    kp, vp, bt = _cache(lay, [300, 300, 300], spare=0)
    kp0, vp0 = kp.clone(), vp.clone()
    table = lay.ac_rope_table()
    x = _rand(3, 8, 128, seed=2)
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    kv = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.empty(3, 4, 128, dtype=torch.bfloat16, device="cuda")
    qo = torch.empty_like(out)

    def step():
        lay.ac_cache_append(x[:, 4:6], x[:, 6:], kp, vp, bt, st, kv, q=x[:, :4], table=table, q_out=qo)
        lay.ac_cache_attn(qo, kp, vp, bt, st, kv, max_q=3, max_kv=300, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for starts, lens in (([0, 1, 2, 3], [1, 130, 299]), ([0, 1, 2, 3], [2, 131, 300]), ([0, 3, 3, 3], [200, 7, 9]),
                         ([0, 0, 1, 1], [5, 40, 6])):
        st.copy_(torch.tensor(starts, dtype=torch.int32))
        kv.copy_(torch.tensor(lens, dtype=torch.int32))
        x.copy_(_rand(3, 8, 128, seed=sum(lens)))
        kp.copy_(kp0)
        vp.copy_(vp0)
        out.fill_(4.0)
        graph.replay()
        a = out.clone()
        kp.copy_(kp0)
        vp.copy_(vp0)
        out.fill_(4.0)
        step()
        assert torch.equal(a, out)
        assert lay.get_status() == 0
        ref, _, absv, big, seen = U.attend(lay.cfg, qo.double().cpu(), kp.double().cpu(), vp.double().cpu(), bt.cpu(),
                                           starts, lens)
        _near(a[seen.cuda()], ref[seen], U.attend_tol(ref, absv, big)[seen], lens)
        assert (a[~seen.cuda()] == 4).all()


def test_graph_of_every_call():
    """Forward, gradients (two kernels), append and split attention (two kernels)
    in one graph, replayed on new inputs."""
    lay = _layer(heads=4, d=64, norm="layer", page_size=16, causal_block=1, rope_dims=(64,), rope_max=(4000,))
    n = 600
    kp, vp, bt = _cache(lay, [2900])
    table = lay.ac_rope_table()
    x = _rand(1, n, 12, 64, seed=2)
    w, b = _rand(64, seed=3), _rand(64, seed=4)
    st, kv = _starts([n]), torch.tensor([2900], dtype=torch.int32).cuda()

    def step():
        q, k = lay.ac_qk_norm_rope(x[:, :, :4], x[:, :, 4:8], table=table, w_q=w, w_k=w, b_q=b, b_k=b)
        g = lay.ac_qk_norm_rope_backward(k, q, x[:, :, :4], x[:, :, 4:8], table=table, w_q=w, w_k=w, b_q=b, b_k=b)
        qo = lay.ac_cache_append(x[0, :, 4:8], x[0, :, 8:], kp, vp, bt, st, kv, q=x[0, :, :4], table=table, w_q=w,
                                 w_k=w)
        return [q, k, *g.values(), qo, *lay.ac_cache_attn(qo, kp, vp, bt, st, kv, lse=True)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (11, 12):
        x.copy_(_rand(1, n, 12, 64, seed=seed))
        graph.replay()
        got = [t.clone() for t in outs]
        want = step()
        assert all(torch.equal(_bits(a), _bits(b)) for a, b in zip(got, want))
    assert lay.get_status() == 0


def test_calls_on_two_streams_at_once():
    """Calls without a workspace may overlap, on one layer and its status word."""
    lay = _layer(heads=16, d=128, norm="rms", rope_dims=(128,), rope_max=(9000,))
    table = lay.ac_rope_table()
    xs = [_rand(1, 8000, 32, 128, seed=i) for i in (1, 2)]
    want = [lay.ac_qk_norm_rope(x[:, :, :16], x[:, :, 16:], table=table) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(5):
        for i, (x, st) in enumerate(zip(xs, streams)):
            with torch.cuda.stream(st):
                got[i].append(lay.ac_qk_norm_rope(x[:, :, :16], x[:, :, 16:], table=table))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(a, b) for pair in got[i] for a, b in zip(pair, want[i]))
    assert lay.get_status() == 0


def test_block_run_together():
    """A clip made three frames at a time: append and attention per chunk equal
    the 64-bit attention, causal by frames, of the whole clip's normed and
    rotated queries and keys; and with every frame visible it is what the
    clustered attention gives when it keeps every cluster."""
    from clustered_sparse_attention_head_b200.api import AdaCluster, Config
    frames, rows, cols, heads, d = 9, 6, 10, 3, 128
    n, fr = frames * rows * cols, rows * cols
    cfg = dict(heads=heads, d=d, norm="rms", rope_dims=(44, 42, 42), rope_max=(frames, rows, cols), page_size=32)
    lay = _layer(causal_block=fr, **cfg)
    table = lay.ac_rope_table()
    x = _rand(n, 3 * heads, d, seed=1)
    wq, wk = _rand(d, seed=2) * 0.3 + 1, _rand(d, seed=3) * 0.3 + 1
    kp, vp, bt = _cache(lay, [n])
    outs = []
    for a in range(0, n, 3 * fr):
        b = a + 3 * fr
        c = x[a:b]
        kv = torch.tensor([b], dtype=torch.int32).cuda()
        st = _starts([b - a])
        qo = lay.ac_cache_append(c[:, heads:2 * heads], c[:, 2 * heads:], kp, vp, bt, st, kv, q=c[:, :heads],
                                 table=table, w_q=wq, w_k=wk)
        outs.append(lay.ac_cache_attn(qo, kp, vp, bt, st, kv))
    assert lay.get_status() == 0
    got = torch.cat(outs).double().cpu()
    qo, ko = lay.ac_qk_norm_rope(x[None, :, :heads], x[None, :, heads:2 * heads], table=table, w_q=wq, w_k=wk)
    q, k = qo[0].double().cpu(), ko[0].double().cpu()      # [heads, n, d]
    v = x[:, 2 * heads:].double().cpu().transpose(0, 1)
    s = q @ k.transpose(1, 2) / math.sqrt(d)
    big = (q.abs() @ k.abs().transpose(1, 2)).amax(-1) / math.sqrt(d)
    f = torch.arange(n) // fr
    w = torch.softmax(s.masked_fill(f[None, :, None] < f[None, None, :], -math.inf), -1)
    ref, absv = w @ v, w @ v.abs()
    _near(got.transpose(0, 1), ref, U.attend_tol(ref, absv, big), "frames")
    # every frame visible, against the clustered attention with every cluster kept
    full = _layer(causal_block=0, **cfg)
    out = full.ac_cache_attn(qo[0].transpose(0, 1), kp, vp, bt, _starts([n]), torch.tensor([n], dtype=torch.int32).cuda())
    ac = AdaCluster(Config(heads=heads, n=n, d=d, kq=6, kk=12, top_p=1.0))
    dense = ac.ac_forward(qo[0], ko[0], x[:, 2 * heads:].transpose(0, 1).contiguous())
    assert ac.get_status() == 0 and full.get_status() == 0
    w = torch.softmax(s, -1)
    ref, absv = w @ v, w @ v.abs()
    tol = U.attend_tol(ref, absv, big)
    _near(out.transpose(0, 1), ref, tol, "all frames")
    _near(dense, ref, tol, "clustered")
    ac.close()


# ------------------------------------------------------------------ refusals
def test_python_refusals():
    from clustered_sparse_attention_head_b200._abi import AcError
    lay = _layer(heads=4, kv_heads=2, d=64, page_size=16, norm="rms", **ROPES["grid64"])
    q, k = _rand(1, 5, 4, 64), _rand(1, 5, 2, 64)
    table = lay.ac_rope_table()
    w = _rand(64)
    ok = dict(table=table, w_q=w, w_k=w)
    lay.ac_qk_norm_rope(q, k, **ok)
    bad = [
        (ValueError, dict(q=q.float())), (ValueError, dict(q=q.cpu())), (ValueError, dict(q=q[..., :32])),
        (ValueError, dict(k=q)), (ValueError, dict(q=q[0])), (ValueError, dict(table=None)),
        (ValueError, dict(table=table[1:])), (ValueError, dict(w_q=w.float())), (ValueError, dict(w_q=w[:32])),
        (ValueError, dict(pos=torch.zeros(5, 2, dtype=torch.int32, device="cuda"))),
        (ValueError, dict(pos=torch.zeros(5, 3, dtype=torch.int64, device="cuda"))),
        (ValueError, dict(q=None, k=None)),
        (ValueError, dict(q=_rand(1, 5, 4, 128)[..., ::2])),
        (AcError, dict(q=_rand(1 * 5 * 4 * 64 + 1)[1:].view(1, 5, 4, 64))),             # 2 bytes off
        (AcError, dict(q=_rand(1, 5, 4, 68)[..., :64])),                                # strides of 136 bytes
        (AcError, dict(q_out=_rand(1, 1, 1, 64).expand(1, 4, 5, 64))),                  # rows on top of one another
    ]
    for err, kw in bad:
        args = dict(q=q, k=k, **ok)
        args.update(kw)
        with pytest.raises(err):
            lay.ac_qk_norm_rope(**args)
    buf = _rand(1, 6, 4, 64)  # an output shifted by one token over its input
    with pytest.raises(AcError):
        lay.ac_qk_norm_rope(buf[:, :5], None, q_out=buf[:, 1:].transpose(1, 2), **ok)
    with pytest.raises(ValueError):
        lay.ac_qk_norm_rope_backward(q.transpose(1, 2), None, None, None, **ok)
    # the cache
    kp, vp, bt = _cache(lay, [20])
    st, kv = _starts([5]), torch.tensor([20], dtype=torch.int32).cuda()
    good = dict(q=q[0], k_pages=kp, v_pages=vp, block_table=bt, q_start=st, kv_len=kv)
    lay.ac_cache_attn(**good)
    for kw in (dict(k_pages=kp[:, :, :8]), dict(v_pages=vp[:1]), dict(block_table=bt.long()), dict(block_table=bt[0]),
               dict(q_start=st[:1]), dict(kv_len=kv.long()), dict(q=q[0].float()), dict(kv_len=kv.cpu())):
        with pytest.raises(ValueError):
            lay.ac_cache_attn(**{**good, **kw})
    with pytest.raises(AcError):
        lay.ac_cache_attn(**good, max_q=-1)
    f32 = _layer(heads=4, d=64, dtype="f32", page_size=16)
    p = torch.zeros(2, 4, 16, 64, device="cuda")
    with pytest.raises(AcError):  # the attention takes bf16
        f32.ac_cache_attn(torch.zeros(5, 4, 64, device="cuda"), p, p, bt, st, kv)
    plain = _layer(heads=4, kv_heads=2, d=64)
    with pytest.raises(AcError):  # a layer without a cache
        plain.ac_cache_attn(q[0], kp[:, :, :0], vp[:, :, :0], bt, st, kv)
    with pytest.raises(AcError):  # a layer without a rotation
        plain.ac_rope_table()
    from clustered_sparse_attention_head_b200.layer import AttnLayer
    small = AttnLayer(lay.cfg, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(AcError):
        small.ac_cache_attn(**good)
    torch.cuda.synchronize()
    assert lay.get_status() == 0
