"""The norm, rotation, gradients and append at sizes where the kernels take
their long runs of heads and every CTA several items, against 64-bit forms on
the GPU; and rows whose mean is large against their spread."""
import math

import pytest

import layer_util as U
from test_gpu_layer import ROPES, _bits, _cache, _cuda, _layer, _near, _rand, _starts  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _pos(n, grid):
    i = torch.arange(n, device="cuda")
    inside, cols = i < math.prod(grid), []
    for g in reversed(grid):
        cols.insert(0, torch.where(inside, i % g, -1))
        i = i // g
    return torch.stack(cols, -1)


def _close(got, ref, tol, what):
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), (what, float((err / tol.clamp(min=1e-300)).max()))


# heads, kv heads, d, type, norm, rotation, batch, tokens: more than 296 pieces of 256 threads' tokens
# and 32 heads, so that a run is 32 heads; 30 and 33 heads leave a last step of 2 and of 1, 40 a second
# run of 8
LONG = [
    (30, 30, 64, "bf16", "layer", "grid64", 2, 4801),
    (40, 8, 128, "bf16", "rms", "half", 1, 2503),
    (33, 3, 64, "f32", "rms", "line", 2, 2400),
    (40, 40, 128, "f32", "layer", "half", 1, 1301),
    (40, 40, 128, "bf16", "none", "grid", 1, 2400),
]


def _setup(case):
    hq, hk, d, dt, norm, rope, batch, n = case
    lay = _layer(heads=hq, kv_heads=hk, d=d, dtype=dt, norm=norm, **ROPES[rope])
    x = _rand(batch, n, hq + hk, d, dtype=lay.dtype, seed=3, scale=2.0)
    w = [_rand(d, dtype=lay.dtype, seed=13 + i) for i in range(4)]
    return lay, x[:, :, :hq], x[:, :, hq:], w, lay.ac_rope_table(), _pos(n, lay.cfg.rope_max)


def _ids(c):
    return "-".join(map(str, c))


@pytest.mark.parametrize("case", LONG, ids=_ids)
def test_forward(case):
    lay, q, k, (wq, wk, bq, bk), table, pos = _setup(case)
    qo, ko = lay.ac_qk_norm_rope(q, k, table=table, w_q=wq, w_k=wk, b_q=bq, b_k=bk)
    assert lay.get_status() == 0
    with torch.device("cuda"):
        for x, w, b, got in ((q, wq, bq, qo), (k, wk, bk, ko)):
            x, w, b = x.double(), w.double(), b.double()
            ref = U.forward(lay.cfg, x, w, b, pos)
            _close(got.transpose(1, 2), ref, U.forward_tol(lay.cfg, x, w, b, ref, lay.dtype), "forward")


def _bounds(cfg, g, x, w, pos, rows_a_lane):
    """dx, dw, db in 64 bits and how far the kernel's may be off before their
    rounding to the output's type.

    A turned gradient is two products, one sum and the table's rounding: 4 EPS32
    of turned = |a cos| + |b sin|.  x^ = (x - mean) r: r is off by 8 roundings (9 of a
    sum of squares, halved by the root, the root's own 2 and the products'), and the
    layer norm's mean by 10 of max|x|, which r scales.  dw and db add at most
    rows_a_lane terms in a lane, 32 lanes' sums one after the other and the rest in
    64 bits.  dx adds the two means, 10 roundings of sums of |e| and |e x^|."""
    with torch.device("cuda"):
        dx, dw, db = U.backward(cfg, g, x, w, pos)
        f, axis, mag = U.frequencies(cfg)
        still = (pos < 0).any(-1, keepdim=True)
        ang = pos.double()[..., axis] * f
        c = torch.where(still, 1.0, ang.cos().abs() * mag)[..., None, :]
        s = torch.where(still, 0.0, ang.sin().abs() * mag)[..., None, :]
        r2 = 2 * len(f)
        turned = g.abs()
        half = cfg.rope_layout == "half"
        lo, hi = (slice(0, r2 // 2), slice(r2 // 2, r2)) if half else (slice(0, r2, 2), slice(1, r2, 2))
        a, b = turned[..., lo].clone(), turned[..., hi].clone()
        turned[..., lo], turned[..., hi] = a * c + b * s, a * s + b * c
        if cfg.norm == "none":
            return (dx, 4 * U.EPS32 * turned), None, None
        n, r = U.normed(cfg, x)
        off = 10 * r * x.abs().amax(-1, keepdim=True) if cfg.norm == "layer" else 0.0  # of x^, in roundings
        chain = rows_a_lane + 32
        tdw = U.EPS32 * (turned * ((chain + 16) * n.abs() + off)).sum((0, 1, 2))
        tdb = U.EPS32 * ((chain + 8) * turned).sum((0, 1, 2))
        e = turned * w.abs()
        mean_e, mean_en = e.mean(-1, keepdim=True), (e * n.abs()).mean(-1, keepdim=True)
        tdx = U.EPS32 * r * (32 * (e + mean_e + n.abs() * mean_en) + off * (mean_en + n.abs() * mean_e))
        return (dx, tdx), (dw, tdw), (db, tdb)


@pytest.mark.parametrize("case", LONG, ids=_ids)
def test_backward(case):
    hq, hk, d, dt, norm, rope, batch, n = case
    lay, q, k, (wq, wk, bq, bk), table, pos = _setup(case)
    gq, gk = _rand(batch, hq, n, d, dtype=lay.dtype, seed=8), _rand(batch, hk, n, d, dtype=lay.dtype, seed=9)
    args = dict(table=table, w_q=wq, w_k=wk, b_q=bq, b_k=bk) if norm != "none" else dict(table=table)
    res = lay.ac_qk_norm_rope_backward(gq, gk, q, k, **args)
    assert lay.get_status() == 0
    lanes = torch.cuda.get_device_properties(0).multi_processor_count * 256 // (d // (8 if dt == "bf16" else 4))
    for name, g, x, w, heads in (("q", gq, q, wq, hq), ("k", gk, k, wk, hk)):
        # at least one CTA an SM in proportion to the heads, shared out in runs of up to 32 heads
        a_lane = 2 * batch * n * (hq + hk) / lanes + 64
        parts = _bounds(lay.cfg, g.double().transpose(1, 2), x.double(), w.double(), pos, a_lane)
        for out, part in zip((name, "w_" + name, "b_" + name), parts):
            if part is not None:
                ref, tol = part
                _close(res[out], ref, U.half_step(lay.dtype) * ref.abs() + tol, out)
    # a gradient of the last token's last head alone: it reaches dw and db
    if norm == "none":
        return
    one_q, one_k = torch.zeros_like(gq), torch.zeros_like(gk)
    one_q[-1, -1, -1], one_k[-1, -1, -1] = gq[-1, -1, -1], gk[-1, -1, -1]
    res = lay.ac_qk_norm_rope_backward(one_q, one_k, q, k, **args)
    for name, g, x, w in (("q", one_q, q, wq), ("k", one_k, k, wk)):
        last = (g.double().transpose(1, 2)[-1:, -1:, -1:], x.double()[-1:, -1:, -1:], w.double(), pos[-1:])
        dx, dw, db = _bounds(lay.cfg, *last, 1)
        for out, (ref, tol) in (("w_" + name, dw), ("b_" + name, db)):
            _close(res[out], ref, U.half_step(lay.dtype) * ref.abs() + tol, out)
        _close(res[name][-1:, -1:, -1:], dx[0], U.half_step(lay.dtype) * dx[0].abs() + dx[1], "dx")
        assert int((res[name] != 0).any(-1).sum()) == 1


@pytest.mark.parametrize("dt, hq, hk, d, norm, rope", [
    ("bf16", 13, 13, 128, "rms", "grid"),
    ("f32", 18, 9, 64, "layer", "half3"),
    ("bf16", 20, 10, 64, "none", "line"),
])
def test_append(dt, hq, hk, d, norm, rope):
    """New tokens of enough sequences that runs are 8 heads, heads that are no
    multiple of 8, and rows behind the last sequence."""
    lay = _layer(heads=hq, kv_heads=hk, d=d, dtype=dt, norm=norm, page_size=32, **ROPES[rope])
    new, kv = [900, 0, 1, 1300], [1000, 40, 17, 1300]
    kp, vp, bt = _cache(lay, kv)
    kp0, vp0 = kp.clone(), vp.clone()
    T = sum(new)
    x = _rand(T + 3, hq + 2 * hk, d, dtype=lay.dtype, seed=5)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    w = [_rand(d, dtype=lay.dtype, seed=20 + i) for i in range(4)]
    pos = _pos(max(kv), lay.cfg.rope_max)
    place = torch.cat([torch.arange(n - m, n) for m, n in zip(new, kv)]).cuda()
    # one axis ends before the sequences: its positions are given, so that none is past the table
    given = torch.cat([pos[place], pos[:3]]).int().contiguous() if len(lay.cfg.rope_max) == 1 else None
    qo = torch.full((T + 3, hq, d), 9.0, dtype=lay.dtype, device="cuda")
    lay.ac_cache_append(k, v, kp, vp, bt, _starts(new), torch.tensor(kv, dtype=torch.int32).cuda(), q=q,
                        table=lay.ac_rope_table(), pos=given, q_out=qo, w_q=w[0], w_k=w[1], b_q=w[2], b_k=w[3])
    assert lay.get_status() == 0
    assert (qo[T:] == 9).all()
    seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).cuda()
    pages = bt[seq, place // 32].long()
    with torch.device("cuda"):
        for xx, ww, bb, mine in ((q[:T], w[0], w[2], qo[:T]), (k[:T], w[1], w[3], kp[pages, :, place % 32])):
            xx, ww, bb = xx.double()[None], ww.double(), bb.double()
            ref = U.forward(lay.cfg, xx, ww, bb, pos[place])
            _close(mine, ref[0], U.forward_tol(lay.cfg, xx, ww, bb, ref, lay.dtype)[0], "append")
    assert torch.equal(vp[pages, :, place % 32], v[:T])
    keep = torch.ones(kp.shape[0], 32, dtype=torch.bool, device="cuda")
    keep[pages, place % 32] = False
    for pool, old in ((kp, kp0), (vp, vp0)):
        assert torch.equal(_bits(pool.transpose(1, 2)[keep]), _bits(old.transpose(1, 2)[keep]))


@pytest.mark.parametrize("dt, d, offset", [("bf16", 64, 40.0), ("f32", 128, 1000.0), ("f32", 64, -37.5)])
def test_layer_norm_of_rows_far_from_zero(dt, d, offset):
    lay = _layer(heads=3, d=d, dtype=dt, norm="layer", **ROPES["half" if d == 64 else "grid"])
    x = _rand(1, 50, 6, d, dtype=lay.dtype, seed=3, scale=2.0) + offset
    q, k = x[:, :, :3], x[:, :, 3:]
    w, b = _rand(d, dtype=lay.dtype, seed=4), _rand(d, dtype=lay.dtype, seed=5)
    table, pos = lay.ac_rope_table(), _pos(50, lay.cfg.rope_max)
    qo, ko = lay.ac_qk_norm_rope(q, k, table=table, w_q=w, w_k=w, b_q=b, b_k=b)
    g = _rand(1, 3, 50, d, dtype=lay.dtype, seed=8)
    res = lay.ac_qk_norm_rope_backward(g, g, q, k, table=table, w_q=w, w_k=w, b_q=b, b_k=b)
    with torch.device("cuda"):
        for name, xx, got in (("q", q, qo), ("k", k, ko)):
            xx, ww, bb = xx.double(), w.double(), b.double()
            ref = U.forward(lay.cfg, xx, ww, bb, pos)
            _close(got.transpose(1, 2), ref, U.forward_tol(lay.cfg, xx, ww, bb, ref, lay.dtype), "forward")
            parts = _bounds(lay.cfg, g.double().transpose(1, 2), xx, ww, pos, 150)
            for out, (ref, tol) in zip((name, "w_" + name, "b_" + name), parts):
                _close(res[out], ref, U.half_step(lay.dtype) * ref.abs() + tol, out)


def test_malformed_starts_stay_inside():
    """Starts that fall, overlap or leave the tensors: what lies on either side of
    the outputs and of the pools stays as it was, and the status word says which
    starts the call could not follow."""
    from clustered_sparse_attention_head_b200 import _abi
    lay = _layer(heads=2, d=64, page_size=16, causal_block=1, norm="none")
    kp0, vp0, bt = _cache(lay, [40, 40, 40])
    kv = torch.tensor([40, 40, 40], dtype=torch.int32).cuda()
    x = _rand(30, 2, 64, seed=7)
    pages = kp0.shape[0]
    # starts -> (attention's status, append's): the attention reports starts that fall or leave
    # [0, 30]; a token of the append is reported when its place is not in the cache, as places
    # below 0 are (70 new tokens of a sequence of 40)
    bad = _abi.AC_ERR_INVALID_ARG
    for starts, attn, append in (([-3, 10, 20, 30], bad, 0), ([0, 10, 20, 90], bad, bad), ([0, 20, 10, 30], bad, 0),
                                 ([5, 5, 5, 5], 0, 0), ([40, 50, 60, 70], bad, 0), ([0, 10, 20, 30], 0, 0)):
        st = torch.tensor(starts, dtype=torch.int32).cuda()
        out, qo = (torch.full((90, 2, 64), 4.0, dtype=lay.dtype, device="cuda") for _ in "ab")
        pools = [torch.full((3 * pages, 2, 16, 64), 4.0, dtype=lay.dtype, device="cuda") for _ in "kv"]
        kp, vp = (p[pages:2 * pages] for p in pools)
        kp.copy_(kp0)
        vp.copy_(vp0)
        lay.ac_cache_attn(x, kp, vp, bt, st, kv, out=out[30:60])
        assert lay.get_status() == attn, starts
        lay.ac_cache_append(x, x, kp, vp, bt, st, kv, q=x, q_out=qo[30:60])
        assert lay.get_status() == append, starts
        for t, n in ((out, 30), (qo, 30), (pools[0], pages), (pools[1], pages)):
            assert (t[:n] == 4).all() and (t[2 * n:] == 4).all(), starts
        # rows of no sequence
        a, b = max(0, min(starts[0], 30)), max(0, min(max(starts), 30))
        for t in (out, qo):
            assert (t[30:30 + a] == 4).all() and (t[30 + b:60] == 4).all(), starts
