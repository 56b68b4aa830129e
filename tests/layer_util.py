"""Plain 64-bit forms of the calls around the attention, for their tests."""
from __future__ import annotations

import math

import torch

EPS32 = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def frequencies(cfg):
    """Angle per position of every pair, the pair's axis, the magnitude."""
    f, axis, mag = [], [], 1.0
    for a, dim in enumerate(cfg.rope_dims):
        for j in range(dim // 2):
            theta = cfg.rope_theta
            if cfg.rope_scaling == "ntk":
                theta *= cfg.rope_factor ** (dim / (dim - 2))
            w = theta ** (-2 * j / dim)
            if cfg.rope_scaling == "linear":
                w /= cfg.rope_factor
            if cfg.rope_scaling == "yarn":
                turns = cfg.rope_orig * w / (2 * math.pi)
                keep = (turns - cfg.rope_beta_slow) / (cfg.rope_beta_fast - cfg.rope_beta_slow)
                keep = min(1.0, max(0.0, keep))
                w = w * keep + w / cfg.rope_factor * (1 - keep)
                mag = 0.1 * math.log(cfg.rope_factor) + 1
            f.append(w)
            axis.append(a)
    return torch.tensor(f, dtype=torch.float64), torch.tensor(axis, dtype=torch.long), mag


def grid_pos(n, grid):
    """Row-major coordinates of 0 .. n - 1; -1 behind the grid."""
    out = torch.full((n, len(grid)), -1, dtype=torch.long)
    cells = math.prod(grid)
    for i in range(min(n, cells)):
        k = i
        for a in reversed(range(len(grid))):
            out[i, a] = k % grid[a]
            k //= grid[a]
    return out


def turn(cfg, x, pos, back=False):
    """x [..., n, heads, d] float64, pos [..., n, axes]."""
    if not cfg.rope_dims:
        return x
    f, axis, mag = frequencies(cfg)
    ang = pos.double()[..., axis] * f
    c, s = mag * ang.cos(), mag * ang.sin()
    if back:
        s = -s
    still = (pos < 0).any(-1, keepdim=True)
    c, s = torch.where(still, 1.0, c)[..., None, :], torch.where(still, 0.0, s)[..., None, :]
    r = 2 * len(f)
    y = x.clone()
    lo = slice(0, r // 2) if cfg.rope_layout == "half" else slice(0, r, 2)
    hi = slice(r // 2, r) if cfg.rope_layout == "half" else slice(1, r, 2)
    a, b = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = a * c - b * s, a * s + b * c
    return y


def normed(cfg, x):
    if cfg.norm == "none":
        return x, None
    if cfg.norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = 1 / (x.square().mean(-1, keepdim=True) + cfg.eps).sqrt()
    return x * r, r


def forward(cfg, x, w, b, pos):
    """x [batch, n, heads, d], pos [n, axes] or [batch, n, axes] -> the same layout."""
    y, _ = normed(cfg, x)
    if cfg.norm != "none":
        y = y * w if w is not None else y
        y = y + b if b is not None else y
    return turn(cfg, y, pos)


def forward_tol(cfg, x, w, b, ref, dtype):
    """Half a step of the output's type, and the fp32 path: sums of d <= 128
    elements are at most 4 + 5 additions deep, so mean and mean square are within
    10 roundings, their root, quotient and products 6 more, and the pair's two
    products 3 more with the table's own rounding: under 32 roundings of the
    row's largest intermediate value, r max|x| max|w| + max|b|, times 2 for a
    pair and times the table's magnitude (< 1.5)."""
    big = x.abs().amax(-1, keepdim=True)
    if cfg.norm != "none":
        _, r = normed(cfg, x)
        # the layer norm's mean is off by 10 roundings of max|x| before r scales it
        big = big * r * (1.0 if w is None else w.abs().max()) + (0.0 if b is None else b.abs().max())
    return half_step(dtype) * ref.abs() + 32 * 2 * 1.5 * EPS32 * big


def backward(cfg, g, x, w, pos):
    """g in the layout of x -> dx, dw, db."""
    g = turn(cfg, g, pos, back=True)
    if cfg.norm == "none":
        return g, None, None
    n, r = normed(cfg, x)
    dw, db = (g * n).sum((0, 1, 2)), g.sum((0, 1, 2))
    e = g if w is None else g * w
    dx = e - n * (e * n).mean(-1, keepdim=True)
    if cfg.norm == "layer":
        dx = dx - e.mean(-1, keepdim=True)
    return dx * r, dw, db


def attend(cfg, q, k_pages, v_pages, table, q_start, kv_len, max_q=None, max_kv=None):
    """q [tokens, heads, d] and the pools, as float64 with the cache's own
    values; returns out, lse, and per output element the weighted mean of |v| and
    per row the largest sum |q k| scale (for the tolerance)."""
    T, H, D = q.shape
    g = H // k_pages.shape[1]
    page = k_pages.shape[2]
    scale = cfg.scale or D ** -0.5
    out, absv = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    big = torch.zeros(T, H, dtype=torch.float64)
    seen = torch.zeros(T, dtype=torch.bool)
    for s in range(len(kv_len)):
        new, n = int(q_start[s + 1] - q_start[s]), int(kv_len[s])
        p0 = n - new
        n = min(n, max_kv if max_kv is not None else n, table.shape[1] * page)
        j = torch.arange(n)
        pages = table[s][j // page].long().clamp(0, k_pages.shape[0] - 1)
        k, v = k_pages[pages, :, j % page], v_pages[pages, :, j % page]   # [n, heads, d]
        for i in range(min(new, max_q if max_q is not None else new)):
            p, t = p0 + i, int(q_start[s]) + i
            seen[t] = True
            ok = torch.ones(n, dtype=torch.bool)
            if cfg.causal_block:
                ok &= j // cfg.causal_block <= p // cfg.causal_block  # floor, also below 0
            if cfg.window:
                ok &= j > p - cfg.window
            if not ok.any():
                continue
            kk, vv = k[ok].repeat_interleave(g, 1), v[ok].repeat_interleave(g, 1)
            sc = torch.einsum("hd,nhd->hn", q[t], kk) * scale
            big[t] = torch.einsum("hd,nhd->hn", q[t].abs(), kk.abs()).amax(-1) * scale
            lse[t] = torch.logsumexp(sc, -1)
            w = torch.softmax(sc, -1)
            out[t] = torch.einsum("hn,nhd->hd", w, vv)
            absv[t] = torch.einsum("hn,nhd->hd", w, vv.abs())
    return out, lse, absv, big, seen


def attend_tol(ref, absv, big):
    """Every weight is off by its rounding to bf16 (2^-8), by 2^x (a cubic within
    1.1e-4) and by the score's fp32 error, at most 128 + 8 roundings of sum |q k|
    scale in its exponent, which numerator and denominator both carry; the output
    by half a step of bf16."""
    return (2.0 ** -8 + 2 * 1.1e-4) * absv + 2 * 136 * EPS32 * big[..., None] * absv + 2.0 ** -8 * ref.abs() + 1e-30
